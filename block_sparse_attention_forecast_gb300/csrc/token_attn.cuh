// The work of the attention of many new tokens per sequence (token_attn.cu) and its division among the
// CTAs. The lengths are read on the device, so that a captured call serves any batch.
//
// An entry e = b*G + g is one KV group of one sequence. Its new tokens are cut into items of tpi tokens
// (times the group's H query heads: at most 128 or 256 rows); an item attends nctx 64-token blocks of
// the cache and the new tokens' blocks up to its own last token (causal), or all of them (tree), two
// blocks (a key tile) at a time. Three ways to share the items out:
//   whole items   position u of all items, entry by entry, the longest of an entry first: CTA c takes item c, and
//                 then whatever item is next, from a counter. CTAs that run at one time attend the same
//                 keys, and the last items are the short ones;
//   key tiles     position u of all items' key tiles, each item's behind item_tiles positions that stand for its
//                 beginning and end: each CTA takes an equal range of positions, whatever items they belong to, and
//                 first those of the items that begin in it. So all start at their caches' first keys and those
//                 that share a cache meet in L2 (next turns of 4 sequences over up to 32768 tokens, 0.44 GB of
//                 caches: 1.1 GB of DRAM reads and 555 us; in the order of the positions 2.9 GB and 586 us);
//   equal parts   where there are fewer items than CTAs and they are about as long: each item to the same number
//                 of CTAs, so that no CTA begins and ends more than one.
// An item that is cut leaves partial results, which token_attn_join_kernel joins.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace sparda {
namespace tok {

typedef unsigned long long u64;
typedef uint32_t u32;

struct Entry {
  int n;        // new tokens, 0: none, or a length out of range
  int P;        // tokens in the cache
  int nctx;     // blocks of the cache that are attended
  int row0;     // packed prompts: the sequence's first row
  bool bad;     // a length out of range
};

struct Item {
  int e;
  Entry en;
  int tok0;     // first token of the item
  int nblk;     // blocks attended, the cache's first
  int nkt;      // key tiles: ceil(nblk / 2)
  int k0, k1;   // the key tiles of this segment
  int slot;     // partial result it goes to; -1: the whole item
  u32 start;    // position of its first key tile (key-tile division)
};

__device__ __forceinline__ Entry load_entry(const TokenAttnArgs& a, int e) {
  const int b = a.by_G.div(e);
  Entry en;
  en.P = a.ctx_len ? a.ctx_len[b] : 0;
  const int cnt = a.idx ? a.cnt[e] : 0;
  if (a.cu) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    en.row0 = lo;
    en.n = hi - lo;
    en.bad = lo < 0 || hi < lo || hi > a.n_rows;
  } else {
    en.row0 = 0;
    en.n = a.n_nodes ? a.n_nodes[b] : a.n_rows;
    en.bad = en.n < 0 || en.n > a.n_rows;
  }
  en.bad = en.bad || en.P < 0 || en.P > a.max_ctx;
  if (en.bad) en.n = en.P = 0;
  en.nctx = a.idx ? min(max(cnt, 0), a.kslots) : (en.P + kBlock - 1) / kBlock;
  return en;
}

__device__ __forceinline__ int n_items(const TokenAttnArgs& a, const Entry& en) { return a.by_item.div(en.n + a.by_item.d - 1); }

__device__ __forceinline__ int item_blocks(const TokenAttnArgs& a, const Entry& en, int i, int tpi) {
  const int last = (a.causal ? min((i + 1) * tpi, en.n) : en.n) - 1;
  return en.nctx + last / kBlock + 1;
}

// sum over 0 <= i < n of floor((a*i + b) / m), by the Euclidean recurrence on the lattice points under a line
__device__ __forceinline__ u32 floor_sum(u32 n, u32 m, u32 a, u32 b) {
  u32 s = 0;
  while (n > 0) {
    s += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
    a %= m;
    b %= m;
    const u32 top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const u32 t = m;
    m = a;
    a = t;
  }
  return s;
}

// Positions of an entry's items before item i (i < its number of items). Key-tile division only, whose few
// items (split_items at most) of at most 2^24 / 128 + 2^11 key tiles each keep every sum below 2^32.
__device__ __forceinline__ u32 tiles_before(const TokenAttnArgs& a, const Entry& en, int i, int tpi) {
  const u32 own = i * a.item_tiles;
  if (!a.causal) return own + (u32)i * ((item_blocks(a, en, 0, tpi) + 1) / 2);
  return own + floor_sum(i, 2 * kBlock, tpi, kBlock * (en.nctx + 2) + tpi - 1);
}
__device__ __forceinline__ u32 entry_tiles(const TokenAttnArgs& a, const Entry& en, int tpi) {
  const int ni = n_items(a, en);
  return ni == 0 ? 0 : tiles_before(a, en, ni - 1, tpi) + a.item_tiles + (item_blocks(a, en, ni - 1, tpi) + 1) / 2;
}

// W positions in n even parts: the first of part c, and the part of a position.
struct Parts {
  u32 q, r;     // r parts of q + 1, then parts of q
  __device__ __forceinline__ Parts(u32 W, u32 n) : q(W / n), r(W % n) {}
  __device__ __forceinline__ u32 start(u32 c) const { return q * c + min(c, r); }
  __device__ __forceinline__ u32 owner(u32 pos) const {
    return pos < r * (q + 1) ? pos / (q + 1) : r + (pos - r * (q + 1)) / q;
  }
};

// The segments of CTA c, in order, for one warp (every lane calls every function). Lane l holds entry e0 + l.
struct Segments {
  const TokenAttnArgs& a;
  const int tpi, lane;
  const u32 c;
  bool split;          // key-tile division
  u32 per_item;        // equal parts: CTAs per item; else 0
  u32 n_ctas, total;   // CTAs that take part; items or key tiles
  u32 base, incl, sum; // 32 entries at a time: the weight before them, up to this lane's, of all
  Entry mine;
  int e0;
  u32 pos, end;
  int segments;        // given out so far (whole items, equal parts)
  u32 first, rest;     // key-tile division: the range's start; where its first item ends, if that is left for last

  __device__ Segments(const TokenAttnArgs& args, int tokens_per_item, int ln, int cta)
      : a(args), tpi(tokens_per_item), lane(ln), c(cta) {}

  __device__ __forceinline__ void fetch() {
    mine = Entry{0, 0, 0, 0, false};
    if (e0 + lane < a.n_entries) mine = load_entry(a, e0 + lane);
  }
  __device__ __forceinline__ void weigh() {
    incl = split ? entry_tiles(a, mine, tpi) : (u32)n_items(a, mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u32 up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    sum = __shfl_sync(0xffffffffu, incl, 31);
  }
  __device__ __forceinline__ Entry entry(int l) const {
    Entry en;
    en.n = __shfl_sync(0xffffffffu, mine.n, l);
    en.P = __shfl_sync(0xffffffffu, mine.P, l);
    en.nctx = __shfl_sync(0xffffffffu, mine.nctx, l);
    en.row0 = __shfl_sync(0xffffffffu, mine.row0, l);
    en.bad = false;
    return en;
  }

  // the division; `report`: sets the error word for bad lengths
  __device__ __forceinline__ void init(bool report) {
    u32 items = 0, longest = 0;
    bool bad = false;
    for (e0 = 0; e0 < a.n_entries; e0 += 32) {
      fetch();
      const int ni = n_items(a, mine);
      items += ni;
      if (ni > 0) longest = max(longest, (u32)(item_blocks(a, mine, ni - 1, tpi) + 1) / 2);
      bad = bad || mine.bad;
    }
    items = __reduce_add_sync(0xffffffffu, items);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (report && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    split = false;
    per_item = 0;
    total = items;
    n_ctas = a.n_ctas;
    // Whole items in one round take as long as the longest one; in several about as long as an even share, the part
    // of a round that stays empty, and half of what the longest has over the average. Cutting costs join_tiles or
    // cut_tiles key tiles beside an even share.
    if (items < (u32)a.split_items && longest > (items <= n_ctas ? a.join_tiles : a.cut_tiles / 2)) {
      u32 tiles = 0;
      for (e0 = 0; e0 < a.n_entries; e0 += 32) {
        if (a.n_entries > 32) fetch();
        tiles += entry_tiles(a, mine, tpi);
      }
      tiles = __reduce_add_sync(0xffffffffu, tiles);
      if (items <= n_ctas) {
        split = longest > tiles / n_ctas + a.join_tiles;
      } else {
        const u32 average = tiles / items, idle = n_ctas - 1 - (items + n_ctas - 1) % n_ctas;   // CTAs in the last round
        split = average * idle / n_ctas + (max(longest, average) - average) / 2 > a.cut_tiles;
      }
      if (split) {
        const u32 ctas = min(n_ctas, max(1u, tiles / a.min_tiles));
        // a range's second segment costs as much as seg_tiles key tiles (its start, its own partial result)
        const u32 k = min(n_ctas / items, max(1u, longest / a.min_tiles));
        if (k > 1 && (longest + k - 1) / k <= tiles / ctas + a.seg_tiles) {
          split = false;
          per_item = k;
        } else {
          total = tiles;
          n_ctas = ctas;
        }
      }
    }
    e0 = 0;
    base = 0;
    if (a.n_entries > 32) fetch();
    weigh();
    segments = 0;
    pos = end = first = rest = 0;
    if (split && c < n_ctas) {
      const Parts parts(total, n_ctas);
      pos = first = parts.start(c);
      end = parts.start(c + 1);
    }
  }

  // the lane of the entry of position p < total (not below one asked for before), and the position inside it
  __device__ __forceinline__ int seek(u32 p, u32& off) {
    while (p >= base + sum) {
      base += sum;
      e0 += 32;
      fetch();
      weigh();
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, base + incl > p)) - 1;
    const u32 before = __shfl_sync(0xffffffffu, incl, (l + 31) & 31);
    off = p - base - (l == 0 ? 0 : before);
    return l;
  }

  __device__ __forceinline__ void fill(Item& it, int l, const Entry& en, int i) const {
    it.e = e0 + l;
    it.en = en;
    it.tok0 = i * tpi;
    it.nblk = item_blocks(a, en, i, tpi);
    it.nkt = (it.nblk + 1) / 2;
    it.k1 = it.nkt;
    it.slot = -1;
  }

  // The counter of whole items. In a call it is taken from `total` times in all (each CTA that has a first item goes on
  // until what it takes is past the last one), and the last time leaves it at zero.
  __device__ __forceinline__ u32 take() const {
    u32 u = 0;
    if (lane == 0) u = atomicInc(a.queue, total - 1);
    return __shfl_sync(0xffffffffu, u, 0);
  }

  __device__ __forceinline__ bool next(Item& it) {
    u32 off;
    if (per_item > 0) {
      const u32 i = c / per_item, part = c - i * per_item;
      if (segments++ > 0 || i >= total) return false;
      const int l = seek(i, off);
      const Entry en = entry(l);
      fill(it, l, en, n_items(a, en) - 1 - (int)off);
      const u32 k = min(per_item, (u32)it.nkt);
      if (part >= k) return false;
      const Parts parts(it.nkt, k);
      it.k0 = parts.start(part);
      it.k1 = parts.start(part + 1);
      if (k > 1) it.slot = 2 * c;
      return true;
    }
    if (!split) {
      u32 u = c;
      if (segments++ > 0) u = n_ctas + take();
      if (u >= total || u < pos) return false;               // (the latter: a workspace that was not zeroed)
      pos = u;
      const int l = seek(u, off);
      const Entry en = entry(l);
      fill(it, l, en, n_items(a, en) - 1 - (int)off);
      it.k0 = 0;
      return true;
    }
    for (;;) {
      if (pos >= end) {
        if (rest <= first) return false;
        pos = first;
        end = rest;
        rest = 0;
        if (e0 > 0) {
          e0 = 0;
          base = 0;
          fetch();
          weigh();
        }
      }
      const int at = seek(pos, off);
      const Entry en = entry(at);
      // the last item with tiles_before <= off, 32 candidates at a time
      int lo = 0, len = n_items(a, en);
      while (len > 1) {
        const int step = (len + 31) / 32;
        const int i = lo + lane * step;
        const bool below = i < lo + len && tiles_before(a, en, min(i, lo + len - 1), tpi) <= off;
        const int l = 31 - __clz(__ballot_sync(0xffffffffu, below));
        const int stop = lo + len;
        lo += l * step;
        len = min(step, stop - lo);
      }
      fill(it, at, en, lo);
      const u32 in = off - tiles_before(a, en, lo, tpi), left = in + (end - pos);   // positions of the item: first, end
      it.start = pos - in + a.item_tiles;
      it.k0 = (int)(max(in, a.item_tiles) - a.item_tiles);
      it.k1 = (int)min((u32)it.nkt, max(left, a.item_tiles) - a.item_tiles);
      pos = it.start + it.nkt;                               // (the next item, if the range goes on)
      if (it.k0 == it.k1) continue;                          // the range ends before its first key tile
      if (it.k0 > 0 && pos < end) {
        rest = pos;
        continue;
      }
      if (it.k0 > 0 || it.k1 < it.nkt) it.slot = 2 * c + (it.start - a.item_tiles > first ? 1 : 0);
      return true;
    }
  }

  // Whether the segment's item is cut, and what this CTA does to join it: all CTAs c1 .. c1+k-1 that have a part
  // of it join an equal share of its rows. CTA q's part is in slot 2q, that of c1 in first_slot.
  __device__ __forceinline__ bool join(const Item& it, TokenJoin& j) const {
    if (it.slot < 0) return false;
    u32 c1;
    if (per_item > 0) {
      c1 = c - c % per_item;
      j.k = min(per_item, (u32)it.nkt);
      j.first_slot = 2 * c1;
    } else {
      const Parts parts(total, n_ctas);
      c1 = parts.owner(it.start);
      j.k = parts.owner(it.start + it.nkt - 1) - c1 + 1;
      j.first_slot = 2 * c1 + (parts.start(c1) < it.start - a.item_tiles ? 1 : 0);
    }
    j.c1 = c1;
    const u32 rows = min(tpi, it.en.n - it.tok0) * a.H;
    j.r0 = (int)(rows * (c - c1) / j.k);
    j.r1 = (int)(rows * (c - c1 + 1) / j.k);
    const int b = a.by_G.div(it.e);
    j.g = it.e - b * a.G;
    j.out_row = (a.cu ? it.en.row0 : b * a.n_rows) + it.tok0;
    return true;
  }
};

}  // namespace tok
}  // namespace sparda
