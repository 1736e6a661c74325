// The work of the attention of many new tokens per sequence (token_attn.cu) and its division among the
// CTAs. The lengths are read on the device, so that a captured call serves any batch.
//
// An entry e = b*G + g is one KV group of one sequence. Its new tokens are cut into items of tpi tokens
// (times the group's H query heads: at most 128 or 256 rows); an item attends nctx 64-token blocks of
// the cache and the new tokens' blocks up to its own last token (causal), or all of them (tree), two
// blocks (a key tile) at a time. Two ways to share the items out:
//   whole items   position u of all items, entry by entry, the longest of an entry first, dealt out to the
//                 CTAs in snake order (0 .. n-1, n-1 .. 0, ...): CTAs that run at one time attend the
//                 same keys, and the last items are the short ones;
//   key tiles     position u of all items' key tiles: CTA c of n takes the positions W*c/n .. W*(c+1)/n,
//                 whatever items they belong to. An item cut by such a border leaves partial results,
//                 which token_attn_join_kernel joins.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace sparda {
namespace tok {

typedef unsigned long long u64;

struct Entry {
  int n;        // new tokens, 0: none, or a length out of range
  int P;        // tokens in the cache
  int nctx;     // blocks of the cache that are attended
  int row0;     // packed prompts: the sequence's first row
  bool bad;     // a length out of range
};

struct Item {
  int b, g;
  Entry en;
  int tok0;     // first token of the item
  int nblk;     // blocks attended, the cache's first
  int nkt;      // key tiles: ceil(nblk / 2)
  int k0, k1;   // the key tiles of this segment
  int slot;     // partial result it goes to; -1: the whole item
  u64 start;    // key-tile position of its first key tile (key-tile division)
};

__device__ __forceinline__ Entry load_entry(const TokenAttnArgs& a, int e) {
  const int b = e / a.G;
  Entry en;
  en.P = a.ctx_len ? a.ctx_len[b] : 0;
  en.bad = en.P < 0 || en.P > a.max_ctx;
  if (a.cu) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    en.row0 = lo;
    en.n = hi - lo;
    en.bad = en.bad || lo < 0 || hi < lo || hi > a.n_rows;
  } else {
    en.row0 = 0;
    en.n = a.n_nodes ? a.n_nodes[b] : a.n_rows;
    en.bad = en.bad || en.n < 0 || en.n > a.n_rows;
  }
  if (en.bad) en.n = en.P = 0;
  en.nctx = a.idx ? min(max(a.cnt[e], 0), a.kslots) : (en.P + kBlock - 1) / kBlock;
  return en;
}

__device__ __forceinline__ int n_items(const Entry& en, int tpi) { return (en.n + tpi - 1) / tpi; }

__device__ __forceinline__ int item_blocks(const TokenAttnArgs& a, const Entry& en, int i, int tpi) {
  const int last = (a.causal ? min((i + 1) * tpi, en.n) : en.n) - 1;
  return en.nctx + last / kBlock + 1;
}

// sum over 0 <= i < n of floor((a*i + b) / m), by the Euclidean recurrence on the lattice points under a line
__device__ __forceinline__ u64 floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  u64 s = 0;
  while (n > 0) {
    s += (u64)(a / m) * ((u64)n * (n - 1) / 2) + (u64)(b / m) * n;
    a %= m;
    b %= m;
    const u64 top = (u64)a * n + b;
    if (top < m) break;
    n = (unsigned)(top / m);
    b = (unsigned)(top % m);
    const unsigned t = m;
    m = a;
    a = t;
  }
  return s;
}

// key tiles of an entry's items before item i (i < its number of items)
__device__ __forceinline__ u64 tiles_before(const TokenAttnArgs& a, const Entry& en, int i, int tpi) {
  if (!a.causal) return (u64)i * ((item_blocks(a, en, 0, tpi) + 1) / 2);
  return floor_sum(i, 2 * kBlock, tpi, kBlock * (en.nctx + 2) + tpi - 1);
}
__device__ __forceinline__ u64 entry_tiles(const TokenAttnArgs& a, const Entry& en, int tpi) {
  const int ni = n_items(en, tpi);
  return ni == 0 ? 0 : tiles_before(a, en, ni - 1, tpi) + (item_blocks(a, en, ni - 1, tpi) + 1) / 2;
}

// Key-tile division: CTAs that take part, the first position of CTA c, and the CTA of a position.
__device__ __forceinline__ u64 range_start(u64 W, int n, int c) { return W * c / n; }
__device__ __forceinline__ int range_owner(u64 W, int n, u64 pos) { return (int)(((pos + 1) * n - 1) / W); }

// Walks the entries for one warp (every lane calls every function): positions asked for must not decrease.
struct Cursor {
  const TokenAttnArgs& a;
  const int tpi, lane;
  bool split;        // key-tile division
  int n_ctas;        // that take part
  u64 total;         // items or key tiles
  u64 base, incl, sum;
  int e0;

  __device__ Cursor(const TokenAttnArgs& args, int tokens_per_item, int ln) : a(args), tpi(tokens_per_item), lane(ln) {}

  __device__ __forceinline__ u64 weight(int e) const {
    if (e >= a.n_entries) return 0;
    const Entry en = load_entry(a, e);
    return split ? entry_tiles(a, en, tpi) : (u64)n_items(en, tpi);
  }

  // totals and the division; `report`: this warp sets the error word for bad lengths
  __device__ __forceinline__ void init(bool report) {
    u64 items = 0, tiles = 0;
    bool bad = false;
    for (int e = lane; e < a.n_entries; e += 32) {
      const Entry en = load_entry(a, e);
      items += n_items(en, tpi);
      tiles += entry_tiles(a, en, tpi);
      bad = bad || en.bad;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      items += __shfl_xor_sync(0xffffffffu, items, o);
      tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    }
    if (report && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    split = items < (u64)a.split_items;
    total = split ? tiles : items;
    n_ctas = split ? (int)min((u64)a.n_ctas, max((u64)1, tiles / a.min_tiles)) : a.n_ctas;
    e0 = 0;
    base = 0;
    load();
  }

  __device__ __forceinline__ void load() {
    incl = weight(e0 + lane);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    sum = __shfl_sync(0xffffffffu, incl, 31);
  }

  // the entry of position `pos` < total, and the position inside it
  __device__ __forceinline__ int seek(u64 pos, u64& off) {
    while (pos >= base + sum) {
      base += sum;
      e0 += 32;
      load();
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, base + incl > pos)) - 1;
    off = pos - base - (l == 0 ? 0 : __shfl_sync(0xffffffffu, incl, (l + 31) & 31));
    return e0 + l;
  }

  __device__ __forceinline__ void fill(Item& it, int e, const Entry& en, int i) const {
    it.b = e / a.G;
    it.g = e % a.G;
    it.en = en;
    it.tok0 = i * tpi;
    it.nblk = item_blocks(a, en, i, tpi);
    it.nkt = (it.nblk + 1) / 2;
  }

  // whole items: the item at position pos
  __device__ __forceinline__ void item_at(u64 pos, Item& it) {
    u64 off;
    const int e = seek(pos, off);
    const Entry en = load_entry(a, e);
    fill(it, e, en, n_items(en, tpi) - 1 - (int)off);
    it.k0 = 0;
    it.k1 = it.nkt;
    it.slot = -1;
  }

  // key tiles: the item that holds key-tile position pos; it.k0 is pos's tile in it
  __device__ __forceinline__ void tile_at(u64 pos, Item& it) {
    u64 off;
    const int e = seek(pos, off);
    const Entry en = load_entry(a, e);
    // the last item with tiles_before <= off, 32 candidates at a time
    int lo = 0, len = n_items(en, tpi);
    while (len > 1) {
      const int step = (len + 31) / 32;
      const int i = lo + lane * step;
      const bool below = i < lo + len && tiles_before(a, en, min(i, lo + len - 1), tpi) <= off;
      const int l = 31 - __clz(__ballot_sync(0xffffffffu, below));
      const int end = lo + len;
      lo += l * step;
      len = min(step, end - lo);
    }
    fill(it, e, en, lo);
    const u64 before = tiles_before(a, en, lo, tpi);
    it.k0 = (int)(off - before);
    it.k1 = it.nkt;
    it.start = pos - it.k0;
    it.slot = -1;
  }
};

// The segments of CTA c, in order.
struct Segments {
  Cursor cur;
  const int c;
  u64 pos, end, first;
  int round;

  __device__ Segments(const TokenAttnArgs& a, int tpi, int lane, int cta) : cur(a, tpi, lane), c(cta) {}
  __device__ __forceinline__ void init(bool report) {
    cur.init(report);
    round = 0;
    if (cur.split) {
      pos = end = 0;
      if (c < cur.n_ctas) {
        pos = range_start(cur.total, cur.n_ctas, c);
        end = range_start(cur.total, cur.n_ctas, c + 1);
      }
      first = pos;
    }
  }
  __device__ __forceinline__ bool next(Item& it) {
    if (cur.split) {
      if (pos >= end) return false;
      cur.tile_at(pos, it);
      const u64 left = end - pos;
      if ((u64)(it.k1 - it.k0) > left) it.k1 = it.k0 + (int)left;
      if (it.k0 > 0 || it.k1 < it.nkt) it.slot = 2 * c + (pos == first ? 0 : 1);
      pos += it.k1 - it.k0;
      return true;
    }
    const u64 u = (u64)round * cur.n_ctas + ((round & 1) ? cur.n_ctas - 1 - c : c);
    ++round;
    if (u >= cur.total) return false;
    cur.item_at(u, it);
    return true;
  }
};

}  // namespace tok
}  // namespace sparda
