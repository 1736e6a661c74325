// Internal launch interface between the C ABI (api.cu) and the kernel translation units.
// Every struct is passed to its kernel by value; pointers are device (or UVA) addresses.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace sparda {

// The scores-only selection of the fused launch hands out its work dynamically for up to this
// many (sequence, group)s: their forecasts must fit in shared memory beside its ring.
constexpr int kSelDynMaxGroups = 35;

struct AppendArgs {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  __nv_bfloat16* ck;
  __nv_bfloat16* hot_k;
  __nv_bfloat16* hot_v;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  const int32_t* seq_len;
  int* err;
  int G, max_ctx, W_cap, on_host;
};

struct CompressArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* hot_k;
  __nv_bfloat16* ck;
  const int32_t* seq_len;
  int* err;
  int G, max_ctx, W_cap, on_host;
};

struct ProjectArgs {
  const __nv_bfloat16* W;
  const __nv_bfloat16* h;
  __nv_bfloat16* f;
  int rows, hidden, batch;
};

struct SelectArgs {
  const __nv_bfloat16* ck;
  const __nv_bfloat16* f;        // forecast [B, G, d]
  const int32_t* seq_len;
  int32_t* idx;                  // [B, G, topk+2]
  int32_t* cnt;                  // [B, G]
  float* block_scores;           // workspace [B*G, nb_cap]
  unsigned* counters;            // workspace [B*G], zero between calls
  int* err;
  int G, W_cap, max_ctx, nb_cap, topk, chunk_blocks;
  int n_units;                   // B*G*nb_cap, set by the launcher
  int do_topk = 1;               // 0: leave the block scores for a later top-k (decode prologue)
  // scores-only selection of the fused launch with at most 35 (sequence, group)s: sub-chunks
  // are handed out from queue[0] (queue[1] counts the producers that finished); nullptr:
  // contiguous ranges
  unsigned* queue = nullptr;
  // optional: a buffer the next launches read (the next layer's forecast weights), pulled
  // into L2 by the selection CTAs once they have issued their last load
  const void* l2_prefetch = nullptr;
  size_t l2_prefetch_bytes = 0;
};

struct AttnArgs {
  const __nv_bfloat16* q;        // [B, G*H, d]
  const int32_t* idx;
  const int32_t* cnt;
  const int32_t* seq_len;
  __nv_bfloat16* out;            // [B, G*H, d]
  float* part_o;                 // workspace [B*G, n_split, H, d]
  float* part_ml;                // workspace [B*G, n_split, 2, H]
  unsigned* counters;            // workspace [B*G]
  int* err;
  int G, max_ctx, kslots, n_split, offload;
  int n_units;                   // B*G*kslots, set by the launcher
  // > 0: the grid is seg_per_group CTAs per (sequence, group), each taking an equal share of
  // that group's slots (no CTA spans two groups); 0: contiguous balanced unit ranges
  int seg_per_group = 0;
  // offload with the block cache: idx entry u's staged block is in row block
  // (bg * stage_slots + stage_slot[u]) of the staging map; nullptr: row block u
  const int32_t* stage_slot = nullptr;
  int stage_slots = 0;
  uint32_t tl_launch = 0;        // launch number for the timeline build's records
  void* tl_buf = nullptr;        // the timeline build's record store
  // block mass (the standalone launch): (max, sum) [B*G, kslots, 4, 16] and the final max and
  // sum [B*G, 2, 16]; nullptr: not wanted
  float2* stats = nullptr;
  float* ml = nullptr;
  float* mass = nullptr;         // [max_batch, G, max_ctx/64]: added to by the cluster form itself
};

struct MultiheadArgs {
  const __nv_bfloat16* q;        // [B, G*H, d]
  const int32_t* seq_len;
  int32_t* idx;                  // [B, G, topk+2]
  int32_t* cnt;                  // [B, G]
  float* block_scores;           // workspace [B*G, nb_cap]
  int* err;
  int G, W_cap, max_ctx, nb_cap, topk;
  int cluster;                   // CTAs per (sequence, group): one thread-block cluster
  int tiles_per_cta;             // 64-window tiles a CTA holds at most (shared-memory sizing)
};

struct PrefetchArgs {
  const __nv_bfloat16* hk;       // host cache (UVA) [B, G, max_ctx, d]
  const __nv_bfloat16* hv;
  const int32_t* idx;
  const int32_t* cnt;
  const int32_t* seq_len;
  __nv_bfloat16* sk;             // staging [B, G, kslots, 64, d]
  __nv_bfloat16* sv;
  int* err;
  int B, G, max_ctx, kslots;
};

// The cross-step block cache of an offloaded layer (prefetch.cu).
struct CacheArgs {
  const __nv_bfloat16* hk;       // host cache (UVA) [B, G, max_ctx, d]
  const __nv_bfloat16* hv;
  const int32_t* idx;            // [B, G, kslots]
  const int32_t* cnt;            // [B, G]
  const int32_t* seq_len;
  int32_t* cache_blocks;         // [max_batch*G, n_cache], persistent: block held per slot, -1 none
  int32_t* slot;                 // [B, G, kslots] out: cache slot of each idx entry (-1: hot / none)
  int32_t* fetch;                // [max_batch*G, n_cache] scratch: block to fetch per slot, -1 none
  unsigned long long* stats;     // optional [2]: hits, misses (accumulated)
  __nv_bfloat16* ck_cache;       // [max_batch, G, n_cache, 64, d]
  __nv_bfloat16* cv_cache;
  int* err;
  int B, G, max_ctx, kslots, n_cache;
};
void launch_cache_gather(const CacheArgs& a, cudaStream_t s);   // one CTA per (sequence, group)

void launch_append_kv(const AppendArgs& a, int bg_count, cudaStream_t s);
void launch_compress_keys(const CompressArgs& a, int bg_count, cudaStream_t s);
void launch_forecast_project(const ProjectArgs& a, cudaStream_t s);
void launch_forecast_select(const SelectArgs& a, int bg_count, cudaStream_t s);
// maps: K and V of the resident cache or of the staging buffer, then hot K and V (offload).
// *mass_left: whether the block mass (where wanted) is still to be added, by launch_block_mass.
cudaError_t launch_sparse_attn(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CUtensorMap& hk, const CUtensorMap& hv, int bg_count,
                               cudaStream_t s, bool* mass_left = nullptr);
void launch_prefetch(const PrefetchArgs& a, int n_ctas, cudaStream_t s);
void launch_attend_and_select(const AttnArgs& a, const SelectArgs& s, const CUtensorMap& mk,
                              const CUtensorMap& mv, const CUtensorMap& hk, const CUtensorMap& hv,
                              int bg_count, cudaStream_t st);
// One launch of a layer's decode prologue (prologue.cu): the top-k of the layer's block
// scores, the append of its token and the forecast projection for the next layer.
struct PrologueArgs {
  AppendArgs ap;
  ProjectArgs pj;                // pj.W == nullptr: no projection
  const float* block_scores;     // [B*G, nb_cap]; nullptr: no top-k
  int32_t* idx;                  // [B, G, topk+2]
  int32_t* cnt;                  // [B, G]
  int topk, nb_cap, bg_count;
  int n_proj, n_topk;            // CTAs of the projection and top-k roles
  uint32_t tl_launch;            // launch number for the timeline build's records
  void* tl_buf;                  // the timeline build's record store
};
void launch_decode_prologue(const PrologueArgs& a, cudaStream_t s);
void launch_multihead_select(const MultiheadArgs& a, const CUtensorMap& mck, int bg_count, cudaStream_t s);

// Chunked prefill (prefill.cu): 64-token query chunks, chunk c of sequence-group bg at row
// bg * nb_cap + c of idx [.., topk+2], cnt and the block scores [.., nb_cap].
struct PrefillArgs {
  const __nv_bfloat16* ck;       // [max_batch, G, W_cap, d]
  const __nv_bfloat16* f;        // per-token forecasts [max_batch, max_ctx, G, d]
  const __nv_bfloat16* q;        // per-token queries [max_batch, max_ctx, G*H, d]
  __nv_bfloat16* out;            // attention output [max_batch, max_ctx, G*H, d]
  const int32_t* seq_len;        // prompt lengths [B]
  int32_t* idx;                  // [B*G, nb_cap, topk+2]
  int32_t* cnt;                  // [B*G, nb_cap]
  float* block_scores;           // workspace [B*G, nb_cap, nb_cap]
  int* err;
  int G, W_cap, max_ctx, nb_cap, topk;
};
void launch_prefill_forecast_select(const PrefillArgs& a, int batch, cudaStream_t s);
// mq: the queries [B*max_ctx*G*16 rows, 128] in boxes of 16 rows; mck: the compressed keys.
void launch_prefill_multihead_select(const PrefillArgs& a, const CUtensorMap& mq, const CUtensorMap& mck, int batch,
                                     cudaStream_t s);
// the causal block-sparse prefill attention on tcgen05 tensor cores; mq: the queries as
// [rows, 128] in 64 x 16 boxes, mk / mv: the layer's K and V as [rows, 128] in 64 x 64 boxes
void launch_prefill_attn_tc(const PrefillArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                            const CUtensorMap& mv, int batch, cudaStream_t s);
int multihead_tiles(int w_cap);
int multihead_cluster_size(int n_tiles_cap, int bg_count);

// The 4-bit cache (kv4_cache.cu): writing it, one token or a whole prompt, and reading it back.
struct Kv4CacheArgs {
  uint8_t* kv;                   // [max_batch, G, nb_cap, SPARDA_KV4_BLOCK_BYTES]
  __nv_bfloat16* ck;             // [max_batch, G, W_cap, d] (append)
  const __nv_bfloat16* k;        // quantize: [max_batch, G, max_ctx, d]; append: [B, G, d]
  const __nv_bfloat16* v;
  __nv_bfloat16* k_out;          // dequantize: [max_batch, G, max_ctx, d] or [max_batch, G, kslots, 64, d]
  __nv_bfloat16* v_out;
  const int32_t* idx;            // dequantize of selected blocks: [B, G, kslots]; nullptr: all blocks
  const int32_t* cnt;
  const int32_t* seq_len;
  int* err;
  int G, max_ctx, nb_cap, W_cap, kslots;
};
void launch_kv4_quantize(const Kv4CacheArgs& a, int bg_count, cudaStream_t s);
void launch_kv4_dequantize(const Kv4CacheArgs& a, int bg_count, cudaStream_t s);
void launch_kv4_append(const Kv4CacheArgs& a, int bg_count, cudaStream_t s);

// Decode attention over the 4-bit cache (kv4_attn.cu).
constexpr int kKv4MaxCtas = 160;                  // at most this many CTAs share the blocks
struct Kv4AttnArgs {
  const uint8_t* kv;
  const __nv_bfloat16* q;        // [B, G*H, d]
  const int32_t* idx;            // [B, G, kslots]; nullptr: every block of the sequence
  const int32_t* cnt;
  const int32_t* seq_len;
  __nv_bfloat16* out;            // [B, G*H, d]
  float* part_o;                 // workspace [kKv4MaxCtas, 2, 16, d]
  float* part_ml;                // workspace [kKv4MaxCtas, 2, 2, 16]
  unsigned* counters;            // workspace [max_batch*G], zero between calls
  unsigned* join_counters;       // workspace [kKv4MaxCtas, 2], zero between calls
  float2* stats;                 // block mass: (max, sum) [B*G, slots, parts, 16]; nullptr: not wanted
  float* ml;                     // block mass: final max and sum [B*G, 2, 16]
  float* mass;                   // [max_batch, G, nb_cap]: added to by the cluster form itself
  int* err;
  int G, H, max_ctx, nb_cap, kslots, bg_count;
};
// *parts: the stats' parts per block (2 or 4) where the block mass is still to be added by launch_block_mass,
// else 0.
cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s, int* parts);

// Accumulates the attention weight of each attended block (block_mass.cu).
struct BlockMassArgs {
  const float2* stats;           // [B*G, slots, parts, 16] (max, sum) per part of a block and head
  const float* ml;               // [B*G, 2, 16]
  float* mass;                   // [max_batch, G, nb_cap]
  const int32_t* idx;            // [B, G, kslots]; nullptr: slot j is block j
  const int32_t* cnt;
  const int32_t* seq_len;
  int G, H, max_ctx, nb_cap, slots, parts;   // parts: 2 or 4 per block
};
void launch_block_mass(const BlockMassArgs& a, int bg_count, cudaStream_t s);

// Eviction (evict.cu). A cache is one or two planes of fixed bytes per block.
struct EvictArgs {
  const uint8_t* src[2];         // [max_batch*G, src_nb, block_bytes]
  uint8_t* dst[2];               // [max_batch*G, dst_nb, block_bytes]
  const __nv_bfloat16* src_ck;   // [max_batch*G, 4*src_nb-1, d]
  __nv_bfloat16* dst_ck;
  const float* src_mass;         // [max_batch*G, src_nb]
  float* dst_mass;
  const int32_t* src_len;        // [B]
  int32_t* dst_len;
  int32_t* kept;                 // [B*G, keep]
  int* err;
  int planes, block_bytes, kv4;  // kv4: one plane in the 4-bit layout; else K and V planes of bf16
  int B, G, src_nb, dst_nb, keep, recent, in_place;
};
// Launches nothing behind a launch that failed, whose error it returns. In place, weights and lengths are
// written by the launches behind the one that moves the blocks: an error leaves them, and the cache, as they were.
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

// Attention of many new tokens per sequence over a cache (token_attn.cu): packed prompts and trees.
constexpr int kTokenPartFloats = 128 * (128 + 2); // a partial result of a query tile: O, maximum, sum
constexpr int kTokenMaxSms = 160;                 // SMs that are used, at most: by a CTA of two tiles, or two of one
constexpr int kTokenMaxNodes = 128;               // nodes of a tree, at most
// Division by a number that the host knows, for dividends below 2^31: one product and two shifts where the
// hardware has no divide (T. Granlund and P. Montgomery, "Division by invariant integers using multiplication",
// PLDI 1994, figure 4.1).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t n) : d(n), mul(0), shift(0) {
    while ((1ull << shift) < n) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - n)) / n + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return (__umulhi(mul, x) + x) >> shift; }
#endif
};

// A CTA's share in joining one item that was cut (token_attn.cuh); r0 == r1: none
struct TokenJoin {
  int c1, k, first_slot, r0, r1, g, out_row;
};
struct TokenAttnArgs {
  const int32_t* ctx_len;        // [B] tokens in the cache; nullptr: none
  const int32_t* cu;             // packed prompts: [B+1] first row of each; nullptr: n_rows rows per sequence
  const int32_t* n_nodes;        // [B] rows that are used (cu == nullptr); nullptr: all
  const int32_t* parent;         // [B, n_rows], tree; nullptr: each token attends those before it
  const int32_t* idx;            // [B, G, kslots], the attended blocks of the cache; nullptr: all
  const int32_t* cnt;
  __nv_bfloat16* out;            // [rows, G*H, d]
  float* part;                   // workspace [2 n_ctas][tiles of a CTA][kTokenPartFloats], 32-byte aligned
  TokenJoin* joins;              // workspace [n_ctas][2]
  unsigned* queue;               // workspace: items taken from the queue, zero between calls
  int* err;
  int n_entries, G, H, max_ctx, kslots;
  int n_rows;                    // rows of all prompts, or of each sequence
  int tp;                        // tokens per 128-row query tile
  int causal;                    // parent == nullptr
  int wide_out;                  // out is 32-byte aligned
  int n_ctas;                    // SMs that are used; the launch makes CTAs of them
  int split_items;               // fewer items than this: key tiles are divided, not items
  uint32_t min_tiles;            // a CTA's share of key tiles, at least
  uint32_t item_tiles;           // what an item costs beside its key tiles, in key tiles
  uint32_t join_tiles;           // what cutting items costs, in key tiles, where there is at most one per CTA,
  uint32_t cut_tiles;            //   and where there are more
  uint32_t seg_tiles;            // what another segment costs a CTA, in key tiles
  FastDiv by_G, by_H, by_item;   // by the groups, the heads of a group, the tokens of an item
};
// maps: queries (d, head, group, token, sequence); the cache's K and V [rows, 128]; the new tokens' K and V
// (d, group, token, sequence)
cudaError_t launch_token_attn(const TokenAttnArgs& a, const CUtensorMap* maps, cudaStream_t s);

// New tokens into the cache with the compressed keys of the windows that they complete (token_append.cu).
struct TokenAppendArgs {
  __nv_bfloat16* k;              // [max_batch, G, max_ctx, d]
  __nv_bfloat16* v;
  __nv_bfloat16* ck;             // [max_batch, G, W_cap, d]
  const __nv_bfloat16* k_new;    // rows of G*d, kv_stride apart
  const __nv_bfloat16* v_new;
  long long kv_stride;
  const int32_t* cu;             // packed prompts: [B+1]; nullptr: path
  const int32_t* path;           // [B, n_rows]: row numbers inside the sequence's n_rows rows
  const int32_t* n_path;         // [B]
  const int32_t* seq_len;        // [B]; nullptr: empty caches
  int32_t* new_len;              // [B]; nullptr: not wanted
  int* err;
  int B, G, max_ctx, W_cap, n_rows;
};
cudaError_t launch_token_append(const TokenAppendArgs& a, cudaStream_t s);

// Device address of the library's device error word on the current device (api.cu).
int* dev_error_word();

// Sizes the C ABI needs to lay out workspaces.
int select_chunk_blocks(int nb_cap, int bg_count);
int attn_blocks_per_cta();
size_t smem_select_bytes(int chunk_blocks);
int sm_count();                                   // of the current device (attn.cu)

// A kernel's opt-in to more than 48 KB of shared memory, once per device (each call of the runtime for
// it costs as much as a small check).
struct SmemOptIn {
  std::atomic<bool> done[64] = {};
  template <typename K>
  bool set(K kern, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done[dev].store(true, std::memory_order_release);
    return true;
  }
};

// A launch that may begin while the kernel before it in the stream still runs (programmatic
// dependent launch); the kernel waits for that one with grid_dep_wait().
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace sparda
