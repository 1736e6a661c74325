// The attention weight that each attended block received, summed over the group's heads and added
// to the sequence's running totals: mass[b, g, j] += sum_h sum_{t in block j} softmax_h(t).
//
// The attention kernels leave, for every quarter or half (16 or 32 tokens) of an attended block and
// every head, a reference m and the sum l of exp2(s - m), and for every head the final reference M
// and sum L over all blocks; the weight of the part is l exp2(m - M) / L. So no score is stored or
// computed twice: 256 or 512 bytes per block beside the block's 10 to 32 KiB. Where a (sequence,
// group) is one thread-block cluster, the attention adds the weights itself (its CTAs tell each other their
// partial M and L), which saves this launch (11.4 -> 10.9 us for 34 blocks of each of 16 sequences in 4
// bits when it was added, 9.8 now).
// This kernel serves the other forms, one warp per attended block; a block's weights are added in a
// fixed order (add_block_mass).
#include "block_mass.cuh"
#include "kernels.h"

#include "common.cuh"

namespace sparda {

constexpr int kMassWarps = 8;

__global__ void __launch_bounds__(kMassWarps * 32) block_mass_kernel(const BlockMassArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int per = (a.slots + kMassWarps - 1) / kMassWarps;
  const int bg = blockIdx.x / per, s = (blockIdx.x % per) * kMassWarps + (int)threadIdx.x / 32, lane = threadIdx.x & 31;
  const int T = a.seq_len[bg / a.G];
  if (s >= a.slots || T < 1 || T > a.max_ctx) return;
  const int32_t* idx = a.idx ? a.idx + (size_t)bg * a.slots : nullptr;
  const int n = idx ? min(a.cnt[bg], a.slots) : a.slots, h = lane & 15;
  if (s >= n) return;
  add_block_mass(a.stats + (size_t)bg * a.slots * a.parts * kHeads, a.parts, a.H, a.ml[bg * 2 * kHeads + h],
                 a.ml[bg * 2 * kHeads + kHeads + h], slot_blocks(idx, n), s, (T - 1) / kBlock,
                 a.mass + (size_t)bg * a.nb_cap);
}

void launch_block_mass(const BlockMassArgs& a, int bg_count, cudaStream_t s) {
  const unsigned per = (unsigned)(a.slots + kMassWarps - 1) / kMassWarps;
  launch_pdl(block_mass_kernel, dim3(per * (unsigned)bg_count), dim3(kMassWarps * 32), 0, s, a);
}

}  // namespace sparda
