// Rows streamed through shared memory for the norm's kernels: a worker (one warp, or a whole CTA)
// walks over rows, each row's inputs arrive by bulk copies in a ring of stages, and every thread
// holds four (or two) chunks of one block of the row in registers (train_ops.cuh).  The copies need no
// registers and stay in flight across the reductions, which is what keeps HBM busy.
#pragma once

#include "tc_ptx.cuh"
#include "train_ops.cuh"

namespace qnf4 {

constexpr int kRingN = 4;                        // chunks a thread holds, where nothing else is said
constexpr int kRingStagesMax = 4;
constexpr size_t kRingSmemMax = 200 * 1024;      // a CTA's ring at most; two stages must fit
constexpr int kRingWarpWorkers = 4;              // workers of a CTA where a worker is a warp

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Threads of a worker, workers of a CTA, stages, and the grid for M rows whose inputs take
// `bytes` a row.  stages = 0: the rows do not fit.
struct RingShape {
  int G, workers, stages;
  unsigned grid;
  size_t smem;
};
inline RingShape ring_shape(int64_t M, int64_t K, size_t bytes, int regs, int n = kRingN) {
  RingShape s{};
  const int64_t lanes = (K + kActBlock - 1) / kActBlock * (kActLanes / n);
  if (lanes < 16 || lanes > 512) return s;   // under half a warp busy, or over the registers
  s.G = static_cast<int>((lanes + 31) / 32 * 32);
  s.workers = s.G == 32 ? kRingWarpWorkers : 1;
  const int threads = s.G * s.workers;
  // the CTAs that the registers allow share the SM's memory; then as many stages as fit
  int ctas = std::max(1, std::min(65536 / regs / threads, 16));
  while (ctas > 1 && kRingSmemMax / ctas / s.workers / bytes < 2) --ctas;
  s.stages = static_cast<int>(std::min<size_t>(kRingSmemMax / ctas / s.workers / bytes, kRingStagesMax));
  if (s.stages < 2) {
    s.stages = 0;
    return s;
  }
  s.smem = s.workers * s.stages * bytes;
  const int64_t want = (M + s.workers - 1) / s.workers;
  s.grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(ctas) * device_sm_count()));
  return s;
}

// Sum over a worker's threads: a warp, or the CTA (red: [2][32] floats, `turn` alternates).
__device__ __forceinline__ float worker_sum(float v, int G, float* red, int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 32) return v;
  if ((threadIdx.x & 31) == 0) red[turn * 32 + (threadIdx.x >> 5)] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < G / 32 ? red[turn * 32 + (threadIdx.x & 31)] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 8 values of chunk c from a row in shared memory (zeros past the row's end).
template <typename T>
__device__ __forceinline__ void ring8(const uint8_t* row, int64_t c, int64_t K, float (&v)[8]) {
  load8<T, true>(reinterpret_cast<const T*>(row), c, K, v);
}

}  // namespace qnf4
