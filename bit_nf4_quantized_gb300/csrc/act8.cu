// 8-bit activation checkpoints: storing, reading back, and the adapter gradient
// dA = s G^T x taken straight from the codes.
#include <algorithm>

#include "train_ops.cuh"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;

// One lane per 8 values, 16 lanes per block (train_ops.cuh).  Bound by HBM: the activation
// once, one byte a value and 4 / 128 out.
template <typename T, bool kVec>
__global__ void act8_quantize(const T* x, int64_t M, int64_t K, Act8View out, int* status) {
  pdl_allow_next();
  pdl_wait();
  const int64_t C = (K + kActBlock - 1) / kActBlock * kActLanes;
  const int64_t n = M * C;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const bool on = i < n;     // whole blocks of 16 lanes
  const int64_t m = on ? i / C : 0, c = on ? i - m * C : 0;
  float v[8];
  load8<T, kVec>(x + m * K, c, K, v);
  const Quantized q = quantize_block(v);
  if (on) store_codes<kVec>(out, m, c, K, q);
  if (on && q.bad) atomicCAS(status, 0, static_cast<int>(NF4_ERR_NONFINITE));
}

template <typename T, bool kVec>
__global__ void act8_dequantize(Act8View in, int64_t M, int64_t K, const float* weight, T* out) {
  pdl_allow_next();
  pdl_wait();
  const int64_t C = (K + kActBlock - 1) / kActBlock * kActLanes, nb = C / kActLanes;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= M * C) return;
  const int64_t m = i / C, c = i - m * C;
  const uint2 q = load_codes<kVec>(in.codes + m * K, c, K);
  const float sc = in.scales[m * nb + c / kActLanes];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = code_value(q, j) * sc;
  if (weight != nullptr) {
    float w[8];
    load8<float, kVec>(weight, c, K, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= w[j];
  }
  store8<T, kVec>(out + m * K, c, K, v);
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t M, int64_t K, Act8View out, int* status, cudaStream_t st) {
  const int64_t n = M * ((K + kActBlock - 1) / kActBlock) * kActLanes;
  const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads));
  note_launch();
  return K % 8 == 0 ? launch_pdl(act8_quantize<T, true>, grid, dim3(kThreads), 0, st, 1, static_cast<const T*>(x), M, K,
                                 out, status)
                    : launch_pdl(act8_quantize<T, false>, grid, dim3(kThreads), 0, st, 1, static_cast<const T*>(x), M,
                                 K, out, status);
}

template <typename T>
cudaError_t dequantize_t(Act8View in, int64_t M, int64_t K, const float* weight, void* out, cudaStream_t st) {
  const int64_t n = M * ((K + kActBlock - 1) / kActBlock) * kActLanes;
  const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads));
  note_launch();
  return K % 8 == 0 ? launch_pdl(act8_dequantize<T, true>, grid, dim3(kThreads), 0, st, 1, in, M, K, weight,
                                 static_cast<T*>(out))
                    : launch_pdl(act8_dequantize<T, false>, grid, dim3(kThreads), 0, st, 1, in, M, K, weight,
                                 static_cast<T*>(out));
}

// ---- dA ---------------------------------------------------------------------------------
constexpr int kGradRanks = 16;     // ranks of a CTA
constexpr int kGradTokens = 64;    // tokens staged at a time

// One block of 128 features (a thread each), 16 ranks, one slice of the tokens: fp32 products
// and sums.  part: [slice][r][K].
__global__ void act8_grad(const ActGradArgs a, int64_t slice_tokens, float* part) {
  __shared__ float g[kGradTokens][kGradRanks];
  __shared__ float sc[kGradTokens];
  pdl_allow_next();
  pdl_wait();
  const int64_t nb = (a.K + kActBlock - 1) / kActBlock;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kActBlock + threadIdx.x;
  const int j0 = blockIdx.z * kGradRanks;
  const int64_t m0 = blockIdx.y * slice_tokens, m1 = min(m0 + slice_tokens, a.M);
  float acc[kGradRanks];
#pragma unroll
  for (int j = 0; j < kGradRanks; ++j) acc[j] = 0.0f;
  for (int64_t mb = m0; mb < m1; mb += kGradTokens) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kGradTokens), m1 - mb));
    __syncthreads();
    for (int i = threadIdx.x; i < n * kGradRanks; i += kActBlock) {
      const int t = i / kGradRanks, j = i % kGradRanks;
      g[t][j] = j0 + j < a.r ? a.G[(mb + t) * a.r + j0 + j] : 0.0f;
    }
    if (threadIdx.x < n) sc[threadIdx.x] = a.act.scales[(mb + threadIdx.x) * nb + blockIdx.x];
    __syncthreads();
    if (k < a.K) {
      for (int t = 0; t < n; ++t) {
        const float x = static_cast<float>(a.act.codes[(mb + t) * a.K + k]) * sc[t];
#pragma unroll
        for (int j = 0; j < kGradRanks; ++j) acc[j] = fmaf(g[t][j], x, acc[j]);
      }
    }
  }
  if (k < a.K) {
#pragma unroll
    for (int j = 0; j < kGradRanks; ++j)
      if (j0 + j < a.r) part[(static_cast<int64_t>(blockIdx.y) * a.r + j0 + j) * a.K + k] = acc[j];
  }
}

// dA = s * weight * (the slices' sums in order)
__global__ void act8_grad_finish(const ActGradArgs a, const float* part, int slices) {
  pdl_allow_next();
  pdl_wait();
  const int64_t n = static_cast<int64_t>(a.r) * a.K;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int q = 0; q < slices; ++q) s += part[q * n + i];
  s *= a.s;
  a.dA[i] = a.weight != nullptr ? s * a.weight[i % a.K] : s;
}

int grad_slices(int64_t M, int64_t K, int r) {
  const int64_t ctas = (K + kActBlock - 1) / kActBlock * ((r + kGradRanks - 1) / kGradRanks);
  const int64_t want = (device_sm_count() * 8 + ctas - 1) / ctas;
  return static_cast<int>(std::max<int64_t>(1, std::min({want, (M + kGradTokens - 1) / kGradTokens, int64_t(64)})));
}

}  // namespace

cudaError_t launch_act8_quantize(const void* x, nf4_dtype dt, int64_t M, int64_t K, Act8View out, int* status,
                                 cudaStream_t st) {
  if (M == 0) return cudaSuccess;
  switch (dt) {
    case NF4_F32: return quantize_t<float>(x, M, K, out, status, st);
    case NF4_BF16: return quantize_t<__nv_bfloat16>(x, M, K, out, status, st);
    default: return quantize_t<__half>(x, M, K, out, status, st);
  }
}

cudaError_t launch_act8_dequantize(Act8View in, int64_t M, int64_t K, const float* weight, void* out, nf4_dtype dt,
                                   cudaStream_t st) {
  if (M == 0) return cudaSuccess;
  switch (dt) {
    case NF4_F32: return dequantize_t<float>(in, M, K, weight, out, st);
    case NF4_BF16: return dequantize_t<__nv_bfloat16>(in, M, K, weight, out, st);
    default: return dequantize_t<__half>(in, M, K, weight, out, st);
  }
}

size_t act8_grad_ws_bytes(int64_t M, int64_t K, int r) {
  return M == 0 ? 0 : sizeof(float) * static_cast<size_t>(grad_slices(M, K, r)) * static_cast<size_t>(r) * K;
}

cudaError_t launch_act8_grad(const ActGradArgs& a, void* ws, cudaStream_t st) {
  if (a.M == 0) return cudaMemsetAsync(a.dA, 0, sizeof(float) * static_cast<size_t>(a.r) * a.K, st);
  const int want = grad_slices(a.M, a.K, a.r);
  const int64_t per = (a.M + want - 1) / want;
  const int slices = static_cast<int>((a.M + per - 1) / per);
  auto* part = static_cast<float*>(ws);
  const dim3 grid(static_cast<unsigned>((a.K + kActBlock - 1) / kActBlock), static_cast<unsigned>(slices),
                  static_cast<unsigned>((a.r + kGradRanks - 1) / kGradRanks));
  note_launch();
  cudaError_t e = launch_pdl(act8_grad, grid, dim3(kActBlock), 0, st, 1, a, per, part);
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(a.r) * a.K;
  note_launch();
  return launch_pdl(act8_grad_finish, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                    1, a, static_cast<const float*>(part), slices);
}

}  // namespace qnf4
