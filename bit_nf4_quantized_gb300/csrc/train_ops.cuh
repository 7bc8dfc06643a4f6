// The bandwidth operators around the linear in a training step: RMS norm with the residual's
// addition, 8-bit activation checkpoints, and the adapter gradient read from one.
//
// Checkpoint format: int8 codes [M][K] and one fp32 scale for each token and block of 128
// features, [M][ceil(K / 128)].  amax = largest |x| of the block; scale = amax / 127, code =
// rint(x * (127 / amax)), ties to even, value = code * scale.  A block with amax < 2^-116
// (127 / amax could overflow) is stored as zeros.  A block holding a NaN or an infinity gets
// the scale NaN, so that everything read from it is NaN, and sets NF4_ERR_NONFINITE.
//
// Layout shared by the kernels: the 128 features of a block belong to 16 neighbouring lanes,
// 8 values each.  With K % 8 == 0 every row is 16-byte aligned and a lane's 8 values are
// contiguous (kVec: 16-byte accesses); otherwise lane i takes features i, i + 16, ... of its
// block, so that the 16 lanes' narrow accesses stay within the same sectors.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace qnf4 {

constexpr int kActBlock = 128;
constexpr int kActLanes = 16;          // lanes of a block, 8 values each
constexpr float kActTiny = 0x1p-116f;

struct Act8View {
  int8_t* codes;
  float* scales;
};

// ---- rms_norm_fwd.cu / rms_norm_bwd.cu ------------------------------------------------
struct NormFwdArgs {
  int64_t M, K;
  float eps;
  const void* x;
  const void* residual;   // or nullptr
  const float* weight;
  void* y;
  void* h;                // or nullptr
  float* rstd;
  Act8View act;           // codes nullptr: no checkpoint
};
cudaError_t launch_rms_norm_fwd(const NormFwdArgs& a, nf4_dtype dt, int* status, cudaStream_t st);

struct NormBwdArgs {
  int64_t M, K;
  const void* dy;
  const void* h;          // or nullptr: the checkpoint
  Act8View act;
  const float* rstd;
  const float* weight;
  const void* dresidual;  // or nullptr
  void* dx;
  float* dweight;         // or nullptr
  float* partial;         // rms_norm_bwd_ws_bytes, with dweight
};
size_t rms_norm_bwd_ws_bytes(int64_t M, int64_t K);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, nf4_dtype dt, cudaStream_t st);

// ---- act8.cu ------------------------------------------------------------------------------
cudaError_t launch_act8_quantize(const void* x, nf4_dtype dt, int64_t M, int64_t K, Act8View out, int* status,
                                 cudaStream_t st);
cudaError_t launch_act8_dequantize(Act8View in, int64_t M, int64_t K, const float* weight, void* out, nf4_dtype dt,
                                   cudaStream_t st);

// dA[j][k] = s * weight[k] * sum over m of G[m][j] * code[m][k] * scale[m][k / 128]
struct ActGradArgs {
  int64_t M, K;
  int r;
  float s;
  const float* G;         // [M][r]
  Act8View act;
  const float* weight;    // [K] or nullptr
  float* dA;              // [r][K]
};
size_t act8_grad_ws_bytes(int64_t M, int64_t K, int r);
cudaError_t launch_act8_grad(const ActGradArgs& a, void* ws, cudaStream_t st);

// ---- device helpers -----------------------------------------------------------------------
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

// The 8 values of chunk c (16 chunks a block) of a row of K: zeros past the row's end.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t K, float (&v)[8]) {
  if (kVec) {
    alignas(16) T raw[8];
    if (c * 8 < K) {
      const uint4* src = reinterpret_cast<const uint4*>(row + c * 8);
      *reinterpret_cast<uint4*>(raw) = src[0];
      if (sizeof(T) == 4) *reinterpret_cast<uint4*>(raw + 4) = src[1];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = Elem<T>::to(raw[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
  } else {
    const int64_t e = (c / kActLanes) * kActBlock + c % kActLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e + 16 * j < K ? Elem<T>::to(row[e + 16 * j]) : 0.0f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t K, const float (&v)[8]) {
  if (kVec) {
    if (c * 8 < K) {
      alignas(16) T raw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = Elem<T>::from(v[j]);
      uint4* dst = reinterpret_cast<uint4*>(row + c * 8);
      dst[0] = *reinterpret_cast<uint4*>(raw);
      if (sizeof(T) == 4) dst[1] = *reinterpret_cast<uint4*>(raw + 4);
    }
  } else {
    const int64_t e = (c / kActLanes) * kActBlock + c % kActLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + 16 * j < K) row[e + 16 * j] = Elem<T>::from(v[j]);
  }
}

// A lane's 8 codes, packed in feature order (byte j: value j).
template <bool kVec>
__device__ __forceinline__ uint2 load_codes(const int8_t* row, int64_t c, int64_t K) {
  uint2 q = make_uint2(0, 0);
  if (kVec) {
    if (c * 8 < K) q = *reinterpret_cast<const uint2*>(row + c * 8);
  } else {
    const int64_t e = (c / kActLanes) * kActBlock + c % kActLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = e + 16 * j < K ? static_cast<uint8_t>(row[e + 16 * j]) : 0u;
      if (j < 4) q.x |= b << (8 * j);
      else q.y |= b << (8 * (j - 4));
    }
  }
  return q;
}

// Byte j of the codes as a float: the byte with its sign bit flipped (0..255) placed in the
// mantissa of 2^23, minus 2^23 + 128 (exact).
__device__ __forceinline__ float code_value(uint2 q, int j) {
  const uint32_t w = (j < 4 ? q.x : q.y) ^ 0x80808080u;
  const uint32_t f = __byte_perm(w, 0x4b000000u, 0x7440u | static_cast<uint32_t>(j & 3));
  return __uint_as_float(f) - 8388736.0f;
}

// Quantizes the 16 lanes' block: every lane of the warp calls it.  Returns the codes of this
// lane's values and the block's scale.
struct Quantized {
  uint2 codes;
  float scale;
  bool bad;
};
__device__ __forceinline__ Quantized quantize_block(const float (&v)[8]) {
  float amax = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(v[j]);
    bad |= !(a < INFINITY);
    amax = fmaxf(amax, a);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    bad |= __shfl_xor_sync(0xffffffffu, static_cast<int>(bad), o) != 0;
  }
  Quantized q;
  q.bad = bad;
  const bool live = amax >= kActTiny && !bad;
  const float inv = live ? 127.0f / amax : 0.0f;
  q.scale = bad ? __int_as_float(0x7fc00000) : live ? amax / 127.0f : 0.0f;
  uint32_t w[2] = {0, 0};
  if (!bad) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j / 4] |= (static_cast<uint32_t>(__float2int_rn(v[j] * inv)) & 0xffu) << (8 * (j & 3));
  }
  q.codes = make_uint2(w[0], w[1]);
  return q;
}

// Stores a lane's codes, and the scale from the block's first lane.
template <bool kVec>
__device__ __forceinline__ void store_codes(const Act8View& a, int64_t m, int64_t c, int64_t K, const Quantized& q) {
  if ((c / kActLanes) * kActBlock >= K) return;
  int8_t* row = a.codes + m * K;
  if (kVec) {
    if (c * 8 < K) *reinterpret_cast<uint2*>(row + c * 8) = q.codes;
  } else {
    const int64_t e = (c / kActLanes) * kActBlock + c % kActLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + 16 * j < K) row[e + 16 * j] = static_cast<int8_t>((j < 4 ? q.codes.x : q.codes.y) >> (8 * (j & 3)));
  }
  if (c % kActLanes == 0) a.scales[m * ((K + kActBlock - 1) / kActBlock) + c / kActLanes] = q.scale;
}

// Sum over a row's group of threads (threadIdx.x of a (G, R) block, G a multiple of 32);
// red: [2][R][32] floats, `turn` alternates between calls so that one barrier a call is enough.
__device__ __forceinline__ float group_sum(float v, float* red, int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  float* slot = red + (turn * blockDim.y + threadIdx.y) * 32;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  float s = (threadIdx.x & 31) < warps ? slot[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Threads of a row and rows of a CTA for C chunks with NV chunks a thread.
struct RowShape {
  int G, R;
};
inline RowShape row_shape(int64_t C, int nv) {
  const int64_t per = (C + nv - 1) / nv;
  const int G = static_cast<int>((per + 31) / 32 * 32);
  return RowShape{G, G >= 256 ? 1 : 256 / G};
}

}  // namespace qnf4
