// The bandwidth operators around the linear in a training step: RMS norm with the residual's
// addition, 8-bit activation checkpoints, and the adapter gradient read from one.
//
// Checkpoint format: int8 codes [M][K] and one fp32 scale for each token and block of 128
// features, [M][ceil(K / 128)].  amax = largest |x| of the block; scale = amax / 127, code =
// rint(x * (127 / amax)), ties to even, value = code * scale.  A block with amax < 2^-116
// (127 / amax could overflow) is stored as zeros.  A block holding a NaN or an infinity gets
// the scale NaN, so that everything read from it is NaN, and sets NF4_ERR_NONFINITE.
//
// Layout shared by the kernels: a row is cut in chunks of 8 values, 16 chunks a block.  With
// K % 8 == 0 every row is 16-byte aligned and a chunk is contiguous (kVec: 16-byte accesses);
// otherwise chunk i of a block takes features i, i + 16, ... of it, so that neighbouring lanes'
// narrow accesses stay within the same sectors.  A thread may hold n = 1, 2 or 4 chunks of one
// block, 16 / n lanes then sharing it (chunk_of): the block's scale costs two divisions a lane.
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
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, nf4_dtype dt, int* status, cudaStream_t st);

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

// Chunk u of thread t's n: lanes t % (16 / n) + (16 / n) u of block t / (16 / n).
__device__ __forceinline__ int64_t chunk_of(int64_t t, int n, int u) {
  const int lanes = kActLanes / n;
  return t / lanes * kActLanes + t % lanes + lanes * u;
}

__device__ __forceinline__ float max_abs_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// Quantizes a block held by 16 / kN neighbouring lanes, kN chunks each; every lane of the warp
// calls it.  Codes are rint(v * inv) by way of 1.5 * 2^23: the product is rounded to fp32, then
// the sum's last byte is the code in two's complement.
template <int kN>
struct Quantized {
  uint2 codes[kN];
  float scale;
  bool bad;
};
template <int kN>
__device__ __forceinline__ Quantized<kN> quantize_block(const float (&v)[kN][8]) {
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < kN; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max_abs_nan(amax, v[u][j]);
#pragma unroll
  for (int o = kActLanes / kN / 2; o > 0; o >>= 1) amax = max_abs_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  Quantized<kN> q;
  q.bad = !(amax < INFINITY);
  const bool live = amax >= kActTiny && !q.bad;
  const float inv = live ? 127.0f / amax : 0.0f;
  q.scale = q.bad ? __int_as_float(0x7fc00000) : live ? amax / 127.0f : 0.0f;
#pragma unroll
  for (int u = 0; u < kN; ++u) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[u][j], inv), 12582912.0f));
    q.codes[u].x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    q.codes[u].y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
    if (q.bad) q.codes[u] = make_uint2(0, 0);
  }
  return q;
}

// Stores chunk c's codes.
template <bool kVec>
__device__ __forceinline__ void store_codes(int8_t* row, int64_t c, int64_t K, uint2 q) {
  if (kVec) {
    if (c * 8 < K) *reinterpret_cast<uint2*>(row + c * 8) = q;
  } else {
    const int64_t e = (c / kActLanes) * kActBlock + c % kActLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + 16 * j < K) row[e + 16 * j] = static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// Stores what a thread quantized: its chunks' codes, and the scale from the block's first lane.
template <bool kVec, int kN>
__device__ __forceinline__ void store_block(const Act8View& a, int64_t m, int64_t t, int64_t K, const Quantized<kN>& q,
                                            int* status) {
  const int64_t b = t / (kActLanes / kN);
  if (b * kActBlock >= K) return;
#pragma unroll
  for (int u = 0; u < kN; ++u) store_codes<kVec>(a.codes + m * K, chunk_of(t, kN, u), K, q.codes[u]);
  if (t % (kActLanes / kN) == 0) {
    a.scales[m * ((K + kActBlock - 1) / kActBlock) + b] = q.scale;
    if (q.bad) atomicCAS(status, 0, static_cast<int>(NF4_ERR_NONFINITE));
  }
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
