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
// K % 8 == 0 every row is 16-byte aligned and a chunk is contiguous (kVec: 16-byte accesses).
// Otherwise a chunk is four pairs of features, each one aligned access (8 bytes of floats, 4 of
// 16-bit elements, 2 of codes), neighbouring chunks' pairs next to each other.  Where a row starts
// at an odd element (p = 1) the pairs begin one feature earlier, and the feature before the block's
// first, which belongs to the block before, is replaced by the block's last.  A thread may hold
// n = 1, 2 or 4 chunks of one block, 16 / n lanes then sharing it (chunk_of): the block's scale costs
// two divisions a lane.
#pragma once

#include <algorithm>

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
// Parity of row m's first element in a [M][K] tensor.
__device__ __forceinline__ int row_parity(int64_t m, int64_t K) { return static_cast<int>(m & K & 1); }

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

// The pair layout's features of chunk c, counted from the block's first one (`base`): values 2u and
// 2u + 1 are at + 32 u and the next one, except value 0 of a chunk with at = -1, which is the
// block's last feature.  `left`: the block's features inside the row.
template <typename I>
struct PairAt {
  I base;
  int at, left;
  __device__ __forceinline__ PairAt(I c, I K, int p)
      : base((c / kActLanes) * kActBlock), at(2 * static_cast<int>(c % kActLanes) - p),
        left(static_cast<int>(max(min(K - base, static_cast<I>(kActBlock)), static_cast<I>(0)))) {}
  PairAt() = default;
  static __device__ __forceinline__ PairAt in(I base, int at, int left) {
    PairAt q;
    q.base = base, q.at = at, q.left = left;
    return q;
  }
  __device__ __forceinline__ int feature(int j) const {   // value j's, in the block
    return j == 0 && at < 0 ? kActBlock - 1 : at + 32 * (j / 2) + j % 2;
  }
};

// Two neighbouring elements as one access.
template <typename T>
struct Pair {
  using Word = uint32_t;
};
template <>
struct Pair<float> {
  using Word = float2;
};
__device__ __forceinline__ float2 unpack2(float2 w, float) { return w; }
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 pack2(float a, float b, float) { return make_float2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A pair layout's chunk, from whole pairs (an odd row's first one starts with the last element of the
// row before).
template <typename T, typename I>
__device__ __forceinline__ void load_pairs(const T* row, const PairAt<I>& q, float (&v)[8]) {
  using Word = typename Pair<T>::Word;
  const Word* src = reinterpret_cast<const Word*>(row + q.base + q.at);
  Word w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = src[16 * u];
  T last{};
  if (q.at < 0) last = row[q.base + kActBlock - 1];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float2 f = unpack2(w[u], T{});
    v[2 * u] = f.x, v[2 * u + 1] = f.y;
  }
  if (q.at < 0) v[0] = Elem<T>::to(last);
}

// The same of any block: zeros past the row's end.
template <typename T, typename I>
__device__ __forceinline__ void load_chunk(const T* row, const PairAt<I>& q, float (&v)[8]) {
  if (q.left == kActBlock) {
    load_pairs(row, q, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q.feature(j) < q.left ? Elem<T>::to(row[q.base + q.feature(j)]) : 0.0f;
  }
}

// The 8 values of chunk c (16 chunks a block) of a row of K: zeros past the row's end.  p: parity
// of the row's start (row_parity; kVec: unused).
template <typename T, bool kVec, typename I>
__device__ __forceinline__ void load8(const T* row, I c, I K, float (&v)[8], int p = 0) {
  if constexpr (kVec) {
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
    load_chunk(row, PairAt<I>(c, K, p), v);
  }
}

template <typename T, typename I>
__device__ __forceinline__ void store_pairs(T* row, const PairAt<I>& q, const float (&v)[8]) {
  using Word = typename Pair<T>::Word;
  Word* dst = reinterpret_cast<Word*>(row + q.base + q.at);
#pragma unroll
  for (int u = 1; u < 4; ++u) dst[16 * u] = pack2(v[2 * u], v[2 * u + 1], T{});
  if (q.at < 0) {
    row[q.base + kActBlock - 1] = Elem<T>::from(v[0]);
    row[q.base] = Elem<T>::from(v[1]);
  } else {
    dst[0] = pack2(v[0], v[1], T{});
  }
}
template <typename T, typename I>
__device__ __forceinline__ void store_chunk(T* row, const PairAt<I>& q, const float (&v)[8]) {
  if (q.left == kActBlock) {
    store_pairs(row, q, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (q.feature(j) < q.left) row[q.base + q.feature(j)] = Elem<T>::from(v[j]);
  }
}
template <typename T, bool kVec, typename I>
__device__ __forceinline__ void store8(T* row, I c, I K, const float (&v)[8], int p = 0) {
  if constexpr (kVec) {
    if (c * 8 < K) {
      alignas(16) T raw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = Elem<T>::from(v[j]);
      uint4* dst = reinterpret_cast<uint4*>(row + c * 8);
      dst[0] = *reinterpret_cast<uint4*>(raw);
      if (sizeof(T) == 4) dst[1] = *reinterpret_cast<uint4*>(raw + 4);
    }
  } else {
    store_chunk(row, PairAt<I>(c, K, p), v);
  }
}

// The same features of a [K] vector, whose start is even whatever the row's is.
template <bool kVec, typename I>
__device__ __forceinline__ void load_vector8(const float* w, I c, I K, float (&v)[8], int p) {
  if (kVec || p == 0) {
    load8<float, kVec>(w, c, K, v);
  } else {
    const PairAt<I> q(c, K, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q.feature(j) < q.left ? w[q.base + q.feature(j)] : 0.0f;
  }
}

template <typename I>
__device__ __forceinline__ uint2 load_code_pairs(const int8_t* row, const PairAt<I>& f) {
  const uint16_t* src = reinterpret_cast<const uint16_t*>(row + f.base + f.at);
  uint2 q = make_uint2(__byte_perm(src[0], src[16], 0x5410), __byte_perm(src[32], src[48], 0x5410));
  if (f.at < 0) q.x = (q.x & 0xffffff00u) | static_cast<uint8_t>(row[f.base + kActBlock - 1]);
  return q;
}

template <typename I>
__device__ __forceinline__ uint2 load_code_chunk(const int8_t* row, const PairAt<I>& f) {
  if (f.left == kActBlock) return load_code_pairs(row, f);
  uint2 q = make_uint2(0, 0);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = f.feature(j) < f.left ? static_cast<uint8_t>(row[f.base + f.feature(j)]) : 0u;
    if (j < 4) q.x |= b << (8 * j);
    else q.y |= b << (8 * (j - 4));
  }
  return q;
}

// A lane's 8 codes, packed in order (byte j: value j).
template <bool kVec, typename I>
__device__ __forceinline__ uint2 load_codes(const int8_t* row, I c, I K, int p = 0) {
  uint2 q = make_uint2(0, 0);
  if constexpr (kVec) {
    if (c * 8 < K) q = *reinterpret_cast<const uint2*>(row + c * 8);
  } else {
    q = load_code_chunk(row, PairAt<I>(c, K, p));
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
struct BlockScale {
  float scale, inv;
  bool bad;
  __device__ __forceinline__ explicit BlockScale(float amax) {
    bad = !(amax < INFINITY);
    const bool live = amax >= kActTiny && !bad;
    inv = live ? 127.0f / amax : 0.0f;
    scale = bad ? __int_as_float(0x7fc00000) : live ? amax / 127.0f : 0.0f;
  }
};
__device__ __forceinline__ float chunk_amax(const float (&v)[8], float amax) {
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max_abs_nan(amax, v[j]);
  return amax;
}
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float inv, bool bad) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f));
  const uint32_t x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  const uint32_t y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
  return bad ? make_uint2(0, 0) : make_uint2(x, y);
}
template <int kN>
__device__ __forceinline__ Quantized<kN> quantize_block(const float (&v)[kN][8]) {
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < kN; ++u) amax = chunk_amax(v[u], amax);
#pragma unroll
  for (int o = kActLanes / kN / 2; o > 0; o >>= 1) amax = max_abs_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const BlockScale s(amax);
  Quantized<kN> q;
  q.bad = s.bad, q.scale = s.scale;
#pragma unroll
  for (int u = 0; u < kN; ++u) q.codes[u] = codes_of(v[u], s.inv, s.bad);
  return q;
}

// The scales of kN = 2 or 4 blocks that a half warp holds, one chunk of each a lane (v[u]: of block u).
// Lanes 16 / kN of it come to hold one block's largest magnitude (exchanges of halves, then of
// whole values, for what kN reductions one by one take four each), find its scale, which is
// returned, and pass its inverse on (-1: not finite).  Every lane of the warp calls it.
template <int kN>
__device__ __forceinline__ BlockScale shared_scales(const float (&v)[kN][8], int t, float (&inv)[kN]) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kOwn = kActLanes / kN;
  float k[kN];
#pragma unroll
  for (int u = 0; u < kN; ++u) k[u] = chunk_amax(v[u], 0.0f);
#pragma unroll
  for (int o = 8, n = kN / 2; n > 0; o /= 2, n /= 2)
#pragma unroll
    for (int u = 0; u < n; ++u) {
      const float keep = t & o ? k[u + n] : k[u], give = t & o ? k[u] : k[u + n];
      k[u] = max_abs_nan(keep, __shfl_xor_sync(kAll, give, o));
    }
#pragma unroll
  for (int o = kOwn / 2; o > 0; o /= 2) k[0] = max_abs_nan(k[0], __shfl_xor_sync(kAll, k[0], o));
  const BlockScale s(k[0]);
  const float own = s.bad ? -1.0f : s.inv;
#pragma unroll
  for (int u = 0; u < kN; ++u) inv[u] = __shfl_sync(kAll, own, (t & 16) + kOwn * u);
  return s;
}

template <typename I>
__device__ __forceinline__ void store_code_pairs(int8_t* row, const PairAt<I>& f, uint2 q) {
  uint16_t* dst = reinterpret_cast<uint16_t*>(row + f.base + f.at);
  dst[16] = static_cast<uint16_t>(q.x >> 16);
  dst[32] = static_cast<uint16_t>(q.y);
  dst[48] = static_cast<uint16_t>(q.y >> 16);
  if (f.at < 0) {
    row[f.base + kActBlock - 1] = static_cast<int8_t>(q.x);
    row[f.base] = static_cast<int8_t>(q.x >> 8);
  } else {
    dst[0] = static_cast<uint16_t>(q.x);
  }
}

template <typename I>
__device__ __forceinline__ void store_code_chunk(int8_t* row, const PairAt<I>& f, uint2 q) {
  if (f.left == kActBlock) {
    store_code_pairs(row, f, q);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (f.feature(j) < f.left) row[f.base + f.feature(j)] = static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// Stores chunk c's codes.
template <bool kVec, typename I>
__device__ __forceinline__ void store_codes(int8_t* row, I c, I K, uint2 q, int p) {
  if constexpr (kVec) {
    if (c * 8 < K) *reinterpret_cast<uint2*>(row + c * 8) = q;
  } else {
    store_code_chunk(row, PairAt<I>(c, K, p), q);
  }
}

// Stores what a thread quantized: its chunks' codes, and the scale from the block's first lane.
template <bool kVec, int kN>
__device__ __forceinline__ void store_block(const Act8View& a, int64_t m, int64_t t, int64_t K, const Quantized<kN>& q,
                                            int* status, int p = 0) {
  const int64_t b = t / (kActLanes / kN);
  if (b * kActBlock >= K) return;
#pragma unroll
  for (int u = 0; u < kN; ++u) store_codes<kVec>(a.codes + m * K, chunk_of(t, kN, u), K, q.codes[u], p);
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

// CTAs for `want` rounds of rows where `most` are resident: as few as take no more turns each (a
// weight gradient has a part from each), and an even number, so that all of a CTA's rows start at
// the same parity.
inline int64_t even_grid(int64_t want, int64_t most) {
  const int64_t turns = std::max<int64_t>(1, (want + std::max<int64_t>(most, 1) - 1) / std::max<int64_t>(most, 1));
  return turns == 1 ? want : ((want + turns - 1) / turns + 1) / 2 * 2;
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
