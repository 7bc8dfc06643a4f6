// Backward pass of the RMS norm, from the residual stream or from the 8-bit checkpoint.
//
//   n = h rstd (or code * scale),  dn = dy weight,
//   dx = rstd (dn - n mean(dn n)) + dresidual,   dweight = sum over tokens of dy n
//
// One pass: a row's dn and n live in the registers of a group of threads between the sum and
// the store.  CTAs walk over rows with a fixed set of columns for each thread, so dweight's
// sums stay in registers too; each group writes them once and norm_dweight adds the groups in
// a fixed order.  Bound by HBM: dy, dresidual, dx and h (or one byte a value) once each.
#include <algorithm>

#include "train_ops.cuh"

namespace qnf4 {
namespace {

constexpr int kDwCols = 32, kDwRows = 32;

// kNv = 0: rows longer than the registers of a CTA hold; the row is read twice and dweight's
// sums live in `partial`.
template <typename T, bool kVec, int kNv, bool kDw>
__global__ void __launch_bounds__(512) rms_norm_bwd(const NormBwdArgs a) {
  __shared__ float red[2 * 8 * 32];
  pdl_allow_next();
  pdl_wait();
  constexpr int kN = kNv > 0 ? kNv : 1;
  const int64_t C = (a.K + kActBlock - 1) / kActBlock * kActLanes;
  const int64_t nb = (a.K + kActBlock - 1) / kActBlock;
  const float invK = 1.0f / static_cast<float>(a.K);
  float* part = kDw ? a.partial + (static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y) * a.K : nullptr;
  constexpr bool kHoldW = kNv == 1 || kNv == 2;   // longer rows read the weight again (from L1)
  float dw[kN][8], w[kN][8];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (kHoldW) load8<float, kVec>(a.weight, threadIdx.x + static_cast<int64_t>(i) * blockDim.x, a.K, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  const int64_t rounds = (a.M + static_cast<int64_t>(gridDim.x) * blockDim.y - 1) / (static_cast<int64_t>(gridDim.x) * blockDim.y);
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t m = (it * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
    const bool on = m < a.M;
    const int64_t at = on ? m * a.K : 0;
    const float rstd = on ? a.rstd[m] : 0.0f;
    auto load_n = [&](int64_t c, float (&n)[8]) {
      if (a.h != nullptr) {
        load8<T, kVec>(static_cast<const T*>(a.h) + at, c, a.K, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] *= rstd;
      } else {
        const uint2 q = load_codes<kVec>(a.act.codes + at, c, a.K);
        const float sc = (c / kActLanes) * kActBlock < a.K ? a.act.scales[(on ? m : 0) * nb + c / kActLanes] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = code_value(q, j) * sc;
      }
    };
    auto finish = [&](int64_t c, const float (&g)[8], const float (&n)[8], float mean) {
      float o[8];
      if (a.dresidual != nullptr) load8<T, kVec>(static_cast<const T*>(a.dresidual) + at, c, a.K, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = rstd * (g[j] - n[j] * mean);
        o[j] = a.dresidual != nullptr ? d + o[j] : d;
      }
      store8<T, kVec>(static_cast<T*>(a.dx) + at, c, a.K, o);
    };
    float s = 0.0f;
    if (kNv > 0) {
      float g[kN][8], n[kN][8];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int64_t c = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
        if (on) {
          load8<T, kVec>(static_cast<const T*>(a.dy) + at, c, a.K, g[i]);
          load_n(c, n[i]);
          if (!kHoldW) load8<float, kVec>(a.weight, c, a.K, w[0]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (kDw) dw[i][j] = fmaf(g[i][j], n[i][j], dw[i][j]);
            g[i][j] *= w[kHoldW ? i : 0][j];
            s = fmaf(g[i][j], n[i][j], s);
          }
        }
      }
      const float mean = group_sum(s, red, static_cast<int>(it & 1)) * invK;
      if (on) {
#pragma unroll
        for (int i = 0; i < kN; ++i) finish(threadIdx.x + static_cast<int64_t>(i) * blockDim.x, g[i], n[i], mean);
      }
    } else {
      float g[8], n[8];
      auto load_g = [&](int64_t c) {
        load8<T, kVec>(static_cast<const T*>(a.dy) + at, c, a.K, g);
        load_n(c, n);
      };
      if (on) {
        for (int64_t c = threadIdx.x; c < C; c += blockDim.x) {
          float wc[8];
          load_g(c);
          load8<float, kVec>(a.weight, c, a.K, wc);
          if (kDw) {
            float p[8];
            if (it > 0) load8<float, kVec>(part, c, a.K, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = fmaf(g[j], n[j], it > 0 ? p[j] : 0.0f);
            store8<float, kVec>(part, c, a.K, p);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) s = fmaf(g[j] * wc[j], n[j], s);
        }
      }
      const float mean = group_sum(s, red, static_cast<int>(it & 1)) * invK;
      if (on) {
        for (int64_t c = threadIdx.x; c < C; c += blockDim.x) {
          float wc[8];
          load_g(c);
          load8<float, kVec>(a.weight, c, a.K, wc);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] *= wc[j];
          finish(c, g, n, mean);
        }
      }
    }
  }
  if (kDw && kNv > 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      store8<float, kVec>(part, threadIdx.x + static_cast<int64_t>(i) * blockDim.x, a.K, dw[i]);
  }
}

// dweight[k] = sum of the P groups' parts: 32 columns a CTA, 32 threads down the groups, then
// their sums in order.
__global__ void norm_dweight(const float* part, int64_t P, int64_t K, float* dweight) {
  __shared__ float red[kDwRows][kDwCols];
  pdl_allow_next();
  pdl_wait();
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kDwCols + threadIdx.x;
  float s = 0.0f;
  if (k < K)
    for (int64_t q = threadIdx.y; q < P; q += kDwRows) s += part[q * K + k];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && k < K) {
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < kDwRows; ++q) t += red[q][threadIdx.x];
    dweight[k] = t;
  }
}

struct BwdShape {
  int nv, grid;
  RowShape row;
};
BwdShape bwd_shape(int64_t M, int64_t K) {
  const int64_t C = (K + kActBlock - 1) / kActBlock * kActLanes;
  BwdShape b;
  b.nv = C <= 512 ? 1 : C <= 1024 ? 2 : C <= 2048 ? 4 : 0;
  b.row = b.nv > 0 ? row_shape(C, b.nv) : RowShape{512, 1};
  // about 1024 threads an SM, each walking over rows
  const int64_t ctas = static_cast<int64_t>(device_sm_count()) * std::max(1, 1024 / (b.row.G * b.row.R));
  b.grid = static_cast<int>(std::min(ctas, (M + b.row.R - 1) / b.row.R));
  return b;
}

template <typename T, bool kVec, bool kDw>
cudaError_t launch(const NormBwdArgs& a, cudaStream_t st) {
  const BwdShape b = bwd_shape(a.M, a.K);
  const dim3 grid(static_cast<unsigned>(b.grid)), block(b.row.G, b.row.R);
  cudaError_t e;
  note_launch();
  switch (b.nv) {
    case 1: e = launch_pdl(rms_norm_bwd<T, kVec, 1, kDw>, grid, block, 0, st, 1, a); break;
    case 2: e = launch_pdl(rms_norm_bwd<T, kVec, 2, kDw>, grid, block, 0, st, 1, a); break;
    case 4: e = launch_pdl(rms_norm_bwd<T, kVec, 4, kDw>, grid, block, 0, st, 1, a); break;
    default: e = launch_pdl(rms_norm_bwd<T, kVec, 0, kDw>, grid, block, 0, st, 1, a); break;
  }
  if (e != cudaSuccess || !kDw) return e;
  note_launch();
  return launch_pdl(norm_dweight, dim3(static_cast<unsigned>((a.K + kDwCols - 1) / kDwCols)), dim3(kDwCols, kDwRows), 0,
                    st, 1, static_cast<const float*>(a.partial), static_cast<int64_t>(b.grid) * b.row.R, a.K, a.dweight);
}

template <typename T>
cudaError_t pick(const NormBwdArgs& a, cudaStream_t st) {
  const bool vec = a.K % 8 == 0;
  if (a.dweight != nullptr) return vec ? launch<T, true, true>(a, st) : launch<T, false, true>(a, st);
  return vec ? launch<T, true, false>(a, st) : launch<T, false, false>(a, st);
}

}  // namespace

size_t rms_norm_bwd_ws_bytes(int64_t M, int64_t K) {
  if (M == 0) return 0;
  const BwdShape b = bwd_shape(M, K);
  return sizeof(float) * static_cast<size_t>(b.grid) * b.row.R * static_cast<size_t>(K);
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, nf4_dtype dt, cudaStream_t st) {
  if (a.M == 0) return a.dweight != nullptr ? cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.K, st) : cudaSuccess;
  switch (dt) {
    case NF4_F32: return pick<float>(a, st);
    case NF4_BF16: return pick<__nv_bfloat16>(a, st);
    default: return pick<__half>(a, st);
  }
}

}  // namespace qnf4
