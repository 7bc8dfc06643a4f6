// RMS norm with the residual's addition and an 8-bit checkpoint of the normalised row.
//
//   h = x + residual (fp32),  rstd = 1 / sqrt(mean h^2 + eps),  n = h rstd,  y = n weight
//
// One pass: a row lives in the registers of a group of threads (kNv chunks of 8 values each)
// from its load to the stores of h, y and n's codes.  Bound by HBM: x, residual, h and y once
// each, one byte a value and 4 / 128 for the checkpoint.  h is rounded when it is stored; the
// norm is taken of the fp32 sum.
#include "train_ops.cuh"

namespace qnf4 {
namespace {

// kNv = 0: rows longer than the registers of a CTA hold; the row is read twice.
template <typename T, bool kVec, int kNv>
__global__ void __launch_bounds__(512) rms_norm_fwd(const NormFwdArgs a, int* status) {
  __shared__ float red[2 * 8 * 32];
  pdl_allow_next();
  pdl_wait();
  const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool on = m < a.M;
  const int64_t C = (a.K + kActBlock - 1) / kActBlock * kActLanes;   // whole blocks of lanes
  const int64_t at = m * a.K;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* res = static_cast<const T*>(a.residual) + (a.residual != nullptr ? at : 0);
  auto load = [&](int64_t c, float (&v)[8]) {
    load8<T, kVec>(x, c, a.K, v);
    if (a.residual != nullptr) {
      float r[8];
      load8<T, kVec>(res, c, a.K, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
  };
  auto finish = [&](int64_t c, const float (&h)[8], float rstd) {
    float n[8], y[8], w[8];
    load8<float, kVec>(a.weight, c, a.K, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = h[j] * rstd, y[j] = n[j] * w[j];
    if (on) store8<T, kVec>(static_cast<T*>(a.y) + at, c, a.K, y);
    if (on && a.h != nullptr) store8<T, kVec>(static_cast<T*>(a.h) + at, c, a.K, h);
    if (a.act.codes != nullptr) {
      const Quantized q = quantize_block(n);
      if (on) store_codes<kVec>(a.act, m, c, a.K, q);
      if (on && q.bad) atomicCAS(status, 0, static_cast<int>(NF4_ERR_NONFINITE));
    }
  };
  float ss = 0.0f;
  if (kNv > 0) {
    float h[kNv > 0 ? kNv : 1][8];
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
      if (on) load(c, h[i]);
      else
        for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    ss = group_sum(ss, red, 0);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.K) + a.eps);
    if (on && threadIdx.x == 0) a.rstd[m] = rstd;
#pragma unroll
    for (int i = 0; i < kNv; ++i) finish(threadIdx.x + static_cast<int64_t>(i) * blockDim.x, h[i], rstd);
  } else {
    float h[8];
    for (int64_t c = threadIdx.x; c < C; c += blockDim.x) {   // one row a CTA: `on` holds
      load(c, h);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[j], h[j], ss);
    }
    ss = group_sum(ss, red, 0);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.K) + a.eps);
    if (threadIdx.x == 0) a.rstd[m] = rstd;
    // every lane of a warp runs the same rounds: the quantizer shuffles
    for (int64_t c0 = 0; c0 < C; c0 += blockDim.x) {
      load(c0 + threadIdx.x, h);
      finish(c0 + threadIdx.x, h, rstd);
    }
  }
}

template <typename T, bool kVec>
cudaError_t launch(const NormFwdArgs& a, int* status, cudaStream_t st) {
  const int64_t C = (a.K + kActBlock - 1) / kActBlock * kActLanes;
  const int nv = C <= 512 ? 1 : C <= 1024 ? 2 : C <= 2048 ? 4 : 0;
  const RowShape s = nv > 0 ? row_shape(C, nv) : RowShape{512, 1};
  const dim3 grid(static_cast<unsigned>((a.M + s.R - 1) / s.R)), block(s.G, s.R);
  note_launch();
  switch (nv) {
    case 1: return launch_pdl(rms_norm_fwd<T, kVec, 1>, grid, block, 0, st, 1, a, status);
    case 2: return launch_pdl(rms_norm_fwd<T, kVec, 2>, grid, block, 0, st, 1, a, status);
    case 4: return launch_pdl(rms_norm_fwd<T, kVec, 4>, grid, block, 0, st, 1, a, status);
    default: return launch_pdl(rms_norm_fwd<T, kVec, 0>, grid, block, 0, st, 1, a, status);
  }
}

}  // namespace

cudaError_t launch_rms_norm_fwd(const NormFwdArgs& a, nf4_dtype dt, int* status, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  const bool vec = a.K % 8 == 0;
  switch (dt) {
    case NF4_F32: return vec ? launch<float, true>(a, status, st) : launch<float, false>(a, status, st);
    case NF4_BF16: return vec ? launch<__nv_bfloat16, true>(a, status, st) : launch<__nv_bfloat16, false>(a, status, st);
    default: return vec ? launch<__half, true>(a, status, st) : launch<__half, false>(a, status, st);
  }
}

}  // namespace qnf4
