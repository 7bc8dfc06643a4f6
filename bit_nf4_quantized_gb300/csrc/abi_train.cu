// C ABI of the operators around the linear: argument checks, workspaces and dispatch.
#include <cmath>

#include "lm_loss.cuh"
#include "train_ops.cuh"

using namespace qnf4;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool known(nf4_dtype d) { return d == NF4_F32 || d == NF4_BF16 || d == NF4_F16; }
nf4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NF4_OK : NF4_ERR_CUDA; }

// A [M, K] tensor's sizes: products and offsets stay far inside 64 bits.
nf4_status check_rows(int64_t M, int64_t K) {
  if (M < 0 || K <= 0) return NF4_ERR_ARG;
  if (M > (int64_t(1) << 40) / K) return NF4_ERR_SHAPE;
  return NF4_OK;
}

nf4_status check_act8(const qlora_act8* a, int64_t M, int64_t K) {
  if (a == nullptr) return NF4_ERR_ARG;
  if (a->rows != M || a->cols != K) return NF4_ERR_SHAPE;
  if (M > 0 && (a->codes == nullptr || a->scales == nullptr)) return NF4_ERR_ARG;
  if (!aligned16(a->codes) || !aligned16(a->scales)) return NF4_ERR_ALIGN;
  return NF4_OK;
}

}  // namespace

extern "C" {

int64_t qlora_act8_scales(int64_t rows, int64_t cols) {
  return rows < 0 || cols <= 0 ? 0 : rows * ((cols + kActBlock - 1) / kActBlock);
}

nf4_status qlora_act8_quantize(const void* x, nf4_dtype dtype, const qlora_act8* out, void* stream) {
  if (out == nullptr) return NF4_ERR_ARG;
  const int64_t M = out->rows, K = out->cols;
  nf4_status st = check_rows(M, K);
  if (st != NF4_OK) return st;
  if (!known(dtype)) return NF4_ERR_DTYPE;
  if ((st = check_act8(out, M, K)) != NF4_OK) return st;
  if (M == 0) return NF4_OK;
  if (x == nullptr) return NF4_ERR_ARG;
  if (!aligned16(x)) return NF4_ERR_ALIGN;
  int* status = nullptr;
  if ((st = device_status_word(&status)) != NF4_OK) return st;
  return from_cuda(launch_act8_quantize(x, dtype, M, K, Act8View{out->codes, out->scales}, status,
                                        static_cast<cudaStream_t>(stream)));
}

nf4_status qlora_act8_dequantize(const qlora_act8* in, const float* weight, void* out, nf4_dtype dtype, void* stream) {
  if (in == nullptr) return NF4_ERR_ARG;
  const int64_t M = in->rows, K = in->cols;
  nf4_status st = check_rows(M, K);
  if (st != NF4_OK) return st;
  if (!known(dtype)) return NF4_ERR_DTYPE;
  if ((st = check_act8(in, M, K)) != NF4_OK) return st;
  if (M == 0) return NF4_OK;
  if (out == nullptr) return NF4_ERR_ARG;
  if (!aligned16(out) || !aligned16(weight)) return NF4_ERR_ALIGN;
  return from_cuda(launch_act8_dequantize(Act8View{in->codes, in->scales}, M, K, weight, out, dtype,
                                          static_cast<cudaStream_t>(stream)));
}

size_t qlora_act8_grad_a_workspace_bytes(int64_t M, int64_t K, int32_t rank) {
  if (check_rows(M, K) != NF4_OK || rank < 1 || rank > 256) return 0;
  return act8_grad_ws_bytes(M, K, rank);
}

nf4_status qlora_act8_grad_a(int32_t rank, float alpha, qlora_scale_mode mode, const float* G, const qlora_act8* x,
                             const float* x_weight, float* dA, void* ws, size_t ws_bytes, void* stream) {
  if (x == nullptr) return NF4_ERR_ARG;
  const int64_t M = x->rows, K = x->cols;
  nf4_status st = check_rows(M, K);
  if (st != NF4_OK) return st;
  if (rank < 1 || rank > 256 || !std::isfinite(alpha)) return NF4_ERR_ARG;
  if (mode != QLORA_SCALE_LORA && mode != QLORA_SCALE_RSLORA) return NF4_ERR_ARG;
  if ((st = check_act8(x, M, K)) != NF4_OK) return st;
  if (dA == nullptr || (M > 0 && G == nullptr)) return NF4_ERR_ARG;
  if (!aligned16(dA) || !aligned16(G) || !aligned16(x_weight)) return NF4_ERR_ALIGN;
  const size_t need = act8_grad_ws_bytes(M, K, rank);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return NF4_ERR_WORKSPACE;
  if (!aligned16(ws)) return NF4_ERR_ALIGN;
  const float s = mode == QLORA_SCALE_LORA
                      ? alpha / static_cast<float>(rank)
                      : static_cast<float>(static_cast<double>(alpha) / std::sqrt(static_cast<double>(rank)));
  return from_cuda(launch_act8_grad(ActGradArgs{M, K, rank, s, G, Act8View{x->codes, x->scales}, x_weight, dA}, ws,
                                    static_cast<cudaStream_t>(stream)));
}

nf4_status qlora_rms_norm_fwd(int64_t M, int64_t K, float eps, nf4_dtype dtype, const void* x, const void* residual,
                              const float* weight, void* y, void* h, float* rstd, const qlora_act8* checkpoint,
                              void* stream) {
  nf4_status st = check_rows(M, K);
  if (st != NF4_OK) return st;
  if (!known(dtype)) return NF4_ERR_DTYPE;
  if (!std::isfinite(eps) || eps < 0.0f || weight == nullptr) return NF4_ERR_ARG;
  if (M > 0 && (x == nullptr || y == nullptr || rstd == nullptr)) return NF4_ERR_ARG;
  if (checkpoint != nullptr && (st = check_act8(checkpoint, M, K)) != NF4_OK) return st;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(y) || !aligned16(h) || !aligned16(rstd))
    return NF4_ERR_ALIGN;
  int* status = nullptr;
  if (M == 0) return NF4_OK;
  if ((st = device_status_word(&status)) != NF4_OK) return st;
  const NormFwdArgs a{M, K, eps, x, residual, weight, y, h, rstd,
                      checkpoint != nullptr ? Act8View{checkpoint->codes, checkpoint->scales} : Act8View{}};
  return from_cuda(launch_rms_norm_fwd(a, dtype, status, static_cast<cudaStream_t>(stream)));
}

size_t qlora_rms_norm_bwd_workspace_bytes(int64_t M, int64_t K) {
  return check_rows(M, K) != NF4_OK ? 0 : rms_norm_bwd_ws_bytes(M, K);
}

nf4_status qlora_rms_norm_bwd(int64_t M, int64_t K, nf4_dtype dtype, const void* dy, const void* h,
                              const qlora_act8* checkpoint, const float* rstd, const float* weight,
                              const void* dresidual, void* dx, float* dweight, void* ws, size_t ws_bytes,
                              void* stream) {
  nf4_status st = check_rows(M, K);
  if (st != NF4_OK) return st;
  if (!known(dtype)) return NF4_ERR_DTYPE;
  if (weight == nullptr || (h != nullptr && checkpoint != nullptr)) return NF4_ERR_ARG;
  if (checkpoint != nullptr && (st = check_act8(checkpoint, M, K)) != NF4_OK) return st;
  if (M > 0 && (dy == nullptr || rstd == nullptr || dx == nullptr || (h == nullptr && checkpoint == nullptr)))
    return NF4_ERR_ARG;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(rstd) || !aligned16(weight) || !aligned16(dresidual) ||
      !aligned16(dx) || !aligned16(dweight))
    return NF4_ERR_ALIGN;
  const size_t need = dweight != nullptr ? rms_norm_bwd_ws_bytes(M, K) : 0;
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return NF4_ERR_WORKSPACE;
  if (need > 0 && !aligned16(ws)) return NF4_ERR_ALIGN;
  const NormBwdArgs a{M, K, dy, h, checkpoint != nullptr ? Act8View{checkpoint->codes, checkpoint->scales} : Act8View{},
                      rstd, weight, dresidual, dx, dweight, static_cast<float*>(ws)};
  int* status = nullptr;
  if ((st = device_status_word(&status)) != NF4_OK) return st;
  return from_cuda(launch_rms_norm_bwd(a, dtype, status, static_cast<cudaStream_t>(stream)));
}

size_t qlora_lm_loss_workspace_bytes(int64_t M, int64_t V, int64_t D, int32_t stored, int32_t gradient) {
  if (M <= 0 || V <= 0 || D <= 0) return 0;
  return lm_loss_ws_bytes(M, V, D, stored != 0, gradient != 0);
}

nf4_status qlora_lm_loss(int64_t M, int64_t V, int64_t D, nf4_dtype compute, const void* x, const nf4_tensor* W,
                         const void* w16, const int64_t* targets, int64_t ignore_index, const float* grad_scale,
                         int32_t grad_scale_per_row, float* loss, float* lse, void* dx, void* ws, size_t ws_bytes,
                         void* stream) {
  if (M < 0 || V <= 0 || D <= 0) return NF4_ERR_ARG;
  if (compute != NF4_BF16 && compute != NF4_F16) return NF4_ERR_DTYPE;
  if (V > (int64_t(1) << 40) / D || V > (int64_t(1) << 30) || D > (int64_t(1) << 24) || M > (int64_t(1) << 40) / D)
    return NF4_ERR_SHAPE;
  nf4_status st;
  if (w16 == nullptr && (st = check_nf4_tensor(W, V * D)) != NF4_OK) return st;
  if (D < 64 || D % (w16 == nullptr ? 64 : 8) != 0) return NF4_ERR_SHAPE;
  if (M > 0 && (x == nullptr || targets == nullptr || loss == nullptr)) return NF4_ERR_ARG;
  if (!aligned16(x) || !aligned16(w16) || !aligned16(targets) || !aligned16(grad_scale) || !aligned16(loss) ||
      !aligned16(lse) || !aligned16(dx))
    return NF4_ERR_ALIGN;
  if (M == 0) return NF4_OK;
  const size_t need = lm_loss_ws_bytes(M, V, D, w16 == nullptr, dx != nullptr);
  if (ws == nullptr || ws_bytes < need) return NF4_ERR_WORKSPACE;
  if (!aligned16(ws)) return NF4_ERR_ALIGN;
  int* status = nullptr;
  if ((st = device_status_word(&status)) != NF4_OK) return st;
  LmLossArgs a{};
  a.M = M;
  a.V = V;
  a.D = D;
  a.f16 = compute == NF4_F16;
  a.x = x;
  a.w16 = w16;
  if (w16 == nullptr) a.W = nf4_view(W);
  a.targets = targets;
  a.ignore_index = ignore_index;
  a.grad_scale = grad_scale;
  a.grad_scale_per_row = grad_scale_per_row != 0;
  a.loss = loss;
  a.lse = lse;
  a.dx = dx;
  return from_cuda(lm_loss(a, ws, status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
