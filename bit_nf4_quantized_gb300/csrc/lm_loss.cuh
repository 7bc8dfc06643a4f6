// Softmax cross entropy of a frozen head over a large vocabulary, with its gradient.
#pragma once

#include "common.cuh"

namespace qnf4 {

struct LmLossArgs {
  int64_t M, V, D;
  bool f16;                 // x, the head and dx are IEEE half (else bf16)
  const void* x;            // [M, D]
  const void* w16;          // [V, D], or nullptr: W is decoded piece by piece
  Nf4View W;
  const int64_t* targets;   // [M]
  int64_t ignore_index;
  const float* grad_scale;  // [M] or [1], or nullptr: 1
  int grad_scale_per_row;
  float* loss;              // [M]
  float* lse;               // [M] or nullptr
  void* dx;                 // [M, D] or nullptr: no gradient
};

// stored: the head is given as NF4; grad: dx is asked for.
size_t lm_loss_ws_bytes(int64_t M, int64_t V, int64_t D, bool stored, bool grad);
cudaError_t lm_loss(const LmLossArgs& a, void* ws, int* status, cudaStream_t st);

}  // namespace qnf4
