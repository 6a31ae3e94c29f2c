// Host-side launchers of the loss over a large vocabulary (internal to libzs). Each assumes
// its arguments were validated by the C-ABI entry point.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zs.h"

namespace zs {

// Workspace of the loss of n tokens over [vocab, dim]: where each array starts (bytes from the
// workspace's start) and how the work is cut. Depends on the sizes and types alone, so the sums
// have one order.
struct HeadPlan {
  int planes;        // bf16 planes of the hidden states and of the head's weight
  int gplanes;       // of the logits' gradient
  bool half;         // fp32 logits from pairs of fp16
  bool few;          // few tokens' fp32 gradients take the head as it lies
  int64_t np;        // tokens rounded up to 64
  int64_t dp;        // dim rounded up to 64
  int64_t dq;        // dim rounded up to 4: a row of the hidden states' gradient in fp32
  int64_t piece;     // rows of the head at a time (a multiple of 256), where it is laid out anew or has a gradient
  int64_t pieces;
  int splits;        // parts of the sum over a piece for the hidden states' gradient
  int64_t label, coef, lse, rest, map, inverse, count, own, parts, hidden, weight, hpower, wpower, hhalf, whalf, z,
      g, dhidden, bytes;
};
HeadPlan head_plan(int64_t n, int64_t vocab, int64_t dim, int dtype, int grad_dtype);  // grad_dtype -1: the loss alone

hipError_t launch_head_forward(const void* hidden, int64_t hidden_ld, int dtype, const void* weight,
                               int64_t weight_ld, const void* labels, int index_type, int64_t n, int64_t vocab,
                               int64_t dim, float* loss, float* lse, void* workspace, hipStream_t s);

hipError_t launch_head_backward(const void* hidden, int64_t hidden_ld, int dtype, const void* weight,
                                int64_t weight_ld, const void* labels, int index_type, const float* lse,
                                const float* dloss, float scale, int64_t n, int64_t vocab, int64_t dim, void* dhidden,
                                int64_t dhidden_ld, void* dweight, int grad_dtype, int64_t dweight_ld, bool first,
                                void* workspace, hipStream_t s);

}  // namespace zs
