// Host-side launchers of the embedding and layer norm kernels (internal to libzs), apart from
// those of the update: measurements of the update's kernels are tied to the header that they include.
// Each launcher assumes its arguments were validated by the C-ABI entry point.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zs.h"

namespace zs {

// Workspace of the embedding's gradient over n tokens of a [vocab, dim] table:
// where each array starts (bytes from the workspace's start) and how the work
// is cut. Depends on the sizes alone, so the sums have one order.
struct EmbedPlan {
  int chunk;         // sorted entries per chunk (a workgroup's)
  int64_t chunks;    // chunks of the n entries
  int64_t pitch;     // fp32 values per partial row (dim rounded up to 8)
  int bits, passes, digit;  // bits of a key, passes of the sort, bits of a pass's digit
  int64_t tiles;     // tiles of the sort's passes
  int64_t keys[2], pos[2], counts, totals, touched, partials, bytes;
};
EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t dim);

hipError_t launch_embed_forward(const void* table, int dtype, int64_t vocab, int64_t dim, int64_t table_ld,
                                const void* pos_table, int64_t pos_rows, int64_t pos_ld, const void* tokens,
                                const void* positions, int index_type, int64_t n, float scale, void* out,
                                int out_dtype, int64_t out_ld, hipStream_t s);

hipError_t launch_embed_backward(const void* dout, int dtype, int64_t dout_ld, const void* tokens, int index_type,
                                 int64_t n, int64_t vocab, int64_t dim, int64_t padding_idx, float scale, void* grad,
                                 int grad_dtype, int64_t grad_ld, bool first, void* workspace, hipStream_t s);

// Workgroups of the layer norm's backward pass, each leaving one partial sum
// per column of the weight's and of the bias's gradient, and the partials'
// row length.
struct LnPlan {
  int64_t parts;
  int64_t pitch;
};
LnPlan ln_plan(int64_t rows, int64_t dim);

hipError_t launch_layer_norm_forward(const void* x, int dtype, int64_t x_ld, const void* w, const void* b, int wdtype,
                                     int64_t rows, int64_t dim, float eps, void* y, int64_t y_ld, float* mean,
                                     float* rstd, hipStream_t s);

hipError_t launch_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int dtype,
                                      const void* w, int wdtype, const float* mean, const float* rstd, int64_t rows,
                                      int64_t dim, void* dx, int64_t dx_ld, void* dw, void* db, int grad_dtype,
                                      bool first, void* workspace, hipStream_t s);

}  // namespace zs
