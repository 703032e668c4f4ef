// Layers of at most 64 inputs and outputs (linear_rows_kernels.h).
#pragma once
#include "linear_common.h"

// Arrays of fewer than eight elements, which a 16-byte access would pass, go the other way.
static inline bool linear_by_rows(const splat_dense *d) {
  return d->in >= 1 && d->in <= 64 && d->out <= 64 && d->rows * (d->in < d->out ? d->in : d->out) >= 8;
}

// The forward also of up to 256 outputs, in slices of 64 that each read x again, where rows are
// many: 1M of 32 to 256 bf16 with silu 164 us, 233 by tiles; 1M of 64 to 128 fp16 123 and 187.
// 20000 rows of 64 to 256 take 14 either way, and with dropout, which leaves the kernel too few
// registers there, 300000 of 64 to 128 bf16, trained, 260 and 247.
static inline bool linear_forward_by_rows(const splat_dense *d) {
  return linear_by_rows(d) || (d->in >= 1 && d->in <= 64 && d->out > 64 && d->out <= 256 && d->rows >= 65536 && d->drop.p == 0.0);
}

// Workgroups of the backward at most, each with sums of its own.
static inline int linear_rows_groups(const splat_dense *d) {
  const int64_t g = (d->rows + 63) / 64, most = d->in <= 32 && d->out <= 32 ? 1024 : 512;
  return (int)(g < most ? g : most);
}
static inline size_t linear_rows_workspace_bytes(const splat_dense *d) {
  return ws_align(sizeof(float) * (size_t)linear_rows_groups(d) * (d->in + 1) * d->out);
}

int launch_linear_rows_f32(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream);
int launch_linear_rows_bwd_f32(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                               void *dw, void *db, void *ws, hipStream_t stream);
int launch_linear_rows_f16(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream);
int launch_linear_rows_bwd_f16(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                               void *dw, void *db, void *ws, hipStream_t stream);
int launch_linear_rows_bf16(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream);
int launch_linear_rows_bwd_bf16(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                               void *dw, void *db, void *ws, hipStream_t stream);
