// Layers of at most 64 inputs and outputs, in fp32: a file for each type, so that they compile side by side.
#include "linear_rows_kernels.h"

int launch_linear_rows_f32(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream) {
  return run_rows<float>(d, x, w, l, y, stream);
}
int launch_linear_rows_bwd_f32(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                                void *dw, void *db, void *ws, hipStream_t stream) {
  return run_rows_bwd<float>(d, dy, x, w, l, dx, dw, db, ws, stream);
}
