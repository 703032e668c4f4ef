// Layers of at most 64 inputs and outputs (linear_rows.hip).
#pragma once
#include "linear_common.h"

bool linear_by_rows(const splat_dense *d);
size_t linear_rows_workspace_bytes(const splat_dense *d);   // of the backward; the forward needs none
int launch_linear_rows(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream);
int launch_linear_rows_bwd(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                           void *dw, void *db, void *ws, hipStream_t stream);
