// Dropout whose mask is drawn from a counter and never stored, with a residual added in the
// same pass: y = residual + keep(u_i) x / (1 - p). The gradient is the same call on d_y.
//
// Bound by memory: 2 (with a residual 3) accesses an element, beside one Philox draw of ten
// rounds per eight elements: 20 products of 32 x 32 to 64 bits, which issue at a quarter of
// the rate, and 20 three-way exclusive ors. 66M fp16 elements with a residual: 68 us, 5.9 TB/s,
// with inputs that change from call to call; 60 us with the same ones, part of which the caches
// hold (70 when the second draw, for ties, was made by all).
#include "eight.h"
#include "random.h"

namespace {

constexpr int DR_THREADS = 256;

struct DropoutArgs {
  const void *x, *res;
  void *y;
  int64_t rows, cols, xs, rs, ys;
  int64_t blocks;                // of eight elements
  DropArgs drop;
};

// Packed arrays: a thread takes eight elements, at any alignment.
template <typename T, bool RES, bool DRAW>
__global__ __launch_bounds__(DR_THREADS) void k_dropout(DropoutArgs a) {
  const DropKey key = DRAW ? drop_key(a.drop) : DropKey{};
  const int64_t n = a.rows * a.cols;
  for (int64_t b = (int64_t)blockIdx.x * DR_THREADS + threadIdx.x; b < a.blocks; b += (int64_t)gridDim.x * DR_THREADS) {
    const int64_t at = b * 8;
    const int m = n - at < 8 ? (int)(n - at) : 8;
    float v[8], r[8];
    load8<T>((const T *)a.x + at, m, v);
    if constexpr (RES) load8<T>((const T *)a.res + at, m, r);
    if constexpr (DRAW) drop8<true>(v, at, a.drop, key);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = RES ? v[j] + r[j] : v[j];
    stream8<T>((T *)a.y + at, m, v);
  }
}

// Rows a stride apart: the same eight elements, each at its own row.
template <typename T>
__global__ __launch_bounds__(DR_THREADS) void k_dropout_rows(DropoutArgs a, bool draw) {
  const DropKey key = draw ? drop_key(a.drop) : DropKey{};
  const int64_t n = a.rows * a.cols;
  for (int64_t b = (int64_t)blockIdx.x * DR_THREADS + threadIdx.x; b < a.blocks; b += (int64_t)gridDim.x * DR_THREADS) {
    const int64_t at = b * 8;
    int64_t row[8], col[8];
    float v[8];
    row[0] = at / a.cols;
    col[0] = at - row[0] * a.cols;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (j > 0) {
        const bool next = col[j - 1] + 1 == a.cols;
        row[j] = row[j - 1] + (next ? 1 : 0);
        col[j] = next ? 0 : col[j - 1] + 1;
      }
      v[j] = at + j < n ? (float)((const T *)a.x)[row[j] * a.xs + col[j]] : 0.0f;
    }
    if (draw) drop8<true>(v, at, a.drop, key);
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (at + j < n) {
        const float r = a.res ? (float)((const T *)a.res)[row[j] * a.rs + col[j]] : 0.0f;
        ((T *)a.y)[row[j] * a.ys + col[j]] = (T)(a.res ? v[j] + r : v[j]);
      }
  }
}

template <typename T>
int run_dropout(const DropoutArgs &a, bool packed, bool draw, hipStream_t stream) {
  const int64_t need = (a.blocks + DR_THREADS - 1) / DR_THREADS;
  const dim3 grid((unsigned)(need < 16384 ? need : 16384)), block(DR_THREADS);
  if (!packed) hipLaunchKernelGGL(k_dropout_rows<T>, grid, block, 0, stream, a, draw);
  else if (a.res && draw) hipLaunchKernelGGL((k_dropout<T, true, true>), grid, block, 0, stream, a);
  else if (a.res) hipLaunchKernelGGL((k_dropout<T, true, false>), grid, block, 0, stream, a);
  else if (draw) hipLaunchKernelGGL((k_dropout<T, false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_dropout<T, false, false>), grid, block, 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

}  // namespace

int launch_dropout(const splat_drop *drop, int dtype, int64_t rows, int64_t cols, const void *x, int64_t xs,
                   const void *res, int64_t rs, void *y, int64_t ys, hipStream_t stream) {
  DropoutArgs a = {x, res, y, rows, cols, xs, rs, ys, (rows * cols + 7) / 8, drop_args(drop)};
  const bool packed = xs == cols && ys == cols && (!res || rs == cols), draw = drop->p > 0.0;
  if (dtype == SPLAT_F32) return run_dropout<float>(a, packed, draw, stream);
  if (dtype == SPLAT_F16) return run_dropout<f16_t>(a, packed, draw, stream);
  return run_dropout<bf16_t>(a, packed, draw, stream);
}
