// Dropout whose mask is drawn from a counter and never stored, with a residual added in the
// same pass: y = residual + keep(u_i) x / (1 - p). The gradient is the same call on d_y.
//
// Bound by memory: 2 (with a residual 3) accesses an element, beside one Philox draw of ten
// rounds per eight elements: 20 products of 32 x 32 to 64 bits, which issue at a quarter of
// the rate, and 20 three-way exclusive ors.
#include "learn_common.h"
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

template <typename T>
__device__ __forceinline__ float dropped(float x, float r, bool res, bool keep, float scale) {
  const float v = keep ? x * scale : 0.0f;
  return res ? v + r : v;
}

// Packed arrays: a thread takes eight elements at any alignment.
template <typename T, bool RES, bool DRAW>
__global__ __launch_bounds__(DR_THREADS) void k_dropout(DropoutArgs a) {
  constexpr int N = 16 / sizeof(T), M = 8 / N;
  const DropKey key = DRAW ? drop_key(a.drop) : DropKey{};
  const int64_t n = a.rows * a.cols;
  const T *x = (const T *)a.x, *r = (const T *)a.res;
  T *y = (T *)a.y;
  for (int64_t b = (int64_t)blockIdx.x * DR_THREADS + threadIdx.x; b < a.blocks; b += (int64_t)gridDim.x * DR_THREADS) {
    const int64_t at = b * 8;
    if (at + 8 <= n) {
      Raw<T, N> xv[M], rv[M] = {};
#pragma unroll
      for (int m = 0; m < M; m++) xv[m] = *reinterpret_cast<const typename Loose<T, N>::type *>(x + at + m * N);
      if constexpr (RES) {
#pragma unroll
        for (int m = 0; m < M; m++) rv[m] = *reinterpret_cast<const typename Loose<T, N>::type *>(r + at + m * N);
      }
      const uint32_t keep = DRAW ? drop_keeps((uint64_t)b, a.drop, key) : 0xFFu;
#pragma unroll
      for (int m = 0; m < M; m++) {
        float f[N], q[N], o[N];
        to_f32<T, N>(xv[m], f);
        to_f32<T, N>(rv[m], q);
#pragma unroll
        for (int j = 0; j < N; j++) o[j] = dropped<T>(f[j], q[j], RES, keep >> (m * N + j) & 1, a.drop.scale);
        stream_loose<T, N>(y + at + m * N, o);
      }
    } else {
      const uint32_t keep = DRAW ? drop_keeps((uint64_t)b, a.drop, key) : 0xFFu;
      for (int j = 0; at + j < n; j++)
        y[at + j] = (T)dropped<T>((float)x[at + j], RES ? (float)r[at + j] : 0.0f, RES, keep >> j & 1, a.drop.scale);
    }
  }
}

// Rows a stride apart: the same eight elements, each at its own row.
template <typename T>
__global__ __launch_bounds__(DR_THREADS) void k_dropout_rows(DropoutArgs a, bool draw) {
  const DropKey key = draw ? drop_key(a.drop) : DropKey{};
  const int64_t n = a.rows * a.cols;
  const T *x = (const T *)a.x, *r = (const T *)a.res;
  T *y = (T *)a.y;
  for (int64_t b = (int64_t)blockIdx.x * DR_THREADS + threadIdx.x; b < a.blocks; b += (int64_t)gridDim.x * DR_THREADS) {
    const int64_t at = b * 8;
    const uint32_t keep = draw ? drop_keeps((uint64_t)b, a.drop, key) : 0xFFu;
    int64_t row = at / a.cols, col = at - row * a.cols;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (at + j >= n) break;
      y[row * a.ys + col] = (T)dropped<T>((float)x[row * a.xs + col], r ? (float)r[row * a.rs + col] : 0.0f, r != nullptr,
                                          keep >> j & 1, a.drop.scale);
      if (++col == a.cols) {
        col = 0;
        row++;
      }
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
