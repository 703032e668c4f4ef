// Dense layers of a shading network: y = residual + drop(act(x W + b)) in one launch, and
// the gradient dz = drop'(dy) act'(z), dx = dz W^T, dW = x^T dz, db = sums of dz.
//
// Every product is C[i][j] = sum over c of Q[i][c] P[j][c] with j the axis along which C is
// stored: Q and P are x, W, dz or their transposes, read where they lie, whichever of
// their two axes is contiguous.
#include "linear_common.h"
#include "linear_rows.h"
#include "linear_tiles.h"

namespace {

// ---- dz and its column sums ------------------------------------------------------------

struct SlopeArgs {
  const void *dy, *z;            // z packed
  void *dz;                      // packed, or NULL: only the sums
  void *dz2;                     // what dz's rounding lost, or NULL
  float *sums;                   // [chunks][N], or NULL
  int64_t M, N, ys, chunk;       // rows per workgroup
  int act, draw;
  float part;                    // of dz that is stored
  DropArgs drop;
};

constexpr int SL_COLS = 64;      // columns per workgroup: eight threads a row, 32 rows at once

// dz = drop'(dy) act'(z) for some rows by 64 columns, and the columns' sums over them. 8191 x
// 4096 bf16 with gelu and dropout: 54 us, 3.7 TB/s; some 50 instructions a value take 45 of them.
template <typename T>
__global__ __launch_bounds__(LN_THREADS) void k_linear_slope(SlopeArgs a) {
  __shared__ float s[LN_THREADS / 8][SL_COLS + 1];
  const int c = (threadIdx.x & 7) * 8, r = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * SL_COLS + c, m0 = blockIdx.y * a.chunk;
  const int64_t m1 = m0 + a.chunk < a.M ? m0 + a.chunk : a.M;
  const int n = col >= a.N ? 0 : a.N - col < 8 ? (int)(a.N - col) : 8;
  DropKey key = {};
  if (a.draw) key = drop_key(a.drop);
  float t[8] = {};
  if (n > 0) {
    // two rows at once: their loads are on the way together
    constexpr int AT_ONCE = 2, STEP = LN_THREADS / 8;
    for (int64_t m = m0 + r; m < m1; m += AT_ONCE * STEP) {
      float d[AT_ONCE][8], z[AT_ONCE][8];
#pragma unroll
      for (int u = 0; u < AT_ONCE; u++) {
        const int64_t k = m + u * STEP;
        const int w = k < m1 ? n : 0;
        load8<T>((const T *)a.dy + k * a.ys + col, w, d[u]);
        if (a.act != SPLAT_ACT_NONE) load8<T>((const T *)a.z + k * a.N + col, w, z[u]);
      }
#pragma unroll
      for (int u = 0; u < AT_ONCE; u++) {
        const int64_t k = m + u * STEP;
        if (k >= m1) break;
        if (a.act != SPLAT_ACT_NONE) slope_times<T>(d[u], z[u], a.act);
        if (a.draw) drop8<false>(d[u], k * a.N + col, a.drop, key);
        if (a.dz) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = d[u][j] * a.part;
          store8<T>((T *)a.dz + k * a.N + col, n, v);
        }
        if constexpr (sizeof(T) == 2) {
          if (a.dz2) {
            word4 hi, lo;
            float v[8];
            split8<T>(d[u], hi, lo);
            const Pack<T, 8> l = __builtin_bit_cast(Pack<T, 8>, lo);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = (float)l.v[j];
            store8<T>((T *)a.dz2 + k * a.N + col, n, v);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; j++) t[j] += d[u][j];
      }
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int j = 0; j < 8; j++) s[r][c + j] = t[j];
  __syncthreads();
  const int64_t mine = (int64_t)blockIdx.x * SL_COLS + threadIdx.x;
  if (threadIdx.x < SL_COLS && mine < a.N) {
    float v = 0.0f;
    for (int k = 0; k < LN_THREADS / 8; k++) v += s[k][threadIdx.x];
    a.sums[blockIdx.y * a.N + mine] = v;
  }
}

// db: the chunks' sums, 32 columns by 8 slices of the chunks a workgroup, each in order.
template <typename T>
__global__ __launch_bounds__(LN_THREADS) void k_linear_bias(const float *sums, int64_t chunks, int64_t N, void *db, int f32,
                                                            float scale) {
  __shared__ float s[8][33];
  const int e = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + e;
  float v = 0.0f;
  if (col < N) {
#pragma unroll 4
    for (int64_t k = l; k < chunks; k += 8) v += sums[k * N + col];
  }
  s[l][e] = v;
  __syncthreads();
  if (l > 0 || col >= N) return;
#pragma unroll
  for (int k = 1; k < 8; k++) v += s[k][e];
  v *= scale;
  if (f32) ((float *)db)[col] = v;
  else ((T *)db)[col] = (T)v;
}

// C[i][j] of no rows.
template <typename T>
__global__ __launch_bounds__(LN_THREADS) void k_linear_zero(T *c, int64_t I, int64_t J, int64_t cs) {
  for (int64_t t = (int64_t)blockIdx.x * LN_THREADS + threadIdx.x; t < I * J; t += (int64_t)gridDim.x * LN_THREADS)
    c[t / J * cs + t % J] = (T)0.0f;
}

// ---- host ------------------------------------------------------------------------------

unsigned blocks_for(int64_t items) {
  const int64_t b = (items + LN_THREADS - 1) / LN_THREADS;
  return (unsigned)(b < 1 ? 1 : b < 65536 ? b : 65536);
}

int64_t slope_chunks(int64_t M, int64_t N) {
  const int64_t cols = (N + SL_COLS - 1) / SL_COLS;
  int64_t chunks = (2048 + cols - 1) / cols, most = (M + 63) / 64;
  if (chunks > most) chunks = most;
  return chunks < 1 ? 1 : chunks;
}

// W as [in][out], `out` contiguous, or its transpose.
bool w_by_out(int64_t si, int64_t so) { return so == 1 && si != 1; }

// Parts of dz. None's and relu's is exact in one. With silu or gelu one rounding of it adds as much
// error to dx and dW as their own rounding does (1.41 times it in all), and a second part doubles the
// products' operations. fp16 has not the range for one part. bf16 takes two as long as the second costs
// 15 us at most, and one for larger layers (2048 x 512 to 512: 38 us of backward and 31 with one; 2048 x
// 1024 to 1024 55 and 41; 8192 x 1024 to 2048 208 and 125), and two where W is small and dW's few values
// are sums over long arrays, at any length (1M x 100 to 72: 508 and 371).
int parts_of(const splat_dense *d) {
  if (slope_of_bits(d->act) || d->dtype == SPLAT_F32) return 1;
  const int64_t weights = (int64_t)d->in * d->out;
  const bool large = weights >= (1 << 15) && d->rows >= ((1ll << 31) + weights - 1) / weights;
  return d->dtype == SPLAT_BF16 && large ? 1 : 2;
}

struct Plan {
  size_t pre, dz, sums, part, total;
};
Plan plan_of(const splat_dense *d, bool bwd) {
  Plan p = {};
  const int64_t M = d->rows, N = d->out, K = d->in;
  if (M == 0 || N == 0) return p;
  auto most = [&](size_t v) { if (v > p.part) p.part = v; };
  most(product_part_bytes(M, N, K, 1, d->dtype));
  if (bwd) {
    const size_t e = dtype_bytes(d->dtype);
    const int parts = parts_of(d);
    if (d->act != SPLAT_ACT_NONE) p.pre = ws_align((size_t)M * N * e);
    if (d->act != SPLAT_ACT_NONE || d->drop.p > 0.0) p.dz = parts * ws_align((size_t)M * N * e);
    p.sums = ws_align(sizeof(float) * (size_t)slope_chunks(M, N) * N);
    most(product_part_bytes(M, K, N, parts, d->dtype));
    most(product_part_bytes(K, N, M, parts, d->dtype));
    most(product_part_bytes(N, K, M, parts, d->dtype));
  }
  p.total = p.pre + p.dz + p.sums + p.part;
  return p;
}

template <typename T>
int forward(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, int64_t ys, float *part,
            hipStream_t stream) {
  ProductArgs a = {};
  a.I = d->rows;
  a.J = d->out;
  a.K = d->in;
  a.q = {x, d->x_stride, 0};
  a.parts = 1;
  a.c = y;
  a.cs = ys;
  a.part = part;
  a.layer = l;
  if (w_by_out(d->w_in_stride, d->w_out_stride)) {
    a.p = {w, d->w_in_stride, 0};
    return launch_product<T>(a, false, true, OUT_LAYER, stream);
  }
  a.p = {w, d->w_out_stride, 0};
  return launch_product<T>(a, false, false, OUT_LAYER, stream);
}

template <typename T>
int zero(void *c, int64_t I, int64_t J, int64_t cs, hipStream_t stream) {
  if (!c || I == 0 || J == 0) return SPLAT_OK;
  hipLaunchKernelGGL(k_linear_zero<T>, dim3(blocks_for(I * J)), dim3(LN_THREADS), 0, stream, (T *)c, I, J, cs);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T>
int backward(const splat_dense *d, const void *dy, const void *x, const void *w, const void *bias, const void *pre,
             void *dx, void *dw, void *db, void *ws, hipStream_t stream) {
  const int64_t M = d->rows, N = d->out, K = d->in;
  const bool by_out = w_by_out(d->dw_in_stride, d->dw_out_stride);
  const int64_t dws = by_out ? d->dw_in_stride : d->dw_out_stride;
  int st;
  if (M == 0 || N == 0) {
    if (dx && (st = zero<T>(dx, M, K, d->dx_stride, stream))) return st;
    if (dw && (st = zero<T>(dw, by_out ? K : N, by_out ? N : K, dws, stream))) return st;
    if (db) return d->bias_dtype == SPLAT_F32 ? zero<float>(db, 1, N, N, stream) : zero<T>(db, 1, N, N, stream);
    return SPLAT_OK;
  }
  const Plan p = plan_of(d, true);
  char *at = (char *)ws;
  void *my_pre = at, *dz = at + p.pre;
  float *sums = (float *)(at + p.pre + p.dz), *part = (float *)(at + p.pre + p.dz + p.sums);
  const bool draw = d->drop.p > 0.0, shaped = d->act != SPLAT_ACT_NONE || draw;
  const int parts = parts_of(d);
  const float drop_scale = drop_args(&d->drop).scale, scale = drop_scale / dz_part(d);
  const int64_t rest = parts == 2 ? (int64_t)(p.dz / 2) : 0;
  if (d->act != SPLAT_ACT_NONE && !pre) {
    LayerArgs l = {};
    l.bias = bias;
    l.bias_f32 = d->bias_dtype == SPLAT_F32;
    if ((st = forward<T>(d, x, w, l, my_pre, N, part, stream))) return st;
    pre = my_pre;
  }
  if (shaped || db) {
    SlopeArgs s = {};
    s.dy = dy;
    s.z = pre;
    s.dz = shaped ? dz : nullptr;
    s.dz2 = parts == 2 ? (char *)dz + rest : nullptr;
    s.sums = db ? sums : nullptr;
    s.M = M;
    s.N = N;
    s.ys = d->y_stride;
    s.act = d->act;
    s.draw = draw;
    s.part = dz_part(d);
    s.drop = mask_args(&d->drop);
    const int64_t chunks = slope_chunks(M, N);
    s.chunk = (M + chunks - 1) / chunks;
    const dim3 grid((unsigned)((N + SL_COLS - 1) / SL_COLS), (unsigned)((M + s.chunk - 1) / s.chunk));
    hipLaunchKernelGGL(k_linear_slope<T>, grid, dim3(LN_THREADS), 0, stream, s);
    SPLAT_LAUNCH_CHECK();
    if (db) {
      hipLaunchKernelGGL(k_linear_bias<T>, dim3((unsigned)((N + 31) / 32)), dim3(LN_THREADS), 0, stream,
                         (const float *)sums, (int64_t)grid.y, N, db, (int)(d->bias_dtype == SPLAT_F32), drop_scale);
      SPLAT_LAUNCH_CHECK();
    }
  }
  const Operand z = shaped ? Operand{dz, N, rest} : Operand{dy, d->y_stride, 0};
  if (dx && K > 0) {
    ProductArgs a = {};
    a.I = M;
    a.J = K;
    a.K = N;
    a.parts = parts;
    a.scale = scale;
    a.q = z;
    a.c = dx;
    a.cs = d->dx_stride;
    a.part = part;
    if (w_by_out(d->w_in_stride, d->w_out_stride)) {
      a.p = {w, d->w_in_stride, 0};
      st = launch_product<T>(a, false, false, OUT_STORE, stream);
    } else {
      a.p = {w, d->w_out_stride, 0};
      st = launch_product<T>(a, false, true, OUT_STORE, stream);
    }
    if (st) return st;
  }
  if (dw && K > 0) {
    ProductArgs a = {};
    const Operand xo = {x, d->x_stride, 0};
    a.parts = parts;
    a.scale = scale;
    a.I = by_out ? K : N;
    a.J = by_out ? N : K;
    a.K = M;
    a.q = by_out ? xo : z;
    a.p = by_out ? z : xo;
    a.c = dw;
    a.cs = dws;
    a.part = part;
    return launch_product<T>(a, true, true, OUT_STORE, stream);
  }
  return SPLAT_OK;
}

}  // namespace

// The cheapest of the tiles and splits by what a stage (64 bytes of the summed axis of every
// tile at work) was measured to take, in us: with one workgroup on a CU, and with as many as
// fit. Splits cost the writing and reading of their sums and a launch.
Cut product_cut(int64_t I, int64_t J, int64_t K, int parts, int dtype) {
  struct Rate {
    int fit;
    double one, all, rest;       // rest: of a tile outside its stages
  };
  // fp32 has no tiles of 256: four of 128 take 3.9 us a stage on a CU, one of 256 took 4.4
  static constexpr Rate RATES[3] = {{1, 0.99, 0.99, 8.0}, {2, 0.42, 0.64, 5.0}, {3, 0.30, 0.55, 4.0}},
                        RATES_F32[2] = {{2, 1.10, 1.95, 5.0}, {3, 0.60, 1.50, 4.0}};
  constexpr int CUS = 256;
  const int f32 = dtype == SPLAT_F32;
  const int64_t stages = parts * ((K + (f32 ? 16 : 32) - 1) / (f32 ? 16 : 32));
  Cut best = {2, 1};
  double least = 1e30;
  for (int t = f32; t < 3; t++) {
    const Rate &r = f32 ? RATES_F32[t - 1] : RATES[t];
    const int64_t tiles = ((I + TILES[t].i - 1) / TILES[t].i) * ((J + TILES[t].j - 1) / TILES[t].j);
    for (int s = 1; s <= 1024; s = s < 4 ? s + 1 : s + s / 2) {
      if (s > 1 && stages / s < 8) break;
      const int64_t groups = tiles * s, round = (int64_t)CUS * r.fit, full = groups / round, left = groups - full * round;
      const int64_t per = (left + CUS - 1) / CUS;    // of a CU in the last round
      const double last = per == 0 ? 0.0 : per == 1 ? r.one : r.one + (r.all - r.one) * (double)(per - 1) / (r.fit - 1);
      double us = ((double)full * r.all + last) * (double)((stages + s - 1) / s) + r.rest;
      if (s > 1) us += 6.0 + 8e-6 / 4.5 * (double)s * (double)I * (double)J;
      if (us < least) {
        least = us;
        best = {t, s};
      }
      if (groups > 4 * round) break;
    }
  }
  return best;
}

bool linear_saves(const splat_dense *d) { return d->act != SPLAT_ACT_NONE && !linear_by_rows(d); }

size_t linear_workspace_bytes(const splat_dense *d, bool bwd) {
  if (d->rows == 0 || d->out == 0) return 0;
  if (linear_by_rows(d)) return bwd ? linear_rows_workspace_bytes(d) : 0;
  return plan_of(d, bwd).total;
}

int launch_linear(const splat_dense *d, const void *x, const void *w, const void *bias, const void *res, void *y,
                  void *pre, void *ws, hipStream_t stream) {
  LayerArgs l = {bias, res, pre, d->residual_stride, d->bias_dtype == SPLAT_F32, d->act, d->drop.p > 0.0, drop_args(&d->drop)};
  if (linear_forward_by_rows(d)) {
    if (d->dtype == SPLAT_F32) return launch_linear_rows_f32(d, x, w, l, y, stream);
    if (d->dtype == SPLAT_F16) return launch_linear_rows_f16(d, x, w, l, y, stream);
    return launch_linear_rows_bf16(d, x, w, l, y, stream);
  }
  if (d->dtype == SPLAT_F32) return forward<float>(d, x, w, l, y, d->y_stride, (float *)ws, stream);
  if (d->dtype == SPLAT_F16) return forward<f16_t>(d, x, w, l, y, d->y_stride, (float *)ws, stream);
  return forward<bf16_t>(d, x, w, l, y, d->y_stride, (float *)ws, stream);
}

int launch_linear_bwd(const splat_dense *d, const void *dy, const void *x, const void *w, const void *bias, const void *pre,
                      void *dx, void *dw, void *db, void *ws, hipStream_t stream) {
  if (linear_by_rows(d) && d->rows > 0 && d->out > 0) {
    const LayerArgs l = {bias, nullptr, nullptr, 0, d->bias_dtype == SPLAT_F32, d->act, d->drop.p > 0.0, mask_args(&d->drop)};
    if (d->dtype == SPLAT_F32) return launch_linear_rows_bwd_f32(d, dy, x, w, l, dx, dw, db, ws, stream);
    if (d->dtype == SPLAT_F16) return launch_linear_rows_bwd_f16(d, dy, x, w, l, dx, dw, db, ws, stream);
    return launch_linear_rows_bwd_bf16(d, dy, x, w, l, dx, dw, db, ws, stream);
  }
  if (d->dtype == SPLAT_F32) return backward<float>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
  if (d->dtype == SPLAT_F16) return backward<f16_t>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
  return backward<bf16_t>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
}
