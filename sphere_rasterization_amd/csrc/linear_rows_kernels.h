// Dense layers of at most 64 inputs and outputs, the usual ones of a shading network: many
// rows of few channels, bound by memory. Every array is read and written once: W stays in
// registers, a wave takes 32 rows at a time straight from memory into the layout of the
// matrix cores, and the gradient is one pass too, with z computed anew rather than stored
// (fp32, so that the slope sees no rounding) and dW summed in registers.
//
// Products are formed transposed, D[n][m] = sum of W[k][n] x[m][k]: a lane then holds four
// neighbouring outputs of one row in each of two fragments of 16 x 16, and the rows of W are
// dealt to the fragments so that the eight are neighbours. That is what one 16-byte access
// of 16-bit values and one draw of the generator take, and the layout in which dz is the
// operand of dx = dz W^T. Only dW, summed over rows, turns x and dz around, through LDS.
//
// Measured on one MI355X. 2M rows of 32 to 64 fp16 with silu: 80 us, 5.0 TB/s. 1M rows of 32
// to 32 fp32 with silu and residual: forward 78 us, 5.2 TB/s, backward 97 and a join of 5, 4.2.
// 5.5M rows of 24 to 32 bf16 with gelu and dropout: forward 183 to 200 us, backward 273 to
// 302, both bound by gelu's and the generator's instructions rather than by memory (103 and 147).
#pragma once
#include "linear_rows.h"

namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));

struct RowsArgs {
  const void *x, *w, *bias, *dy;
  void *y, *dx;
  int64_t M, xs, ys, dxs, wi, wo;    // rows; strides of x, y or dy, dx; of W along in and out
  int K, N;                          // N: of a slice of at most 64 outputs, one for each blockIdx.y (forward)
  int full;                          // outputs of the layer
  int want_x, want_w;                // want_w: dW or db
  float *part;                       // [workgroups][K + 1][N]: sums of dW, then of db
  float scale;                       // of the sums of dx
  LayerArgs layer;
};

// 16 x 16 products: operand chunks of 16 bytes a lane, fp32 sums.
template <typename T>
__device__ __forceinline__ float4v mul16(const word4 &a, const word4 &b, float4v c);
template <>
__device__ __forceinline__ float4v mul16<f16_t>(const word4 &a, const word4 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ float4v mul16<bf16_t>(const word4 &a, const word4 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8, a), __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ float4v mul16<float>(const word4 &a, const word4 &b, float4v c) {
  const float4v x = __builtin_bit_cast(float4v, a), y = __builtin_bit_cast(float4v, b);
#pragma unroll
  for (int j = 0; j < 4; j++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
  return c;
}

// The same summed over 16 rows of 16-bit values, four a lane.
template <typename T>
__device__ __forceinline__ float4v mul16_short(const uint2 &a, const uint2 &b, float4v c);
template <>
__device__ __forceinline__ float4v mul16_short<f16_t>(const uint2 &a, const uint2 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(half4, a), __builtin_bit_cast(half4, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ float4v mul16_short<bf16_t>(const uint2 &a, const uint2 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4v, a), __builtin_bit_cast(short4v, b), c, 0, 0, 0);
}

// An array's rows as the kernels read them: 16 bytes at a time, at any alignment, and with rows
// that do not end with a chunk (not EASY) past their ends, what lies there masked out. Only the
// array's own end is not passed: the last chunk is read up to it and shifted.
template <typename T>
struct RowEnd {
  const T *end;
  int len;
  // n: of the row's values from p on that are read; all: that are there
  __device__ RowEnd(const void *p, int64_t rows, int64_t stride, int n, int all)
      : end((const T *)p + (rows - 1) * stride + all), len(n) {}
};

// Values at .. of the row, zeros beyond it.
template <typename T, bool EASY>
__device__ __forceinline__ word4 load_chunk(const T *row, int at, const RowEnd<T> &r, bool ok) {
  constexpr int E = 16 / sizeof(T), W = 4 / sizeof(T);
  typedef const typename Loose<T, E>::type *ptr;
  word4 v = {0, 0, 0, 0};
  if constexpr (EASY) {
    if (ok && at < r.len) v = *reinterpret_cast<ptr>(row + at);
    return v;
  }
  if (ok && at < r.len) {
    const T *p = row + at;
    const int over = p + E > r.end ? (int)(p + E - r.end) : 0;
    v = *reinterpret_cast<ptr>(p - over);
    if (over) {                                   // towards the first element
      if (over & (2 * W)) v = word4{v[2], v[3], 0, 0};
      if (over & W) v = word4{v[1], v[2], v[3], 0};
      if (W == 2 && (over & 1))
        v = word4{__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
                  __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16};
    }
    int left = r.len - at;                        // elements of the row from here on
    asm volatile("" : "+v"(left));                // the masks are made anew, not kept in registers
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if (left <= k * W) v[k] = 0;
      else if (W == 2 && left == k * W + 1) v[k] &= 0xFFFFu;
    }
  }
  return v;
}

template <typename T, int KP, int NP, bool EASY>
struct Rows {
  static constexpr int E = 16 / sizeof(T);            // values per chunk
  static constexpr int KC = KP * 32 / (4 * E);        // chunks of a row of x per lane
  static constexpr int DC = 8 / E;                    // chunks of eight values
  static constexpr int KW = KP * 32 + E, NW = NP * 32 + E;    // pitches of W in LDS, by outputs and by inputs
  static constexpr int BY_OUT = NP * 32 * KW, BY_IN = KP * 32 * NW;
  static constexpr int W_BYTES = (BY_OUT + BY_IN) * sizeof(T);
  // Row pitches of the tiles that are read turned around. 16-bit: a transposing read takes
  // eight rows of 32 bytes at once, which a pitch of an odd multiple of 32 bytes spreads over
  // all banks; fp32: four rows of 64 bytes, and a pitch of 64 more than a multiple of 128.
  static constexpr int XP = KP * 32 * sizeof(T) + 16 * sizeof(T), ZP = NP * 32 * sizeof(T) + 16 * sizeof(T);
  static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;   // of dz
  static constexpr int WAVE_BYTES = 16 * (XP + PARTS * ZP);
  // Rows in flight ahead of those at work, in sixteens: a wave waits for its stores too before
  // it sees a load that it issued after them, and with one load ahead it mostly waited.
  static constexpr int SIZE = KP * NP * (int)sizeof(T) / 2;
  static constexpr int AHEAD = EASY && SIZE <= 2 && sizeof(T) == 2 ? 2 : 1;
  static constexpr int SUM_BYTES = (KP * 32 * NP * 32 + NP * 32) * 4;

  // W in LDS by outputs [out][in] and, where the pointer is given, by inputs; zeros beyond it.
  static __device__ __forceinline__ void stage_w(const RowsArgs &a, T *by_out, T *by_in) {
#pragma unroll 4
    for (int t = threadIdx.x; t < KP * 32 * NP * 32; t += LN_THREADS) {
      // neighbouring threads read neighbouring values
      const int k = a.wo == 1 ? t / (NP * 32) : t % (KP * 32), n = a.wo == 1 ? t % (NP * 32) : t / (KP * 32);
      const T v = k < a.K && n < a.N ? ((const T *)a.w)[k * a.wi + n * a.wo] : (T)0.0f;
      by_out[n * KW + k] = v;
      if (by_in) by_in[k * NW + n] = v;
    }
  }

  // Operands of z: row i of fragment t of 32 outputs p stands for output 32 p + 8 (i / 4) + 4 t + i % 4.
  static __device__ __forceinline__ void fragments(const T *by_out, word4 (&f)[NP][2][KC], int p) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int c = 0; c < KC; c++)
        f[p][t][c] = *reinterpret_cast<const word4 *>(by_out + (32 * p + 8 * (i >> 2) + 4 * t + (i & 3)) * KW + (c * 4 + g) * E);
  }
  static __device__ __forceinline__ void fragments(const T *by_out, word4 (&f)[NP][2][KC]) {
#pragma unroll
    for (int p = 0; p < NP; p++) fragments(by_out, f, p);
  }

  // Operands of dx, the same with inputs for outputs: eight neighbouring outputs 32 p + 8 g of
  // input row i in DC chunks.
  static __device__ __forceinline__ void fragments_t(const T *by_in, word4 (&f)[KP][2][NP][DC], int q) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int p = 0; p < NP; p++)
#pragma unroll
        for (int c = 0; c < DC; c++)
          f[q][t][p][c] =
              *reinterpret_cast<const word4 *>(by_in + (32 * q + 8 * (i >> 2) + 4 * t + (i & 3)) * NW + 32 * p + 8 * g + c * E);
  }
  static __device__ __forceinline__ void fragments_t(const T *by_in, word4 (&f)[KP][2][NP][DC]) {
#pragma unroll
    for (int q = 0; q < KP; q++) fragments_t(by_in, f, q);
  }

  // A lane's row of x: its chunks, from `row` = its first value on.
  static __device__ __forceinline__ void load_x(const T *row, const RowEnd<T> &e, bool ok, word4 (&x)[KC]) {
    const int g = threadIdx.x >> 4 & 3;
#pragma unroll
    for (int c = 0; c < KC; c++) x[c] = load_chunk<T, EASY>(row, (c * 4 + g) * E, e, ok);
  }

  // Eight values of a lane's row for each 32 outputs.
  static __device__ __forceinline__ void load_out(const T *row, const RowEnd<T> &e, bool ok, word4 (&d)[NP][DC]) {
    const int g = threadIdx.x >> 4 & 3;
#pragma unroll
    for (int q = 0; q < NP; q++)
#pragma unroll
      for (int c = 0; c < DC; c++) d[q][c] = load_chunk<T, EASY>(row, 32 * q + 8 * g + c * E, e, ok);
  }

  static __device__ __forceinline__ void widen(const word4 (&r)[DC], float (&o)[8]) {
#pragma unroll
    for (int c = 0; c < DC; c++) {
      const Pack<T, E> v = __builtin_bit_cast(Pack<T, E>, r[c]);
#pragma unroll
      for (int e = 0; e < E; e++) o[c * E + e] = (float)v.v[e];
    }
  }

  // z of 16 rows: eight outputs of a lane's row for each 32.
  static __device__ __forceinline__ void product(const word4 (&f)[NP][2][KC], const word4 (&x)[KC], int p, float (&z)[8]) {
    float4v lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < KC; c++) {
      lo = mul16<T>(f[p][0][c], x[c], lo);
      hi = mul16<T>(f[p][1][c], x[c], hi);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      z[j] = lo[j];
      z[4 + j] = hi[j];
    }
  }

  // Sixteen rows of n values from a tile in LDS to memory, neighbouring lanes on neighbouring
  // 16 bytes: rows past 64 bytes straight from the products' layout, four lanes to a row, took
  // 104 us in place of 84 for 2M rows of 64 fp16 outputs. n a multiple of a chunk.
  template <int SIDE>
  static __device__ __forceinline__ void store_rows(const char *tile, int pitch, T *p, int64_t stride, int n, int64_t rows) {
    const int per = n / E;
#pragma unroll
    for (int u = 0; u < SIDE * 16 / E / 64; u++) {
      const int q = (threadIdx.x & 63) + 64 * u, r = q / per, c = q - r * per;
      if (r < 16 && r < rows)
        *reinterpret_cast<typename Loose<T, E>::type *>(p + r * stride + c * E) =
            *reinterpret_cast<const word4 *>(tile + r * pitch + c * 16);
    }
  }

  // Four rows 4 g .. 4 g + 3 of column col + i of a tile of 16-bit values.
  static __device__ __forceinline__ uint2 turned(const char *tile, int pitch, int col) {
    typedef __attribute__((address_space(3))) short4v *lds4;
    const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
    const char *at = tile + (4 * g + (j >> 2)) * pitch + (col + (j & 3) * 4) * 2;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(short4v *)const_cast<char *>(at)));
  }
};

// What a lane's place among the outputs needs: how many of its eight exist, and their bias.
template <typename T, int NP>
__device__ __forceinline__ void lane_outputs(const RowsArgs &a, int (&n)[NP], float (&b)[NP][8]) {
  const int g = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int p = 0; p < NP; p++) {
    n[p] = a.N - (32 * p + 8 * g);
    n[p] = n[p] < 0 ? 0 : n[p] > 8 ? 8 : n[p];
    load_bias<T>(a.layer, 32 * p + 8 * g, n[p], b[p]);
  }
}

// Four waves a SIMD for 16-bit types: their 128 registers do not suffice for 33 to 64 outputs with
// dropout (52 to 108 bytes a lane spill, up to 240 at widths that are not multiples of 8), nor, of up to
// 32 inputs, without it and with none, relu or gelu (12 to 20).
template <typename T, int KP, int NP, int ACT, bool DRAW, bool EASY>
__global__ __launch_bounds__(LN_THREADS, sizeof(T) == 2 ? 4 : KP * NP < 4 ? 3 : 2) void k_rows(RowsArgs a) {
  typedef Rows<T, KP, NP, EASY> R;
  // rows of more than 32 outputs leave through LDS
  constexpr bool BOUNCE = EASY && NP == 2;
  constexpr int OP = NP * 32 * sizeof(T) + 16;
  __shared__ __attribute__((aligned(16))) T lw[R::BY_OUT];
  __shared__ __attribute__((aligned(16))) char lo[BOUNCE ? LN_THREADS / WAVE * 16 * OP : 16];
  char *const ot = lo + (BOUNCE ? (threadIdx.x >> 6) * 16 * OP : 0);
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t step = (int64_t)gridDim.x * (LN_THREADS / WAVE) * 16;
  int64_t base = ((int64_t)blockIdx.x * (LN_THREADS / WAVE) + (threadIdx.x >> 6)) * 16;
  // this slice of the outputs
  const int c0 = blockIdx.y * 64;
  a.N = a.full - c0 < 64 ? a.full - c0 : 64;
  a.w = (const T *)a.w + c0 * a.wo;
  a.y = (T *)a.y + c0;
  if (a.layer.res) a.layer.res = (const T *)a.layer.res + c0;
  if (a.layer.pre) a.layer.pre = (T *)a.layer.pre + c0;
  if (a.layer.bias) a.layer.bias = (const char *)a.layer.bias + (int64_t)c0 * (a.layer.bias_f32 ? 4 : sizeof(T));
  const T *px = (const T *)a.x + (base + i) * a.xs, *pr = (const T *)a.layer.res + (base + i) * a.layer.rs;
  T *py = (T *)a.y + (base + (BOUNCE ? 0 : i)) * a.ys;
  word4 nx[R::AHEAD][R::KC], nr[R::AHEAD][NP][R::DC];
  int64_t ahead = base + i;                      // the row that is loaded next
  const RowEnd<T> ex(a.x, a.M, a.xs, a.K, a.K), er(a.layer.res, a.M, a.layer.rs, a.N, a.full - c0);
  auto load = [&](int d) {
    R::load_x(px, ex, ahead < a.M, nx[d]);
    if (a.layer.res) R::load_out(pr, er, ahead < a.M, nr[d]);
    px += step * a.xs;
    pr += step * a.layer.rs;
    ahead += step;
  };
#pragma unroll
  for (int d = 0; d < R::AHEAD; d++) load(d);
  R::stage_w(a, lw, nullptr);
  __syncthreads();
  word4 f[NP][2][R::KC];
  R::fragments(lw, f);
  float b[NP][8];
  int n[NP];
  lane_outputs<T, NP>(a, n, b);
  DropKey key = {};
  if (DRAW) key = drop_key(a.layer.drop);
  while (base < a.M) {
#pragma unroll
    for (int d = 0; d < R::AHEAD; d++) {
      const bool in = base + i < a.M;
      word4 x[R::KC], r[NP][R::DC];
#pragma unroll
      for (int c = 0; c < R::KC; c++) x[c] = nx[d][c];
#pragma unroll
      for (int p = 0; p < NP; p++)
#pragma unroll
        for (int c = 0; c < R::DC; c++) r[p][c] = nr[d][p][c];
      load(d);
#pragma unroll
      for (int p = 0; p < NP; p++) {
        float v[8];
        R::product(f, x, p, v);
        if (in && n[p] > 0) {
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] += b[p][j];
          if (a.layer.pre) store8<T>((T *)a.layer.pre + (base + i) * a.full + 32 * p + 8 * g, EASY ? 8 : n[p], v);
          if constexpr (ACT == ANY_ACT) activate<T>(v, a.layer.act);
          else activate8<T, ACT>(v);
          if (DRAW) drop8<EASY>(v, (base + i) * a.full + c0 + 32 * p + 8 * g, a.layer.drop, key);
          if (a.layer.res) {
            float q[8];
            R::widen(r[p], q);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += q[j];
          }
          if constexpr (BOUNCE) store8<T>(reinterpret_cast<T *>(ot + i * OP) + 32 * p + 8 * g, 8, v);
          else store8<T>(py + 32 * p + 8 * g, EASY ? 8 : n[p], v);
        }
      }
      if constexpr (BOUNCE) {
        wave_lds_order();
        R::template store_rows<NP * 32>(ot, OP, py, a.ys, a.N, a.M - base);
        wave_lds_order();
      }
      py += step * a.ys;
      base += step;
    }
  }
}

// (16-bit layers of 33 to 64 inputs and outputs at widths that are not multiples of 8 spill up to 212
// bytes a lane with dropout.)
template <typename T, int KP, int NP, int ACT, bool DRAW, bool EASY>
__global__ __launch_bounds__(LN_THREADS, KP * NP > 1 ? 2 : 3) void k_rows_bwd(RowsArgs a) {
  typedef Rows<T, KP, NP, EASY> R;
  constexpr int WAVES = LN_THREADS / WAVE;
  // fp32 and 64 x 64: W, 128 registers a lane, stays in LDS, so that two waves fit a SIMD
  constexpr bool KEEP = sizeof(T) == 4 && KP * NP == 4;
  constexpr int A = R::W_BYTES > R::SUM_BYTES ? R::W_BYTES : R::SUM_BYTES;
  constexpr int LDS = KEEP ? R::W_BYTES + WAVES * R::WAVE_BYTES : WAVES * R::WAVE_BYTES > A ? WAVES * R::WAVE_BYTES : A;
  __shared__ __attribute__((aligned(16))) char lds[LDS];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, w = threadIdx.x >> 6;
  const int64_t step = (int64_t)gridDim.x * WAVES * 16;
  int64_t base = ((int64_t)blockIdx.x * WAVES + w) * 16;
  const int act = ACT == ANY_ACT ? a.layer.act : ACT;
  const bool slope = act != SPLAT_ACT_NONE, shaped = slope || DRAW;
  const bool two = sizeof(T) == 2 && !slope_of_bits(act);    // parts of dz
  constexpr bool APART = REST<T> != 1.0f && (ACT == ANY_ACT || !slope_of_bits(ACT));
  // the sums of second parts in registers of their own, where those suffice: 1M x 32 to 64 fp16 79 us, 84
  // with each sum added to the first parts' at once
  constexpr bool OWN = APART && EASY && KP * NP < 4;
  const T *px = (const T *)a.x + (base + i) * a.xs, *pd = (const T *)a.dy + (base + i) * a.ys;
  T *po = (T *)a.dx + (base + i) * a.dxs;
  word4 nx[R::AHEAD][R::KC], nd[R::AHEAD][NP][R::DC];
  int64_t ahead = base + i;
  const RowEnd<T> ex(a.x, a.M, a.xs, a.K, a.K), ed(a.dy, a.M, a.ys, a.N, a.N);
  auto load = [&](int d) {
    R::load_x(px, ex, ahead < a.M, nx[d]);
    R::load_out(pd, ed, ahead < a.M, nd[d]);
    px += step * a.xs;
    pd += step * a.ys;
    ahead += step;
  };
#pragma unroll
  for (int d = 0; d < R::AHEAD; d++) load(d);
  T *by_out = reinterpret_cast<T *>(lds), *by_in = by_out + R::BY_OUT;
  R::stage_w(a, by_out, by_in);
  __syncthreads();
  word4 f[NP][2][R::KC], ft[KP][2][NP][R::DC];
  if constexpr (!KEEP) {
    R::fragments(by_out, f);
    R::fragments_t(by_in, ft);
    __syncthreads();
  }
  char *xt = lds + (KEEP ? R::W_BYTES : 0) + w * R::WAVE_BYTES, *zt = xt + 16 * R::XP, *zt2 = zt + 16 * R::ZP;
  float b[NP][8];
  int n[NP];
  lane_outputs<T, NP>(a, n, b);
  DropKey key = {};
  if (DRAW) key = drop_key(a.layer.drop);
  float4v dw[2 * KP][2 * NP], dw2[OWN ? 2 * KP : 1][OWN ? 2 * NP : 1];
  float db[NP][8];
#pragma unroll
  for (int k = 0; k < 2 * KP; k++)
#pragma unroll
    for (int q = 0; q < 2 * NP; q++) {
      dw[k][q] = float4v{0, 0, 0, 0};
      if constexpr (OWN) dw2[k][q] = float4v{0, 0, 0, 0};
    }
#pragma unroll
  for (int p = 0; p < NP; p++)
#pragma unroll
    for (int j = 0; j < 8; j++) db[p][j] = 0.0f;
  while (base < a.M) {
#pragma unroll
    for (int d = 0; d < R::AHEAD; d++) {
      const bool in = base + i < a.M;
      word4 x[R::KC], dy[NP][R::DC];
#pragma unroll
      for (int c = 0; c < R::KC; c++) {
        x[c] = nx[d][c];
        *reinterpret_cast<word4 *>(xt + i * R::XP + c * 64 + g * 16) = x[c];
      }
#pragma unroll
      for (int p = 0; p < NP; p++)
#pragma unroll
        for (int c = 0; c < R::DC; c++) dy[p][c] = nd[d][p][c];
      load(d);
      word4 dz[NP][R::DC], dz2[NP];
#pragma unroll
      for (int p = 0; p < NP; p++) {
        float v[8];
        R::widen(dy[p], v);
        if (slope) {
          float z[8];
          if constexpr (KEEP) R::fragments(by_out, f, p);
          R::product(f, x, p, z);
#pragma unroll
          for (int j = 0; j < 8; j++) z[j] += b[p][j];
          if constexpr (ACT == ANY_ACT) slope_times<T>(v, z, act);
          else slope8<T, ACT>(v, z);
        }
        if (DRAW) drop8<EASY>(v, (base + i) * a.N + 32 * p + 8 * g, a.layer.drop, key);
        if (shaped) {
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = in ? v[j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) db[p][j] += v[j];
        if constexpr (sizeof(T) == 2) {
          if (two) {
            split8<T>(v, dz[p][0], dz2[p]);
            *reinterpret_cast<word4 *>(zt2 + i * R::ZP + p * 64 + g * 16) = dz2[p];
          } else if (shaped) {
            dz[p][0] = pack8<T>(v);
          } else {
            dz[p][0] = dy[p][0];
          }
          *reinterpret_cast<word4 *>(zt + i * R::ZP + p * 64 + g * 16) = dz[p][0];
        } else {
#pragma unroll
          for (int c = 0; c < R::DC; c++) {
            dz[p][c] = __builtin_bit_cast(word4, make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
            *reinterpret_cast<word4 *>(zt + i * R::ZP + p * 128 + g * 32 + c * 16) = dz[p][c];
          }
        }
      }
      if (a.want_x) {
#pragma unroll
        for (int q = 0; q < KP; q++) {
          float4v lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
          if constexpr (KEEP) R::fragments_t(by_in, ft, q);
          if constexpr (sizeof(T) == 2) {
            if (two) {
#pragma unroll
              for (int p = 0; p < NP; p++) {
                lo = mul16<T>(ft[q][0][p][0], dz2[p], lo);
                hi = mul16<T>(ft[q][1][p][0], dz2[p], hi);
              }
              if constexpr (APART) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                  lo[j] *= REST<T>;
                  hi[j] *= REST<T>;
                }
              }
            }
          }
#pragma unroll
          for (int p = 0; p < NP; p++) {
#pragma unroll
            for (int c = 0; c < R::DC; c++) {
              lo = mul16<T>(ft[q][0][p][c], dz[p][c], lo);
              hi = mul16<T>(ft[q][1][p][c], dz[p][c], hi);
            }
          }
          const int col = 32 * q + 8 * g, left = a.K - col;
          if (in && left > 0) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
              v[j] = lo[j] * a.scale;
              v[4 + j] = hi[j] * a.scale;
            }
            store8<T>(po + col, EASY && sizeof(T) == 2 || left > 8 ? 8 : left, v);
          }
        }
        po += step * a.dxs;
      }
      if (a.want_w) {
        wave_lds_order();
        if constexpr (sizeof(T) == 2) {
          uint2 xf[2 * KP];
#pragma unroll
          for (int k = 0; k < 2 * KP; k++) xf[k] = R::turned(xt, R::XP, 16 * k);
#pragma unroll
          for (int q = 0; q < 2 * NP; q++) {
            const uint2 zf = R::turned(zt, R::ZP, 16 * q);
#pragma unroll
            for (int k = 0; k < 2 * KP; k++) dw[k][q] = mul16_short<T>(xf[k], zf, dw[k][q]);
          }
          if (two) {
#pragma unroll
            for (int q = 0; q < 2 * NP; q++) {
              const uint2 zf = R::turned(zt2, R::ZP, 16 * q);
#pragma unroll
              for (int k = 0; k < 2 * KP; k++) {
                if constexpr (OWN) {
                  dw2[k][q] = mul16_short<T>(xf[k], zf, dw2[k][q]);
                } else if constexpr (APART) {
                  const float4v sum = mul16_short<T>(xf[k], zf, float4v{0, 0, 0, 0});
#pragma unroll
                  for (int e = 0; e < 4; e++) dw[k][q][e] = __builtin_fmaf(sum[e], REST<T>, dw[k][q][e]);
                } else {
                  dw[k][q] = mul16_short<T>(xf[k], zf, dw[k][q]);
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < 4; s++) {
            const float *xr = reinterpret_cast<const float *>(xt + (4 * s + g) * R::XP);
            const float *zr = reinterpret_cast<const float *>(zt + (4 * s + g) * R::ZP);
            float xv[2 * KP], zv[2 * NP];
#pragma unroll
            for (int k = 0; k < 2 * KP; k++) xv[k] = xr[16 * k + i];
#pragma unroll
            for (int q = 0; q < 2 * NP; q++) zv[q] = zr[16 * q + i];
#pragma unroll
            for (int k = 0; k < 2 * KP; k++)
#pragma unroll
              for (int q = 0; q < 2 * NP; q++) dw[k][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[k], zv[q], dw[k][q], 0, 0, 0);
          }
        }
        wave_lds_order();
      }
      base += step;
    }
  }
  if (!a.want_w) return;
  if constexpr (OWN) {
#pragma unroll
    for (int k = 0; k < 2 * KP; k++)
#pragma unroll
      for (int q = 0; q < 2 * NP; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) dw[k][q][e] = __builtin_fmaf(dw2[k][q][e], REST<T>, dw[k][q][e]);
  }
  // the waves' sums in order, wave after wave
#pragma unroll
  for (int p = 0; p < NP; p++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) db[p][j] += __shfl_xor(db[p][j], s, WAVE);
    }
  float *sum = reinterpret_cast<float *>(lds), *sum_b = sum + KP * 32 * NP * 32;
  for (int v = 0; v < WAVES; v++) {
    __syncthreads();
    if (w != v) continue;
#pragma unroll
    for (int k = 0; k < 2 * KP; k++)
#pragma unroll
      for (int q = 0; q < 2 * NP; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float *s = sum + (16 * k + 4 * g + e) * (NP * 32) + 16 * q + i;
          *s = v == 0 ? dw[k][q][e] : *s + dw[k][q][e];
        }
    if (i == 0) {
#pragma unroll
      for (int p = 0; p < NP; p++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
          float *s = sum_b + 32 * p + 8 * g + j;
          *s = v == 0 ? db[p][j] : *s + db[p][j];
        }
    }
  }
  __syncthreads();
  float *out = a.part + (int64_t)blockIdx.x * (a.K + 1) * a.N;
  for (int t = threadIdx.x; t < (a.K + 1) * a.N; t += LN_THREADS) {
    const int k = t / a.N, c = t - k * a.N;
    out[t] = k < a.K ? sum[k * (NP * 32) + c] : sum_b[c];
  }
}

// The workgroups' sums in order: 32 values by 32 slices of the workgroups per workgroup. scale and
// db_scale: of the sums of dW and of db.
template <typename T>
__global__ __launch_bounds__(1024) void k_rows_join(const float *part, int groups, int K, int N, T *dw, int64_t di, int64_t dn,
                                                    void *db, int f32, float scale, float db_scale) {
  __shared__ float s[32][33];
  const int e = threadIdx.x & 31, l = threadIdx.x >> 5, size = (K + 1) * N, at = blockIdx.x * 32 + e;
  float v = 0.0f;
  if (at < size) {
#pragma unroll 8
    for (int k = l; k < groups; k += 32) v += part[(int64_t)k * size + at];
  }
  s[l][e] = v;
  __syncthreads();
  if (threadIdx.x >= 32 || at >= size) return;
  v = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; k++) v += s[k][e];
  const int k = at / N, n = at - k * N;
  if (k < K) {
    if (dw) dw[k * di + n * dn] = (T)(v * scale);
  } else if (db) {
    v *= db_scale;
    if (f32) ((float *)db)[n] = v;
    else ((T *)db)[n] = (T)v;
  }
}

// As many workgroups as the chip holds at once: a wave's share of the rows is then the same
// for all, and W is staged once for each. (2M rows of 64 to 64 bf16: 100 us, 109 with twice as
// many.) Asked once for each kernel.
template <typename K>
int resident(K kernel) {
  int per = 0, cus = 0, dev = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, LN_THREADS, 0) != hipSuccess || per < 1) per = 1;
  if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus < 1)
    cus = 256;
  return per * cus;
}

template <typename T, int KP, int NP, int ACT, bool DRAW, bool EASY>
int launch_one(const RowsArgs &a, bool bwd, int most, hipStream_t s) {
  const int64_t need = (a.M + 63) / 64;              // four waves of 16 rows
  if (bwd) {
    static const int fit = resident(k_rows_bwd<T, KP, NP, ACT, DRAW, EASY>);
    int groups = fit < most ? fit : most;
    if (need < groups) groups = (int)need;
    hipLaunchKernelGGL((k_rows_bwd<T, KP, NP, ACT, DRAW, EASY>), dim3((unsigned)groups), dim3(LN_THREADS), 0, s, a);
    return groups;
  }
  static const int fit = resident(k_rows<T, KP, NP, ACT, DRAW, EASY>);
  const int slices = (a.full + 63) / 64, share = (fit + slices - 1) / slices, groups = need < share ? (int)need : share;
  hipLaunchKernelGGL((k_rows<T, KP, NP, ACT, DRAW, EASY>), dim3((unsigned)groups, (unsigned)slices), dim3(LN_THREADS), 0, s, a);
  return groups;
}
template <typename T, int KP, int NP, bool DRAW>
int by_act(const RowsArgs &a, bool bwd, int most, hipStream_t s) {
  // rows of whole chunks and of whole draws; for others one kernel serves all activations
  const bool easy = a.K % (16 / (int)sizeof(T)) == 0 && a.full % 8 == 0;
  if (!easy) return launch_one<T, KP, NP, ANY_ACT, DRAW, false>(a, bwd, most, s);
  switch (a.layer.act) {
    case SPLAT_ACT_RELU: return launch_one<T, KP, NP, SPLAT_ACT_RELU, DRAW, true>(a, bwd, most, s);
    case SPLAT_ACT_SILU: return launch_one<T, KP, NP, SPLAT_ACT_SILU, DRAW, true>(a, bwd, most, s);
    case SPLAT_ACT_GELU: return launch_one<T, KP, NP, SPLAT_ACT_GELU, DRAW, true>(a, bwd, most, s);
    default: return launch_one<T, KP, NP, SPLAT_ACT_NONE, DRAW, true>(a, bwd, most, s);
  }
}
template <typename T, int KP, int NP>
int by_draw(const RowsArgs &a, bool bwd, int most, hipStream_t s) {
  return a.layer.draw ? by_act<T, KP, NP, true>(a, bwd, most, s) : by_act<T, KP, NP, false>(a, bwd, most, s);
}
// Workgroups launched.
template <typename T>
int by_size(const RowsArgs &a, bool bwd, int most, hipStream_t s) {
  if (a.K <= 32 && a.N <= 32) return by_draw<T, 1, 1>(a, bwd, most, s);
  if (a.K <= 32) return by_draw<T, 1, 2>(a, bwd, most, s);
  if (a.N <= 32) return by_draw<T, 2, 1>(a, bwd, most, s);
  return by_draw<T, 2, 2>(a, bwd, most, s);
}

RowsArgs rows_args(const splat_dense *d, const void *x, const void *w) {
  RowsArgs a = {};
  a.x = x;
  a.w = w;
  a.M = d->rows;
  a.K = d->in;
  a.N = a.full = d->out;
  a.xs = d->x_stride;
  a.ys = d->y_stride;
  a.dxs = d->dx_stride;
  a.wi = d->w_in_stride;
  a.wo = d->w_out_stride;
  return a;
}

template <typename T>
int run_rows(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream) {
  RowsArgs a = rows_args(d, x, w);
  a.y = y;
  a.layer = l;
  by_size<T>(a, false, 0, stream);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T>
int run_rows_bwd(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx, void *dw,
                 void *db, void *ws, hipStream_t stream) {
  RowsArgs a = rows_args(d, x, w);
  a.dy = dy;
  a.dx = dx;
  a.layer = l;
  a.want_x = dx != nullptr;
  a.want_w = dw || db;
  a.part = (float *)ws;
  const float drop_scale = drop_args(&d->drop).scale;
  a.scale = drop_scale / dz_part(d);
  const int groups = by_size<T>(a, true, linear_rows_groups(d), stream);
  SPLAT_LAUNCH_CHECK();
  if (!a.want_w) return SPLAT_OK;
  hipLaunchKernelGGL(k_rows_join<T>, dim3((unsigned)(((a.K + 1) * a.N + 31) / 32)), dim3(1024), 0, stream, a.part, groups, a.K,
                     a.N, (T *)dw, d->dw_in_stride, d->dw_out_stride, db, (int)(d->bias_dtype == SPLAT_F32), a.scale, drop_scale);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

}  // namespace
