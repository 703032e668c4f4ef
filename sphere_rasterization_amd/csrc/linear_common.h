// What the kernels of the dense layers share: what
// happens to a layer's value on its way to memory.
#pragma once
#include "activation.h"
#include "eight.h"
#include "random.h"

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));
typedef uint32_t word4 __attribute__((ext_vector_type(4)));

constexpr int LN_THREADS = 256;

struct LayerArgs {
  const void *bias, *res;
  void *pre;
  int64_t rs;                    // row stride of the residual; pre is packed
  int bias_f32, act, draw;
  DropArgs drop;
};

// Orders a wave's own LDS accesses: the hardware keeps them in program order.
__device__ __forceinline__ void wave_lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// ---- the end of a value's way ---------------------------------------------------------

template <typename T, int ACT>
__device__ __forceinline__ void activate8(float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = act_of<ACT, sizeof(T) == 4>(v[j]);
}
// d times the slope of the activation at z.
template <typename T, int ACT>
__device__ __forceinline__ void slope8(float (&d)[8], const float (&z)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) d[j] *= act_slope<ACT, sizeof(T) == 4, true>(z[j]);
}
constexpr int ANY_ACT = -1;      // the activation is the launch's
template <typename T>
__device__ __forceinline__ void activate(float (&v)[8], int act) {
  if (act == SPLAT_ACT_RELU) activate8<T, SPLAT_ACT_RELU>(v);
  else if (act == SPLAT_ACT_SILU) activate8<T, SPLAT_ACT_SILU>(v);
  else if (act == SPLAT_ACT_GELU) activate8<T, SPLAT_ACT_GELU>(v);
}
template <typename T>
__device__ __forceinline__ void slope_times(float (&d)[8], const float (&z)[8], int act) {
  if (act == SPLAT_ACT_RELU) slope8<T, SPLAT_ACT_RELU>(d, z);
  else if (act == SPLAT_ACT_SILU) slope8<T, SPLAT_ACT_SILU>(d, z);
  else if (act == SPLAT_ACT_GELU) slope8<T, SPLAT_ACT_GELU>(d, z);
}

template <typename T>
__device__ __forceinline__ void load_bias(const LayerArgs &l, int64_t col, int n, float (&b)[8]) {
  if (!l.bias) {
#pragma unroll
    for (int j = 0; j < 8; j++) b[j] = 0.0f;
  } else if (l.bias_f32) {
    load8<float>((const float *)l.bias + col, n, b);
  } else {
    load8<T>((const T *)l.bias + col, n, b);
  }
}

// The residual's eight values from col of one row, as they lie.
template <typename T>
__device__ __forceinline__ void load_res(const LayerArgs &l, int64_t row, int64_t col, int n, word4 (&r)[sizeof(T) / 2]) {
  constexpr int N = 16 / sizeof(T);
  if (!l.res) return;
  const T *p = (const T *)l.res + row * l.rs + col;
  if (n == 8) {
#pragma unroll
    for (int m = 0; m < (int)sizeof(T) / 2; m++) r[m] = *reinterpret_cast<const typename Loose<T, N>::type *>(p + m * N);
  } else {
    Pack<T, 8> t;
#pragma unroll
    for (int j = 0; j < 8; j++) t.v[j] = j < n ? p[j] : (T)0.0f;
    const Pack<word4, sizeof(T) / 2> q = __builtin_bit_cast(Pack<word4, sizeof(T) / 2>, t);
#pragma unroll
    for (int m = 0; m < (int)sizeof(T) / 2; m++) r[m] = q.v[m];
  }
}

// z = v + b to y (and pre) for n columns from col of one row.
template <typename T>
__device__ __forceinline__ void finish_layer(const LayerArgs &l, const DropKey &key, T *y, int64_t ys, int64_t J,
                                             int64_t row, int64_t col, int n, const float (&b)[8],
                                             const word4 (&res)[sizeof(T) / 2], float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] += b[j];
  if (l.pre) store8<T>((T *)l.pre + row * J + col, n, v);
  activate<T>(v, l.act);
  if (l.draw) drop8<false>(v, row * J + col, l.drop, key);
  if (l.res) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int m = 0; m < (int)sizeof(T) / 2; m++) {
      const Pack<T, N> r = __builtin_bit_cast(Pack<T, N>, res[m]);
#pragma unroll
      for (int j = 0; j < N; j++) v[m * N + j] += (float)r.v[j];
    }
  }
  store8<T>(y + row * ys + col, n, v);
}

// dz as it is multiplied: m act'(z) dy without dropout's factor, by which the sums are multiplied
// in fp32, so that no finite dy leaves the type's range by it. Where the slope is 0 or 1 (none,
// relu) that is dy or 0, exact in the arrays' type. silu's and gelu's slopes pass 1 (1.10 and 1.13):
// of fp16 half of dz is taken, and twice the sums.
__host__ __device__ constexpr bool slope_of_bits(int act) { return act == SPLAT_ACT_NONE || act == SPLAT_ACT_RELU; }
template <typename T>
constexpr float DZ_PART = __is_same(T, f16_t) ? 0.5f : 1.0f;
static inline float dz_part(const splat_dense *d) {
  return d->dtype == SPLAT_F16 && !slope_of_bits(d->act) ? DZ_PART<f16_t> : 1.0f;
}
template <typename T>
__device__ __forceinline__ word4 pack8(const float (&d)[8]) {
  Pack<T, 8> t;
#pragma unroll
  for (int j = 0; j < 8; j++) t.v[j] = (T)d[j];
  return __builtin_bit_cast(word4, t);
}
// dz of silu or gelu in two parts of T, which hold it to twice the type's bits: one would add as much
// error to dx and dW as their own rounding does. fp16 has no room below a small first part: its
// second part is stored times 2^11, the most that cannot overflow, and summed apart, so that
// the two hold dz to 2^-35 from fp16's smallest d_y on (without the factor d_y near 2^-22 was held to
// 3 bits, and below 2^-25 dz was lost). The second part of an infinity is zero.
template <typename T>
constexpr float REST = __is_same(T, f16_t) ? 0x1p-11f : 1.0f;    // what the second part's sums are multiplied by
template <typename T>
__device__ __forceinline__ void split8(const float (&d)[8], word4 &hi, word4 &lo) {
  Pack<T, 8> h, l;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const float v = d[j] * DZ_PART<T>;
    h.v[j] = (T)v;
    const float f = (float)h.v[j];
    l.v[j] = (T)(fabsf(f) < INFINITY ? (v - f) * (1.0f / REST<T>) : 0.0f);
  }
  hi = __builtin_bit_cast(word4, h);
  lo = __builtin_bit_cast(word4, l);
}
