// What the kernels of the dense layers share: accesses of eight neighbouring values, and what
// happens to a layer's value on its way to memory.
#pragma once
#include "activation.h"
#include "learn_common.h"
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

// ---- the end of a value's way ---------------------------------------------------------

// Elements col .. col + 7 of row `row`; `n` of them exist.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float (&o)[8]) {
  constexpr int N = 16 / sizeof(T);
  if (n == 8) {
#pragma unroll
    for (int m = 0; m < 8; m += N) {
      float t[N];
      const Raw<T, N> r = *reinterpret_cast<const typename Loose<T, N>::type *>(p + m);
      to_f32<T, N>(r, t);
#pragma unroll
      for (int j = 0; j < N; j++) o[m + j] = t[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) o[j] = j < n ? (float)p[j] : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float (&o)[8]) {
  constexpr int N = 16 / sizeof(T);
  if (n == 8) {
#pragma unroll
    for (int m = 0; m < 8; m += N) {
      Pack<T, N> t;
#pragma unroll
      for (int j = 0; j < N; j++) t.v[j] = (T)o[m + j];
      *reinterpret_cast<typename Loose<T, N>::type *>(p + m) = __builtin_bit_cast(Raw<T, N>, t);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (j < n) p[j] = (T)o[j];
  }
}

// Which of elements at .. at + 7 are kept, `at` any element.
__device__ __forceinline__ uint32_t keeps_from(int64_t at, const DropArgs &d, const DropKey &k) {
  const uint32_t sh = (uint32_t)at & 7;
  uint32_t bits = drop_keeps((uint64_t)at >> 3, d, k);
  if (sh) bits = (bits | drop_keeps(((uint64_t)at >> 3) + 1, d, k) << 8) >> sh;
  return bits;
}

template <typename T>
__device__ __forceinline__ void activate(float (&v)[8], int act) {
  constexpr bool EXACT = sizeof(T) == 4;
  if (act == SPLAT_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = act_of<SPLAT_ACT_RELU, EXACT>(v[j]);
  } else if (act == SPLAT_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = act_of<SPLAT_ACT_SILU, EXACT>(v[j]);
  } else if (act == SPLAT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = act_of<SPLAT_ACT_GELU, EXACT>(v[j]);
  }
}

// d times the slope of the activation at z.
template <typename T>
__device__ __forceinline__ void slope_times(float (&d)[8], const float (&z)[8], int act) {
  constexpr bool EXACT = sizeof(T) == 4;
  if (act == SPLAT_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < 8; j++) d[j] *= act_slope<SPLAT_ACT_RELU, EXACT>(z[j]);
  } else if (act == SPLAT_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 8; j++) d[j] *= act_slope<SPLAT_ACT_SILU, EXACT>(z[j]);
  } else if (act == SPLAT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 8; j++) d[j] *= act_slope<SPLAT_ACT_GELU, EXACT>(z[j]);
  }
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

// z = v + b to y (and pre) for n columns from col of one row.
template <typename T>
__device__ __forceinline__ void finish_layer(const LayerArgs &l, const DropKey &key, T *y, int64_t ys, int64_t J,
                                             int64_t row, int64_t col, int n, float (&v)[8]) {
  float b[8];
  load_bias<T>(l, col, n, b);
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] += b[j];
  if (l.pre) store8<T>((T *)l.pre + row * J + col, n, v);
  activate<T>(v, l.act);
  if (l.draw) {
    const uint32_t keep = keeps_from(row * J + col, l.drop, key);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = keep >> j & 1 ? v[j] * l.drop.scale : 0.0f;
  }
  if (l.res) {
    float r[8];
    load8<T>((const T *)l.res + row * l.rs + col, n, r);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] += r[j];
  }
  store8<T>(y + row * ys + col, n, v);
}
