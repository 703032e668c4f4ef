// Accesses of eight neighbouring elements, of any type and alignment.
#pragma once
#include "learn_common.h"

// The first n of eight elements at p, zeros beyond them.
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
// A last piece of n < 8 is stored by fours, twos and ones: three accesses in place of eight.
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float (&o)[8]) {
  constexpr int N = 16 / sizeof(T);
  Pack<T, 8> t;
#pragma unroll
  for (int j = 0; j < 8; j++) t.v[j] = (T)o[j];
  if (n == 8) {
    const Pack<Raw<T, N>, 8 / N> r = __builtin_bit_cast(Pack<Raw<T, N>, 8 / N>, t);
#pragma unroll
    for (int m = 0; m < 8 / N; m++) *reinterpret_cast<typename Loose<T, N>::type *>(p + m * N) = r.v[m];
  } else if (n > 0) {
    const Pack<Raw<T, 4>, 2> r = __builtin_bit_cast(Pack<Raw<T, 4>, 2>, t);
    if (n & 4) *reinterpret_cast<typename Loose<T, 4>::type *>(p) = r.v[0];
    const Raw<T, 4> four = n & 4 ? r.v[1] : r.v[0];
    const Pack<Raw<T, 2>, 2> q = __builtin_bit_cast(Pack<Raw<T, 2>, 2>, four);
    if (n & 2) *reinterpret_cast<typename Loose<T, 2>::type *>(p + (n & 4)) = q.v[0];
    const Raw<T, 2> two = n & 2 ? q.v[1] : q.v[0];
    if (n & 1) p[n & 6] = __builtin_bit_cast(Pack<T, 2>, two).v[0];
  }
}
// The same past the caches, for results that this call does not read again.
template <typename T>
__device__ __forceinline__ void stream8(T *p, int n, const float (&o)[8]) {
  constexpr int N = 16 / sizeof(T);
  if (n == 8) {
#pragma unroll
    for (int m = 0; m < 8; m += N) {
      float t[N];
#pragma unroll
      for (int j = 0; j < N; j++) t[j] = o[m + j];
      stream_loose<T, N>(p + m, t);
    }
  } else {
    store8<T>(p, n, o);
  }
}
