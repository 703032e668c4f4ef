// Helpers shared by the appearance operators (lookup, group norm, orthogonalisation):
// element types, packed loads and stores, exact division by a launch constant.
#pragma once
#include "splat_internal.h"

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// N consecutive elements, moved as one access when aligned to their size.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// The bits of a pack as whole words: what the compiler keeps in registers unsplit.
template <int BYTES>
struct RawBits;
template <>
struct RawBits<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <>
struct RawBits<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <>
struct RawBits<4> { typedef uint32_t type; };
template <>
struct RawBits<2> { typedef uint16_t type; };
template <typename T, int N>
using Raw = typename RawBits<sizeof(T) * N>::type;

template <typename T, int N>
__device__ __forceinline__ void to_f32(const Raw<T, N> &r, float (&o)[N]) {
  const Pack<T, N> x = __builtin_bit_cast(Pack<T, N>, r);
#pragma unroll
  for (int i = 0; i < N; i++) o[i] = (float)x.v[i];
}

// The same bits at any element's address: the compiler then asks no more of the address,
// and the hardware takes the access whole, aligned or not.
template <typename T, int N>
struct Loose {
  typedef Raw<T, N> type __attribute__((aligned(alignof(T))));
};

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T *p, float (&o)[N]) {
  to_f32<T, N>(*reinterpret_cast<const Raw<T, N> *>(p), o);
}

// The pack at p, or zeros. Several of these are in flight together when they are
// converted only after the last one: a conversion next to its load, under the load's
// condition, waits for that load alone.
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> load_if(bool ok, const T *p) {
  Raw<T, N> x = {};
  if (ok) x = *reinterpret_cast<const Raw<T, N> *>(p);
  return x;
}

// One rounding to the nearest value of the type.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T *p, const float (&o)[N]) {
  Pack<T, N> x;
#pragma unroll
  for (int i = 0; i < N; i++) x.v[i] = (T)o[i];
  *reinterpret_cast<Pack<T, N> *>(p) = x;
}

// The same for results that this call does not read again: they pass by the caches that
// hold its inputs.
template <typename T, int N>
__device__ __forceinline__ void stream_f32(T *p, const float (&o)[N]) {
  if constexpr (sizeof(T) * N == 16) {
    Pack<T, N> x;
#pragma unroll
    for (int i = 0; i < N; i++) x.v[i] = (T)o[i];
    __builtin_nontemporal_store(__builtin_bit_cast(Raw<T, N>, x), reinterpret_cast<Raw<T, N> *>(p));
  } else {
    store_f32<T, N>(p, o);
  }
}

// load_if and stream_f32 at any element's address.
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> load_loose_if(bool ok, const T *p) {
  Raw<T, N> x = {};
  if (ok) x = *reinterpret_cast<const typename Loose<T, N>::type *>(p);
  return x;
}
template <typename T, int N>
__device__ __forceinline__ void stream_loose(T *p, const float (&o)[N]) {
  Pack<T, N> x;
#pragma unroll
  for (int i = 0; i < N; i++) x.v[i] = (T)o[i];
  __builtin_nontemporal_store(__builtin_bit_cast(Raw<T, N>, x), reinterpret_cast<typename Loose<T, N>::type *>(p));
}

// fp32 sums kept in the workspace: 16-byte accesses where N allows.
template <int N>
__device__ __forceinline__ void load_sums(const float *p, float (&o)[N]) {
  if constexpr (N == 8) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    load_f32<float, N>(p, o);
  }
}
template <int N>
__device__ __forceinline__ void store_sums(float *p, const float (&o)[N]) {
  if constexpr (N == 8) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    store_f32<float, N>(p, o);
  }
}

// x / d for 0 <= x < 2^31 and a divisor known at launch, as one 64-bit product:
// with l = ceil(log2 d) and m = floor(2^(31 + l) / d) + 1, m d - 2^(31 + l) lies in
// (0, 2^l], so floor(x m / 2^(31 + l)) = floor(x / d) for every x < 2^31.
struct FastDiv {
  uint32_t d, m, s;
};
static inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  uint32_t l = 0;
  while ((1ull << l) < d) l++;
  f.d = d;
  f.s = 31 + l;
  f.m = (uint32_t)((1ull << f.s) / d + 1);
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t x, const FastDiv &f) {
  return (uint32_t)(((uint64_t)x * f.m) >> f.s);
}

static inline int dtype_bytes(int dtype) { return dtype == SPLAT_F32 ? 4 : 2; }

// The widest power-of-two number of elements, at most 16 bytes, by which a row can
// be walked: it divides the row length, every stride and every pointer's alignment.
static inline int vec_width(int bytes, int dim, const int64_t *strides, int n_strides, const void *const *ptrs,
                            int n_ptrs) {
  int v = 16 / bytes;
  for (; v > 1; v >>= 1) {
    bool ok = dim % v == 0;
    for (int i = 0; ok && i < n_strides; i++) ok = strides[i] % v == 0;
    for (int i = 0; ok && i < n_ptrs; i++) ok = ((uintptr_t)ptrs[i] % (uintptr_t)(v * bytes)) == 0;
    if (ok) break;
  }
  return v;
}

static inline size_t ws_align(size_t x) { return (x + 255) & ~(size_t)255; }
