// Counter-based random numbers: Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011), and the choice that dropout makes
// for eight neighbouring elements from one or, now and then, two draws.
#pragma once
#include <math.h>

#include "splat_internal.h"

// What a kernel needs to drop: element i is dropped where u_i < threshold, u_i of 32 bits.
struct DropArgs {
  const uint64_t *state;       // seed and offset on the device, or NULL
  uint64_t seed, offset;
  uint32_t high, low;          // threshold >> 16 (up to 65536) and its lower 16 bits
  float scale;                 // 1 / (1 - p), 0 for p = 1
};

// The same with the state read: uniform over the launch.
struct DropKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const DropArgs &d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.state) {
    seed = d.state[0];
    offset += d.state[1];
  }
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// a ^ b ^ c in one instruction (the bits of a truth table).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ uint4 philox(uint32_t x0, uint32_t x1, const DropKey &k) {
  uint32_t x2 = k.o0, x3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; r++) {
    const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = xor3((uint32_t)(b >> 32), x1, k0);
    x2 = xor3((uint32_t)(a >> 32), x3, k1);
    x1 = (uint32_t)b;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// Which of elements 8 block .. 8 block + 7 are kept, as bits.
// u_i is 16 bits of that draw above the same 16 bits of the draw (block, 1); the second is
// needed only where the first equals the threshold's, once in 65536 elements: 32 bits of
// resolution at the price of 16. The branch is one of the whole wave, so that the compiler
// cannot trade it for drawing twice.
__device__ __forceinline__ uint32_t piece_of(const uint4 &w, int j) {
  const uint32_t v = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return j & 1 ? v >> 16 : v & 0xFFFFu;
}
__device__ __forceinline__ bool any_tie(const uint4 &w, uint32_t high) {
  bool tie = false;
#pragma unroll
  for (int j = 0; j < 8; j++) tie |= piece_of(w, j) == high;
  return __builtin_expect(ballot64(tie) != 0, 0);
}
__device__ __forceinline__ uint32_t keep_bits(uint64_t block, const DropArgs &d, const DropKey &k) {
  const uint4 w = philox((uint32_t)block, (uint32_t)(block >> 32), k);
  uint32_t keep = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) keep |= piece_of(w, j) > d.high ? 1u << j : 0u;
  if (any_tie(w, d.high)) {
    const uint4 v = philox((uint32_t)block, (uint32_t)(block >> 32) | 0x80000000u, k);
#pragma unroll
    for (int j = 0; j < 8; j++) keep |= piece_of(w, j) == d.high && piece_of(v, j) >= d.low ? 1u << j : 0u;
  }
  return keep;
}

// Dropout of elements at .. at + 7, `at` any element, or (ALIGNED) a multiple of eight.
template <bool ALIGNED>
__device__ __forceinline__ void drop8(float (&v)[8], int64_t at, const DropArgs &d, const DropKey &k) {
  const uint64_t block = (uint64_t)at >> 3;
  const uint32_t sh = ALIGNED ? 0u : (uint32_t)at & 7;
  const bool apart = !ALIGNED && ballot64(sh != 0) != 0;
  if (!apart) {
    const uint4 w = philox((uint32_t)block, (uint32_t)(block >> 32), k);
    if (!any_tie(w, d.high)) {
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = piece_of(w, j) > d.high ? v[j] * d.scale : 0.0f;
      return;
    }
  }
  uint32_t bits = 0;
#pragma unroll 1
  for (uint32_t t = 0; t < (apart ? 2u : 1u); t++) bits |= keep_bits(block + t, d, k) << (8 * t);
  bits >>= sh;
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = bits >> j & 1 ? v[j] * d.scale : 0.0f;
}

static inline DropArgs drop_args(const splat_drop *d) {
  const uint64_t t = (uint64_t)rint(d->p * 4294967296.0);         // the product is exact; at most 2^32
  DropArgs a = {d->state, d->seed, d->offset, (uint32_t)(t >> 16), (uint32_t)(t & 0xFFFF), 1.0f};
  a.scale = d->p < 1.0 ? (float)(1.0 / (1.0 - d->p)) : 0.0f;
  return a;
}
// The same choice without its factor.
static inline DropArgs mask_args(const splat_drop *d) {
  DropArgs a = drop_args(d);
  a.scale = 1.0f;
  return a;
}
