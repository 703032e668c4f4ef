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

__device__ __forceinline__ uint4 philox(uint32_t x0, uint32_t x1, const DropKey &k) {
  uint32_t x2 = k.o0, x3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; r++) {
    const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
    x1 = (uint32_t)b;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// Which of elements 8 block .. 8 block + 7 are kept, as bits. u_i is 16 bits of the draw
// (block, 0) above the same 16 bits of the draw (block, 1); the second is needed only where
// the first equals the threshold's, once in 65536 elements: 32 bits of resolution at the
// price of 16, which is what leaves dropout of 16-bit images bound by memory.
__device__ __forceinline__ uint32_t drop_keeps(uint64_t block, const DropArgs &d, const DropKey &k) {
  const uint32_t b0 = (uint32_t)block, b1 = (uint32_t)(block >> 32);
  const uint4 w4 = philox(b0, b1, k);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  uint32_t keep = 0, tie = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const uint32_t u = j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
    keep |= u > d.high ? 1u << j : 0u;
    tie |= u == d.high ? 1u << j : 0u;
  }
  if (tie) {
    const uint4 v4 = philox(b0, b1 | 0x80000000u, k);
    const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t u = j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xFFFFu;
      if ((tie >> j & 1) && u >= d.low) keep |= 1u << j;
    }
  }
  return keep;
}

static inline DropArgs drop_args(const splat_drop *d) {
  const uint64_t t = (uint64_t)rint(d->p * 4294967296.0);         // the product is exact; at most 2^32
  DropArgs a = {d->state, d->seed, d->offset, (uint32_t)(t >> 16), (uint32_t)(t & 0xFFFF), 1.0f};
  a.scale = d->p < 1.0 ? (float)(1.0 / (1.0 - d->p)) : 0.0f;
  return a;
}
