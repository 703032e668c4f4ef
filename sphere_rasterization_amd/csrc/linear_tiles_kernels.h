// Products of any size: tiles on the matrix cores. See linear.hip for which products there are.
#pragma once
#include "linear_tiles.h"

namespace {

typedef float float16v __attribute__((ext_vector_type(16)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

// What lanes read in the place of chunks beyond an array.
__device__ const uint4 zero_chunk = {0, 0, 0, 0};

// ---- tiles -------------------------------------------------------------------------------

template <typename T>
struct Cores;
template <>
struct Cores<f16_t> {
  static __device__ __forceinline__ void mul(const word4 &p, const word4 &q, float16v &acc) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, p), __builtin_bit_cast(half8, q), acc, 0, 0, 0);
  }
};
template <>
struct Cores<bf16_t> {
  static __device__ __forceinline__ void mul(const word4 &p, const word4 &q, float16v &acc) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8, p), __builtin_bit_cast(bhalf8, q), acc, 0, 0, 0);
  }
};
template <>
struct Cores<float> {
  static __device__ __forceinline__ void mul(const word4 &p, const word4 &q, float16v &acc) {
    const float4v a = __builtin_bit_cast(float4v, p), b = __builtin_bit_cast(float4v, q);
#pragma unroll
    for (int k = 0; k < 4; k++) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[k], b[k], acc, 0, 0, 0);
  }
};

// Eight neighbours of a row of C on their way to memory: to the split's sums, or to C.
template <typename T, int OUT>
__device__ __forceinline__ void emit8(const ProductArgs &a, const DropKey &key, int64_t row, int64_t col, int n,
                                      const float (&bias)[8], const word4 (&res)[sizeof(T) / 2], float (&v)[8]) {
  if (a.splits > 1) store8<float>(a.part + ((int64_t)blockIdx.y * a.I + row) * a.J + col, n, v);
  else if constexpr (OUT != OUT_LAYER) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= a.scale;
    store8<T>((T *)a.c + row * a.cs + col, n, v);
  } else finish_layer<T>(a.layer, key, (T *)a.c, a.cs, a.J, row, col, n, bias, res, v);
}

// One operand's share of a stage: TL of its outer places by 64 bytes of the summed axis
// (KE values), 16-byte chunks of its contiguous axis. Not transposed: TL rows of four
// chunks; chunk c of row r lies at c ^ ((r >> 2) & 3), which spreads the 16 rows that a
// fragment read serves at once over all banks. Transposed: KE rows of TL values; for
// 16-bit types the 64-byte units of a row are exchanged by the row's low bits, so that the
// four rows by 64 bytes which half a transposing read serves lie in different banks.
template <typename T, int TL, bool TR>
struct Stage {
  static constexpr int E = 16 / sizeof(T);           // values per chunk
  static constexpr int KE = 64 / sizeof(T);          // values of the summed axis per stage
  static constexpr int LOADS = TL / 64;              // chunks per thread
  static constexpr int CPR = TL / E;                 // chunks per row, transposed
  static constexpr int BYTES = TL * 64;

  static __device__ __forceinline__ int unit_swap(int c) { return TL >= 128 ? (c & 3) : ((c >> 1) & 1); }

  // Chunk q of the stage, in LDS order: its place along the outer axis and the summed one.
  static __device__ __forceinline__ void place(int q, int &outer, int &c) {
    if constexpr (!TR) {
      outer = q >> 2;
      c = ((q & 3) ^ ((outer >> 2) & 3)) * E;
    } else {
      c = q / CPR;
      const int slot = q % CPR;
      if constexpr (sizeof(T) == 2) outer = ((((slot >> 2) ^ unit_swap(c)) << 2) | (slot & 3)) * E;
      else outer = slot * E;
    }
  }

  // The chunk from memory, zeros beyond the array: any alignment.
  static __device__ __forceinline__ word4 load(const Operand &o, int64_t outer, int64_t c, int64_t R, int64_t K) {
    word4 v = {0, 0, 0, 0};
    const int64_t row = TR ? c : outer, at = TR ? outer : c, rows = TR ? K : R, len = TR ? R : K;
    if (row < rows && at < len) {
      const T *s = (const T *)o.p + row * o.stride + at;
      if (at + E <= len) {
        v = *reinterpret_cast<const typename Loose<T, E>::type *>(s);
      } else {
        Pack<T, E> t = __builtin_bit_cast(Pack<T, E>, v);
#pragma unroll
        for (int j = 0; j < E; j++)
          if (at + j < len) t.v[j] = s[j];
        v = __builtin_bit_cast(word4, t);
      }
    }
    return v;
  }

  // Fragment of 32 outer places from `at`, block u (32 bytes) of the stage: a lane holds
  // place lane % 32 and chunk 2 u + lane / 32 of the summed axis.
  static __device__ __forceinline__ word4 fragment(const char *l, int at, int u) {
    const int lane = threadIdx.x & 63, r = at + (lane & 31), k = 2 * u + (lane >> 5);
    if constexpr (!TR) {
      return *reinterpret_cast<const word4 *>(l + (r * 4 + (k ^ ((r >> 2) & 3))) * 16);
    } else if constexpr (sizeof(T) == 4) {
      word4 v;
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = *reinterpret_cast<const uint32_t *>(l + ((k * 4 + j) * TL + r) * 4);
      return v;
    } else {
      // 16 lanes read 4 rows of 16 columns and each gets a column
      typedef __attribute__((address_space(3))) short4v *lds4;
      const int j = lane & 15, col = at + (lane & 16) + (j & 3) * 4;        // first of four columns
      word4 v;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = k * 8 + h * 4 + (j >> 2);
        const int unit = (col >> 5) ^ unit_swap(c);
        const short4v t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4)(short4v *)const_cast<char *>(l + (c * TL + unit * 32 + (col & 31)) * 2));
        const uint2 w = __builtin_bit_cast(uint2, t);
        v[2 * h] = w.x;
        v[2 * h + 1] = w.y;
      }
      return v;
    }
  }
};

// TI x TJ tile of C by four waves, a quarter each.
// The sums of second parts, once all of them are in.
template <typename T, int FI, int FJ>
__device__ __forceinline__ void take_rest(float16v (&acc)[FI][FJ]) {
#pragma unroll
  for (int i = 0; i < FI; i++)
#pragma unroll
    for (int j = 0; j < FJ; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] *= REST<T>;
}

template <typename T, int TI, int TJ, bool QT, bool PT, int OUT>
struct Tile {
  typedef Stage<T, TI, QT> SQ;
  typedef Stage<T, TJ, PT> SP;
  static constexpr int FI = TI / 64, FJ = TJ / 64;   // fragments per side of a wave's quarter
  static constexpr int STAGE = SQ::BYTES + SP::BYTES;
  static constexpr int PITCH = 36;                   // floats between rows of the epilogue's patch of 32 x 32
  static constexpr int LDS = 2 * STAGE > 4 * 32 * PITCH * 4 ? 2 * STAGE : 4 * 32 * PITCH * 4;

  static __device__ __forceinline__ void product(const ProductArgs &a, int64_t i0, int64_t j0, int64_t k0, int64_t k1,
                                                 char *lds, float16v (&acc)[FI][FJ]) {
    const int tid = threadIdx.x, w = tid >> 6;
    const int wi = (w & 1) * (TI / 2), wj = (w >> 1) * (TJ / 2);
#pragma unroll
    for (int i = 0; i < FI; i++)
#pragma unroll
      for (int j = 0; j < FJ; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    word4 rq[SQ::LOADS], rp[SP::LOADS];
    // Where a thread's chunks lie in the first stage. Rows beyond the array: any of its own.
    // Whole chunks of the summed axis are read as they lie, and past a row's end where that is
    // C's edge; the last two stages, in which the axis and the array end, value by value.
    typedef const typename Loose<T, SQ::E>::type *ptr;
    const T *sq[SQ::LOADS], *sp[SP::LOADS];
    auto aim = [&](const Operand &o, bool tr, int64_t outer, int64_t R, int c) {
      const int64_t r = outer < R ? outer : tr ? 0 : R - 1;
      return (const T *)o.p + (tr ? c * o.stride + r : r * o.stride + c);
    };
#pragma unroll
    for (int n = 0; n < SQ::LOADS; n++) {
      int o, c;
      SQ::place(tid + n * LN_THREADS, o, c);
      sq[n] = aim(a.q, QT, i0 + o, a.I, c);
    }
#pragma unroll
    for (int n = 0; n < SP::LOADS; n++) {
      int o, c;
      SP::place(tid + n * LN_THREADS, o, c);
      sp[n] = aim(a.p, PT, j0 + o, a.J, c);
    }
    const int64_t dq = QT ? a.q.stride * SQ::KE : SQ::KE, dp = PT ? a.p.stride * SP::KE : SP::KE;
    auto fetch = [&](int64_t stage) {
      const bool first = stage >= a.axis, second = a.parts == 2 && !first;
      const int64_t k = first ? stage - a.axis : stage;
      const int64_t rest_q = second ? a.q.rest : 0, rest_p = second ? a.p.rest : 0;
      if (k < a.axis - 2) {
#pragma unroll
        for (int n = 0; n < SQ::LOADS; n++) rq[n] = *(ptr)((const char *)(sq[n] + k * dq) + rest_q);
#pragma unroll
        for (int n = 0; n < SP::LOADS; n++) rp[n] = *(ptr)((const char *)(sp[n] + k * dp) + rest_p);
        return;
      }
      const Operand q = {(const char *)a.q.p + rest_q, a.q.stride, 0}, p = {(const char *)a.p.p + rest_p, a.p.stride, 0};
#pragma unroll
      for (int n = 0; n < SQ::LOADS; n++) {
        int o, c;
        SQ::place(tid + n * LN_THREADS, o, c);
        rq[n] = SQ::load(q, i0 + o, k * SQ::KE + c, a.I, a.K);
      }
#pragma unroll
      for (int n = 0; n < SP::LOADS; n++) {
        int o, c;
        SP::place(tid + n * LN_THREADS, o, c);
        rp[n] = SP::load(p, j0 + o, k * SP::KE + c, a.J, a.K);
      }
    };
    auto keep = [&](int slot) {
      char *l = lds + slot * STAGE;
#pragma unroll
      for (int n = 0; n < SQ::LOADS; n++) *reinterpret_cast<word4 *>(l + (tid + n * LN_THREADS) * 16) = rq[n];
#pragma unroll
      for (int n = 0; n < SP::LOADS; n++)
        *reinterpret_cast<word4 *>(l + SQ::BYTES + (tid + n * LN_THREADS) * 16) = rp[n];
    };
    if (k0 < k1) {
      fetch(k0);
      keep(0);
    }
    __syncthreads();
    int slot = 0;
    for (int64_t k = k0; k < k1; k++) {
      if (OUT == OUT_PARTS && k == a.axis) take_rest<T>(acc);
      if (k + 1 < k1) fetch(k + 1);
      const char *l = lds + slot * STAGE;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        word4 fq[FI], fp[FJ];
#pragma unroll
        for (int i = 0; i < FI; i++) fq[i] = SQ::fragment(l, wi + i * 32, u);
#pragma unroll
        for (int j = 0; j < FJ; j++) fp[j] = SP::fragment(l + SQ::BYTES, wj + j * 32, u);
#pragma unroll
        for (int i = 0; i < FI; i++)
#pragma unroll
          for (int j = 0; j < FJ; j++) Cores<T>::mul(fp[j], fq[i], acc[i][j]);
      }
      if (k + 1 < k1) keep(slot ^ 1);
      __syncthreads();
      slot ^= 1;
    }
    if (OUT == OUT_PARTS && k1 <= a.axis) take_rest<T>(acc);
  }
};

// The tile's values, 32 x 32 at a time, through a patch of LDS: eight neighbours of a row
// per lane.
template <typename T, int TI, int TJ, bool QT, bool PT, int OUT>
__global__ __launch_bounds__(LN_THREADS) void k_product(ProductArgs a) {
  typedef Tile<T, TI, TJ, QT, PT, OUT> Tl;
  __shared__ __attribute__((aligned(16))) char lds[Tl::LDS];
  const int64_t t = blockIdx.x, i0 = (t / a.tj) * TI, j0 = (t % a.tj) * TJ;
  const int64_t k0 = blockIdx.y * a.per, k1 = k0 + a.per < a.steps ? k0 + a.per : a.steps;
  float16v acc[Tl::FI][Tl::FJ];
  Tl::product(a, i0, j0, k0, k1, lds, acc);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t wi = i0 + (w & 1) * (TI / 2), wj = j0 + (w >> 1) * (TJ / 2);
  float *patch = reinterpret_cast<float *>(lds) + w * 32 * Tl::PITCH;
  DropKey key = {};
  if (OUT == OUT_LAYER && a.layer.draw) key = drop_key(a.layer.drop);
#pragma unroll
  for (int i = 0; i < Tl::FI; i++)
#pragma unroll
    for (int j = 0; j < Tl::FJ; j++) {
      // a lane holds column lane % 32 of Q's places and places 8 e + 4 (lane / 32) .. + 3 of P's
#pragma unroll
      for (int e = 0; e < 4; e++)
        *reinterpret_cast<float4 *>(patch + (lane & 31) * Tl::PITCH + 8 * e + 4 * (lane >> 5)) =
            make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
      wave_lds_order();
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = h * 16 + (lane >> 2), c = (lane & 3) * 8;
        float v[8];
        load8<float>(patch + r * Tl::PITCH + c, 8, v);
        const int64_t row = wi + i * 32 + r, col = wj + j * 32 + c;
        if (row < a.I && col < a.J) {
          const int n = a.J - col < 8 ? (int)(a.J - col) : 8;
          float bias[8];
          word4 res[sizeof(T) / 2];
          if constexpr (OUT == OUT_LAYER) {
            load_bias<T>(a.layer, col, n, bias);
            load_res<T>(a.layer, row, col, n, res);
          }
          emit8<T, OUT>(a, key, row, col, n, bias, res, v);
        }
      }
      wave_lds_order();
    }
}

// The same product for arrays whose rows are whole, aligned chunks: loads go straight to LDS.
// WI x WJ waves share a TI x TJ tile; NST stages form a ring in LDS. In step k, after the wait
// for stage k + 1 and a barrier, stage k (already in registers) is free for stage k + NST, the
// fragments of stage k + 1 are read, and those of stage k are multiplied: loads have NST - 1
// steps to arrive, and fragment reads a step.
// 16 bytes from each lane's address to consecutive places of LDS from `at`, uniform. Written out,
// because the compiler waits for every load that it knows to be on its way to LDS before it
// reads LDS by the transposing instruction, which would leave one stage in flight (8192 x 4096
// by 4096 x 4096 bf16: 359 us).
__device__ __forceinline__ void to_lds(const void *p, uint32_t at) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(at) : "m0", "memory");
}

// Asks the compiler for the step's fragment reads and matrix instructions in turn.
template <int R, int READS, int MULS>
__device__ __forceinline__ void interleave() {
  if constexpr (R < READS) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, (R + 1) * MULS / READS - R * MULS / READS, 0);
    interleave<R + 1, READS, MULS>();
  }
}

template <typename T, int TI, int TJ, int WI, int WJ, int NST, bool QT, bool PT, int OUT>
struct Direct {
  typedef Stage<T, TI, QT> SQ;
  typedef Stage<T, TJ, PT> SP;
  static constexpr int THREADS = WI * WJ * WAVE;
  static constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;
  static constexpr int LQ = TI * 4 / THREADS, LP = TJ * 4 / THREADS, LOADS = LQ + LP;
  static constexpr int STAGE = SQ::BYTES + SP::BYTES;
  static constexpr int PITCH = 68;                   // floats between rows of the epilogue's patch of 32 x 64
  static constexpr int PATCH = 32 * PITCH * 4;
  static constexpr int RING = NST * STAGE;
  // fragment reads and matrix instructions of a step
  static constexpr int READS = FI * 2 * (!QT ? 1 : sizeof(T) == 2 ? 2 : 4) + FJ * 2 * (!PT ? 1 : sizeof(T) == 2 ? 2 : 4);
  static constexpr int MULS = FI * FJ * 2 * (sizeof(T) == 2 ? 1 : 4);
  static constexpr int LDS = RING > WI * WJ * PATCH ? RING : WI * WJ * PATCH;

  static __device__ __forceinline__ void product(const ProductArgs &a, int64_t i0, int64_t j0, int k0, int k1, char *lds,
                                                 float16v (&acc)[FI][FJ]) {
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = (w % WI) * (TI / WI), wj = (w / WI) * (TJ / WJ);
    const char *src[LOADS];
    int at[LOADS];                                   // the chunk's place along the summed axis
    auto aim = [&](const Operand &o, int64_t outer0, int64_t R, bool tr, int outer, int c, int n) {
      int64_t r = outer0 + outer;
      if (tr) r = r < R ? r : 0;                     // columns and rows beyond C: any of the array's
      else r = r < R ? r : R - 1;
      src[n] = (const char *)o.p + (tr ? c * o.stride + r : r * o.stride + c) * (int64_t)sizeof(T);
      at[n] = c;
    };
#pragma unroll
    for (int n = 0; n < LQ; n++) {
      int o, c;
      SQ::place(tid + n * THREADS, o, c);
      aim(a.q, i0, a.I, QT, o, c, n);
    }
#pragma unroll
    for (int n = 0; n < LP; n++) {
      int o, c;
      SP::place(tid + n * THREADS, o, c);
      aim(a.p, j0, a.J, PT, o, c, LQ + n);
    }
    const uint32_t base = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds + w * (WAVE * 16));
    const int64_t dq = (QT ? a.q.stride * SQ::KE : SQ::KE) * (int64_t)sizeof(T);
    const int64_t dp = (PT ? a.p.stride * SP::KE : SP::KE) * (int64_t)sizeof(T);
    const int skip = a.parts == 2 ? (int)a.axis : 0;
    // the last stage; with OUT_PARTS one more may follow it, of zeros, so that a part's are even
    const int last = (int)((a.K - 1) / SQ::KE), left = (int)(a.K - (int64_t)last * SQ::KE);
    // stages past the end load the last one again, so that the count of loads in flight
    // stays a constant
    auto fetch = [&](int k, int slot) {
      const int stage = k < k1 ? k : k1 - 1;
      // second parts come first
      const bool second = OUT != OUT_LAYER && a.parts == 2 && stage < (int)a.axis;
      const int kk = OUT == OUT_LAYER || second ? stage : stage - skip;
      const uint32_t l = base + slot * STAGE;
      const int64_t oq = kk * dq + (second ? a.q.rest : 0), op = kk * dp + (second ? a.p.rest : 0);
      const bool whole = kk < last || (left == SQ::KE && (OUT != OUT_PARTS || kk == last));
      const int there = OUT == OUT_PARTS && kk > last ? 0 : left;
#pragma unroll
      for (int n = 0; n < LOADS; n++) {
        const char *p = src[n] + (n < LQ ? oq : op);
        if (!whole && at[n] >= there) p = reinterpret_cast<const char *>(&zero_chunk);
        to_lds(p, l + (n < LQ ? n * THREADS * 16 : SQ::BYTES + (n - LQ) * THREADS * 16));
      }
    };
#pragma unroll
    for (int i = 0; i < FI; i++)
#pragma unroll
      for (int j = 0; j < FJ; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    word4 fq[2][2][FI], fp[2][2][FJ];
    auto read = [&](int slot, int set) {
      const char *l = lds + slot * STAGE;
#pragma unroll
      for (int u = 0; u < 2; u++) {
#pragma unroll
        for (int i = 0; i < FI; i++) fq[set][u][i] = SQ::fragment(l, wi + i * 32, u);
#pragma unroll
        for (int j = 0; j < FJ; j++) fp[set][u][j] = SP::fragment(l + SQ::BYTES, wj + j * 32, u);
      }
    };
#pragma unroll
    for (int k = 0; k < NST; k++) fetch(k0 + k, k);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NST - 1) * LOADS) : "memory");
    read(0, 0);
    int slot = 0;                                    // of stage k
    auto step = [&](int k, int set) {
      const int next = slot + 1 == NST ? 0 : slot + 1;
      // the oldest stage in flight is in LDS for this wave and its own fragment reads
      // are done (seen by the compiler's own count), then the same of the other waves
      __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0)
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NST - 2) * LOADS) : "memory");
      fetch(k + NST, slot);
      read(next, set ^ 1);
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < FI; i++)
#pragma unroll
          for (int j = 0; j < FJ; j++) Cores<T>::mul(fp[set][u][j], fq[set][u][i], acc[i][j]);
      interleave<0, READS, MULS>();
      __builtin_amdgcn_sched_barrier(0);
      slot = next;
    };
    int k = k0;
    for (; k + 1 < k1; k += 2) {
      // a workgroup has an even number of the second parts' stages
      if (OUT == OUT_PARTS && k == (int)a.axis) take_rest<T>(acc);
      step(k, 0);
      step(k + 1, 1);
    }
    if (k < k1) step(k, 0);
    if (OUT == OUT_PARTS && k1 <= (int)a.axis) take_rest<T>(acc);
    // nothing may land in LDS after this
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
};

// Workgroups go to the eight XCDs in turn. Work item of workgroup b out of n such that each
// XCD takes a run of neighbouring items, whose operands its own L2 then holds.
__device__ __forceinline__ int64_t by_xcd(int64_t b, int64_t n) {
  const int64_t x = b & 7, each = n >> 3, more = n & 7;
  return x * each + (x < more ? x : more) + (b >> 3);
}

// 8192 x 4096 by 4096 x 4096 bf16: 244 to 255 us, 1.1 PFLOP/s with 256 x 256 tiles, whose fragment
// reads and loads take LDS as long as the matrix cores take (a library product 211, 1.3);
// with 128 x 128 tiles 320 to 340, with 64 x 128 390 to 440. 8191 x 1024 by 1024 x 4096 bf16 with
// gelu: 92 to 99 us, a third of it the epilogue, in which the matrix cores rest. 4095 x 1536 by
// 1536 x 1000 fp32: 107 to 122 us, 103 to 117 TFLOP/s of the 154 of a large library product.
template <typename T, int TI, int TJ, int WI, int WJ, int NST, bool QT, bool PT, int OUT>
__global__ __launch_bounds__(WI * WJ * WAVE, TI * TJ > 128 * 128 * WI * WJ / 2 ? 1 : 2) void k_direct(ProductArgs a) {
  typedef Direct<T, TI, TJ, WI, WJ, NST, QT, PT, OUT> D;
  __shared__ __attribute__((aligned(16))) char lds[D::LDS];
  // runs of eight tiles along I by all of J
  const int64_t t = by_xcd(blockIdx.x, a.ti * a.tj), band = t / (8 * a.tj), in = t - band * 8 * a.tj;
  const int64_t high = a.ti - band * 8 < 8 ? a.ti - band * 8 : 8;
  const int64_t i0 = (band * 8 + in % high) * TI, j0 = in / high * TJ;
  const int k0 = (int)(blockIdx.y * a.per), k1 = k0 + a.per < a.steps ? (int)(k0 + a.per) : (int)a.steps;
  float16v acc[D::FI][D::FJ];
  D::product(a, i0, j0, k0, k1, lds, acc);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t wi = i0 + (w % WI) * (TI / WI), wj = j0 + (w / WI) * (TJ / WJ);
  float *patch = reinterpret_cast<float *>(lds + w * D::PATCH);
  DropKey key = {};
  if (OUT == OUT_LAYER && a.layer.draw) key = drop_key(a.layer.drop);
  // 32 x 64 values at a time through a patch of LDS, eight neighbours of a row per lane; the
  // residual of the next eight rows is on its way meanwhile
  constexpr int FJ2 = D::FJ / 2;
  const int pr = lane >> 3, pc = (lane & 7) * 8;
  const bool want_res = OUT == OUT_LAYER && a.layer.res && a.splits == 1;
  word4 next[sizeof(T) / 2];
  auto ahead = [&](int at) {                         // rows 8 at .. of the wave's quarter, FI * 4 of them to a column block
    const int64_t row = wi + at % (D::FI * 4) * 8 + pr, col = wj + at / (D::FI * 4) * 64 + pc;
    if (want_res && row < a.I && col < a.J) load_res<T>(a.layer, row, col, a.J - col < 8 ? (int)(a.J - col) : 8, next);
  };
  ahead(0);
  float bias[8];
#pragma unroll 1
  for (int b = 0; b < D::FI * FJ2; b++) {
    const int64_t col = wj + b / D::FI * 64 + pc;
    const int n = a.J <= col ? 0 : a.J - col < 8 ? (int)(a.J - col) : 8;
    if (OUT == OUT_LAYER && b % D::FI == 0) load_bias<T>(a.layer, col, n, bias);
#pragma unroll
    for (int s = 0; s < D::FI * FJ2; s++)
      if (s == b) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float16v &v = acc[s % D::FI][s / D::FI * 2 + h];
            *reinterpret_cast<float4 *>(patch + (lane & 31) * D::PITCH + h * 32 + 8 * e + 4 * (lane >> 5)) =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
      }
    wave_lds_order();
#pragma unroll 1
    for (int h = 0; h < 4; h++) {
      const int64_t row = wi + b % D::FI * 32 + h * 8 + pr;
      word4 res[sizeof(T) / 2];
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; k++) res[k] = next[k];
      if (b * 4 + h + 1 < D::FI * FJ2 * 4) ahead(b * 4 + h + 1);
      float v[8];
      load8<float>(patch + (h * 8 + pr) * D::PITCH + pc, 8, v);
      if (row < a.I && n > 0) emit8<T, OUT>(a, key, row, col, n, bias, res, v);
    }
    wave_lds_order();
  }
}

// Adds the splits of a product in order, eight neighbours of a row at a time, and finishes
// them. SLICES threads share the splits of the same eight, where there are many for few values.
template <typename T, int OUT, int SLICES>
__global__ __launch_bounds__(LN_THREADS) void k_product_join(ProductArgs a, int splits) {
  constexpr int G = LN_THREADS / SLICES;
  __shared__ float s[SLICES > 1 ? SLICES * G * 9 : 1];
  const int64_t per = (a.J + 7) / 8, n = per * a.I;
  const int g = threadIdx.x % G, l = threadIdx.x / G;
  DropKey key = {};
  if (OUT == OUT_LAYER && a.layer.draw) key = drop_key(a.layer.drop);
  a.splits = 1;
  for (int64_t t0 = (int64_t)blockIdx.x * G; t0 < n; t0 += (int64_t)gridDim.x * G) {
    const int64_t t = t0 + g, row = t / per, col = (t - row * per) * 8;
    const int w = t >= n ? 0 : a.J - col < 8 ? (int)(a.J - col) : 8;
    float v[8] = {};
    if (w > 0) {
#pragma unroll 4
      for (int k = l; k < splits; k += SLICES) {
        float x[8];
        load8<float>(a.part + ((int64_t)k * a.I + row) * a.J + col, w, x);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] += x[j];
      }
    }
    if constexpr (SLICES > 1) {
#pragma unroll
      for (int j = 0; j < 8; j++) s[(l * G + g) * 9 + j] = v[j];
      __syncthreads();
      if (l == 0) {
        for (int k = 1; k < SLICES; k++)
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] += s[(k * G + g) * 9 + j];
      }
      __syncthreads();
      if (l > 0) continue;
    }
    if (w > 0) {
      float bias[8];
      word4 res[sizeof(T) / 2];
      if constexpr (OUT == OUT_LAYER) {
        load_bias<T>(a.layer, col, w, bias);
        load_res<T>(a.layer, row, col, w, res);
      }
      emit8<T, OUT>(a, key, row, col, w, bias, res, v);
    }
  }
}

// ---- few rows --------------------------------------------------------------------------

// Products of at most 16 rows of Q, as for single tokens: bound by reading P once. A workgroup
// takes some columns of C and its waves share the summed axis; P goes from memory straight
// into the layout of the matrix cores, whose 16 columns are Q's rows.
//   P by c: 16-byte chunks of 16 rows of P are operands as they lie.
//   P by j (PT): a lane reads E neighbours of a row of P, for as many rows as a chunk holds
//   values, and turns them around in registers: fragment e stands for columns E i + e. (fp32
//   needs no turning: an instruction takes one value a lane.)
// 1 x 2048 by 2048 x 8192 bf16: 8.3 us, 4.0 TB/s; by 64 x 64 tiles and a join of splits 15.
template <typename T, bool PT>
struct Few {
  static constexpr int E = 16 / sizeof(T), KE = 64 / sizeof(T);
  static constexpr int WAVES = 8, THREADS = WAVES * WAVE;
  static constexpr int TILES_J = PT ? E : 2;         // fragments of 16 columns
  static constexpr int J = 16 * TILES_J;             // columns of a workgroup
  static constexpr int PITCH = J + 4;
  static constexpr int UNROLL = PT ? 2 : 4;          // steps of 64 bytes whose loads are on the way together
};

// 16 x 16 products of one chunk a lane.
template <typename T>
__device__ __forceinline__ float4v few_mul(const word4 &a, const word4 &b, float4v c);
template <>
__device__ __forceinline__ float4v few_mul<f16_t>(const word4 &a, const word4 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ float4v few_mul<bf16_t>(const word4 &a, const word4 &b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8, a), __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ float4v few_mul<float>(const word4 &a, const word4 &b, float4v c) {
  const float4v x = __builtin_bit_cast(float4v, a), y = __builtin_bit_cast(float4v, b);
#pragma unroll
  for (int k = 0; k < 4; k++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[k], y[k], c, 0, 0, 0);
  return c;
}

// Value e of each of the rows' chunks, as one chunk.
template <typename T>
__device__ __forceinline__ word4 turn(const word4 (&rows)[16 / sizeof(T)], int e) {
  word4 v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; k++) v[k] = rows[k][e];
  } else {
#pragma unroll
    for (int k = 0; k < 4; k++)
      v[k] = __builtin_amdgcn_perm(rows[2 * k + 1][e >> 1], rows[2 * k][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
  }
  return v;
}

template <typename T, bool PT, int OUT>
__global__ __launch_bounds__((Few<T, PT>::THREADS)) void k_few(ProductArgs a) {
  typedef Few<T, PT> F;
  constexpr int E = F::E, KE = F::KE, NT = F::TILES_J, U = F::UNROLL, LOADS = PT ? E : NT;
  typedef const typename Loose<T, E>::type *ptr;
  __shared__ __attribute__((aligned(16))) float sums[F::WAVES * 16 * F::PITCH];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, w = threadIdx.x >> 6;
  const int64_t j0 = (int64_t)blockIdx.x * F::J;
  // stages of this workgroup's share of the axis, and of this wave's
  const int K = (int)a.K, from = (int)(blockIdx.y * a.per), to = from + a.per < a.axis ? (int)(from + a.per) : (int)a.axis;
  const int per = (to - from + F::WAVES - 1) / F::WAVES;
  const int s0 = from + w * per, s1 = s0 + per < to ? s0 + per : to;
  constexpr bool REST_APART = OUT == OUT_PARTS;
  float4v acc[NT], acc2[REST_APART ? NT : 1];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    acc[t] = float4v{0, 0, 0, 0};
    if constexpr (REST_APART) acc2[t] = float4v{0, 0, 0, 0};
  }
  const T *q = (const T *)a.q.p + i * a.q.stride + g * E, *q2 = (const T *)((const char *)q + a.q.rest);
  const bool row = i < a.I;
  for (int s = s0; s < s1; s += U) {
    word4 p[U][LOADS], x[U], x2[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = (s + u) * KE + g * E;            // the lane's chunk of the summed axis
      const bool on = s + u < s1 && c < K;           // whole: K is whole chunks
      x[u] = x2[u] = word4{0, 0, 0, 0};
      if (on && row) {
        x[u] = *reinterpret_cast<ptr>(q + (int64_t)(s + u) * KE);
        if (a.parts == 2) x2[u] = *reinterpret_cast<ptr>(q2 + (int64_t)(s + u) * KE);
      }
#pragma unroll
      for (int n = 0; n < LOADS; n++) {
        const int64_t j = PT ? j0 + i * E : j0 + 16 * n + i;
        p[u][n] = word4{0, 0, 0, 0};
        if (on && j < a.J)
          p[u][n] = *reinterpret_cast<ptr>((const T *)a.p.p + (PT ? (int64_t)(c + n) * a.p.stride + j : j * a.p.stride + c));
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int t = 0; t < NT; t++) {
        word4 f;
        if constexpr (PT) f = turn<T>(p[u], t);
        else f = p[u][t];
        acc[t] = few_mul<T>(f, x[u], acc[t]);
        float4v &sum = REST_APART ? acc2[REST_APART ? t : 0] : acc[t];
        if (a.parts == 2) sum = few_mul<T>(f, x2[u], sum);
      }
  }
  if constexpr (REST_APART) {
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int r = 0; r < 4; r++) acc[t][r] = __builtin_fmaf(acc2[t][r], REST<T>, acc[t][r]);
  }
  // a lane holds row i of C: of fragment t rows 4 g + r of P's, columns 16 t + 4 g + r of the
  // tile, or E (4 g + r) + t
  float *mine = sums + (w * 16 + i) * F::PITCH;
  if constexpr (!PT) {
#pragma unroll
    for (int t = 0; t < NT; t++)
      *reinterpret_cast<float4 *>(mine + 16 * t + 4 * g) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int t = 0; t < NT; t += 4)
        *reinterpret_cast<float4 *>(mine + E * (4 * g + r) + t) = make_float4(acc[t][r], acc[t + 1][r], acc[t + 2][r], acc[t + 3][r]);
  }
  __syncthreads();
  DropKey key = {};
  if (OUT == OUT_LAYER && a.layer.draw) key = drop_key(a.layer.drop);
  for (int t = threadIdx.x; t < (int)a.I * (F::J / 8); t += F::THREADS) {
    const int r = t / (F::J / 8), c = t % (F::J / 8) * 8;
    const int64_t col = j0 + c;
    if (col >= a.J) continue;
    const int n = a.J - col < 8 ? (int)(a.J - col) : 8;
    float bias[8], v[8] = {};
    word4 res[sizeof(T) / 2];
    if constexpr (OUT == OUT_LAYER) {
      load_bias<T>(a.layer, col, n, bias);
      load_res<T>(a.layer, r, col, n, res);
    }
#pragma unroll
    for (int k = 0; k < F::WAVES; k++) {
      float o[8];
      load8<float>(sums + (k * 16 + r) * F::PITCH + c, 8, o);
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] += o[j];
    }
    emit8<T, OUT>(a, key, r, col, n, bias, res, v);
  }
}

// ---- host ----------------------------------------------------------------------------

// Whether every row is whole chunks at chunk addresses.
template <typename T>
bool whole_chunks(const Operand &o, bool tr, int64_t R, int64_t K) {
  constexpr int E = 16 / sizeof(T);
  return ((uintptr_t)o.p & 15) == 0 && o.stride % E == 0 && (tr ? R : K) % E == 0;
}

template <typename T, int OUT>
int join(const ProductArgs &a, hipStream_t stream) {
  constexpr int TO = OUT == OUT_LAYER ? OUT_LAYER : OUT_STORE;
  const int64_t items = a.I * ((a.J + 7) / 8);
  auto blocks = [](int64_t n) { return dim3((unsigned)(n < 65536 ? n : 65536)); };
  if (a.splits >= 16 && items < 65536)
    hipLaunchKernelGGL((k_product_join<T, TO, 16>), blocks((items + 15) / 16), dim3(LN_THREADS), 0, stream, a, a.splits);
  else
    hipLaunchKernelGGL((k_product_join<T, TO, 1>), blocks((items + LN_THREADS - 1) / LN_THREADS), dim3(LN_THREADS), 0, stream, a,
                       a.splits);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T, bool QT, bool PT, int OUT>
int run_product(ProductArgs a, hipStream_t stream) {
  constexpr int KE = 64 / sizeof(T);
  constexpr bool FOUR = QT && PT && OUT != OUT_PARTS;    // waves of the largest tiles, or eight
  const Cut cut = product_cut(a.I, a.J, a.K, a.parts, sizeof(T) == 4 ? SPLAT_F32 : SPLAT_F16);
  a.axis = (a.K + KE - 1) / KE;
  if constexpr (!QT) {
    if (a.I <= FEW && a.K > 0 && a.K % (16 / (int)sizeof(T)) == 0 && (!PT || a.J % (16 / (int)sizeof(T)) == 0)) {
      const int splits = few_splits(a.J, a.K, PT, sizeof(T) == 4 ? SPLAT_F32 : SPLAT_F16);
      a.per = (a.axis + splits - 1) / splits;
      a.splits = (int)((a.axis + a.per - 1) / a.per);
      const dim3 grid((unsigned)((a.J + Few<T, PT>::J - 1) / Few<T, PT>::J), (unsigned)a.splits);
      hipLaunchKernelGGL((k_few<T, PT, OUT>), grid, dim3(Few<T, PT>::THREADS), 0, stream, a);
      SPLAT_LAUNCH_CHECK();
      return a.splits > 1 ? join<T, OUT>(a, stream) : SPLAT_OK;
    }
  }
  const bool direct = a.K > 0 && whole_chunks<T>(a.q, QT, a.I, a.K) && whole_chunks<T>(a.p, PT, a.J, a.K), even = direct && OUT == OUT_PARTS;
  if (even) a.axis += a.axis & 1;
  a.steps = a.axis * a.parts;
  a.per = (a.steps + cut.splits - 1) / cut.splits;
  if (even) a.per += a.per & 1;
  a.splits = a.per > 0 ? (int)((a.steps + a.per - 1) / a.per) : 1;
  // arrays that are not whole, aligned chunks: tiles of 128 or 64 through registers; of 16-bit
  // types 128 wherever they fill the chip (4001 x 999 to 1501 bf16: 43 us, 61 with 64)
  const int64_t tiles = ((a.I + 127) / 128) * ((a.J + 127) / 128) * a.splits;
  const int loose = cut.tile < 2 || (sizeof(T) == 2 && tiles >= 256) ? 128 : 64, side_i = !direct ? loose : TILES[cut.tile].i, side_j = !direct ? loose : TILES[cut.tile].j;
  a.ti = (a.I + side_i - 1) / side_i;
  a.tj = (a.J + side_j - 1) / side_j;
  const dim3 grid((unsigned)(a.ti * a.tj), (unsigned)a.splits);
  if (!direct && loose == 128)
    hipLaunchKernelGGL((k_product<T, 128, 128, QT, PT, OUT>), grid, dim3(LN_THREADS), 0, stream, a);
  else if (!direct)
    hipLaunchKernelGGL((k_product<T, 64, 64, QT, PT, OUT>), grid, dim3(LN_THREADS), 0, stream, a);
  else if (cut.tile == 0) {                          // 16-bit types alone
    // transposing reads bring half as much a cycle: with both operands transposed four waves of
    // 128 x 128, which read least, beat eight (4096 by 4096 by 4096 bf16, forward and backward: 381 us, 407 with eight).
    // With sums to multiply on the way their registers do not suffice (532 bytes a lane spill)
    if constexpr (sizeof(T) == 2)
      hipLaunchKernelGGL((k_direct<T, 256, 256, 2, FOUR ? 2 : 4, 4, QT, PT, OUT>), grid, dim3(FOUR ? 256 : 512), 0, stream, a);
  } else if (cut.tile == 1)
    hipLaunchKernelGGL((k_direct<T, 128, 128, 2, 2, 4, QT, PT, OUT>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_direct<T, 64, 128, 2, 2, 4, QT, PT, OUT>), grid, dim3(256), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  return a.splits > 1 ? join<T, OUT>(a, stream) : SPLAT_OK;
}

template <typename T>
int product(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t s) {
  if (out == OUT_LAYER) return pt ? run_product<T, false, true, OUT_LAYER>(a, s) : run_product<T, false, false, OUT_LAYER>(a, s);
  if constexpr (REST<T> != 1.0f) {
    if (a.parts == 2) {
      if (qt) return run_product<T, true, true, OUT_PARTS>(a, s);
      return pt ? run_product<T, false, true, OUT_PARTS>(a, s) : run_product<T, false, false, OUT_PARTS>(a, s);
    }
  }
  if (qt) return run_product<T, true, true, OUT_STORE>(a, s);
  return pt ? run_product<T, false, true, OUT_STORE>(a, s) : run_product<T, false, false, OUT_STORE>(a, s);
}

}  // namespace
