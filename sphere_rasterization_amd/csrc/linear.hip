// Dense layers of a shading network: y = residual + drop(act(x W + b)) in one launch, and
// the gradient dz = drop'(dy) act'(z), dx = dz W^T, dW = x^T dz, db = sums of dz.
//
// Every product is C[i][j] = sum over c of Q[i][c] P[j][c] with j the axis along which C is
// stored: Q and P are x, W, dz or their transposes, read where they lie, whichever of
// their two axes is contiguous.
#include "linear_common.h"
#include "linear_rows.h"

namespace {

typedef float float16v __attribute__((ext_vector_type(16)));
typedef short short4v __attribute__((ext_vector_type(4)));

// What happens to a value on its way to memory.
enum { OUT_STORE, OUT_LAYER, OUT_PART };

struct Operand {
  const void *p;                 // [outer][c] with c contiguous, or [c][outer] (transposed)
  int64_t stride;                // elements between rows of that array
};

struct ProductArgs {
  Operand q, p;
  int64_t I, J, K;               // rows and columns of C, length of the summed axis
  int64_t ti, tj;                // tiles along I and J
  int64_t steps, per;            // stages of the summed axis, and of one split
  void *c;
  int64_t cs;                    // row stride of C
  float *part;                   // [splits][I][J] sums
  LayerArgs layer;
};

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
    typedef float float4v __attribute__((ext_vector_type(4)));
    const float4v a = __builtin_bit_cast(float4v, p), b = __builtin_bit_cast(float4v, q);
#pragma unroll
    for (int k = 0; k < 4; k++) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[k], b[k], acc, 0, 0, 0);
  }
};

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
template <typename T, int TI, int TJ, bool QT, bool PT>
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
    auto fetch = [&](int64_t k) {
#pragma unroll
      for (int n = 0; n < SQ::LOADS; n++) {
        int o, c;
        SQ::place(tid + n * LN_THREADS, o, c);
        rq[n] = SQ::load(a.q, i0 + o, k * SQ::KE + c, a.I, a.K);
      }
#pragma unroll
      for (int n = 0; n < SP::LOADS; n++) {
        int o, c;
        SP::place(tid + n * LN_THREADS, o, c);
        rp[n] = SP::load(a.p, j0 + o, k * SP::KE + c, a.J, a.K);
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
  }
};

// The tile's values, 32 x 32 at a time, through a patch of LDS: eight neighbours of a row
// per lane.
template <typename T, int TI, int TJ, bool QT, bool PT, int OUT>
__global__ __launch_bounds__(LN_THREADS) void k_product(ProductArgs a) {
  typedef Tile<T, TI, TJ, QT, PT> Tl;
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
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = h * 16 + (lane >> 2), c = (lane & 3) * 8;
        float v[8];
        const float4 x = *reinterpret_cast<const float4 *>(patch + r * Tl::PITCH + c);
        const float4 z = *reinterpret_cast<const float4 *>(patch + r * Tl::PITCH + c + 4);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = z.x; v[5] = z.y; v[6] = z.z; v[7] = z.w;
        const int64_t row = wi + i * 32 + r, col = wj + j * 32 + c;
        if (row < a.I && col < a.J) {
          const int n = a.J - col < 8 ? (int)(a.J - col) : 8;
          if constexpr (OUT == OUT_PART) store8<float>(a.part + ((int64_t)blockIdx.y * a.I + row) * a.J + col, n, v);
          else if constexpr (OUT == OUT_STORE) store8<T>((T *)a.c + row * a.cs + col, n, v);
          else finish_layer<T>(a.layer, key, (T *)a.c, a.cs, a.J, row, col, n, v);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
}

// Adds the splits of a product in order; a thread takes eight neighbours of a row.
template <typename T, int OUT>
__global__ __launch_bounds__(LN_THREADS) void k_product_join(ProductArgs a, int splits) {
  const int64_t per = (a.J + 7) / 8, n = per * a.I;
  DropKey key = {};
  if (OUT == OUT_LAYER && a.layer.draw) key = drop_key(a.layer.drop);
  for (int64_t t = (int64_t)blockIdx.x * LN_THREADS + threadIdx.x; t < n; t += (int64_t)gridDim.x * LN_THREADS) {
    const int64_t row = t / per, col = (t - row * per) * 8;
    const int w = a.J - col < 8 ? (int)(a.J - col) : 8;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
      float x[8];
      load8<float>(a.part + ((int64_t)s * a.I + row) * a.J + col, w, x);
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] += x[j];
    }
    if constexpr (OUT == OUT_STORE) store8<T>((T *)a.c + row * a.cs + col, w, v);
    else finish_layer<T>(a.layer, key, (T *)a.c, a.cs, a.J, row, col, w, v);
  }
}

// ---- dz and its column sums ------------------------------------------------------------

struct SlopeArgs {
  const void *dy, *z;            // z packed
  void *dz;                      // packed, or NULL: only the sums
  float *sums;                   // [chunks][N], or NULL
  int64_t M, N, ys, chunk;       // rows per workgroup
  int act, draw;
  DropArgs drop;
};

constexpr int SL_COLS = 64;      // columns per workgroup: eight threads a row, 32 rows at once

// dz = drop'(dy) act'(z) for some rows by 64 columns, and the columns' sums over them.
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
  if (n > 0)
    for (int64_t m = m0 + r; m < m1; m += LN_THREADS / 8) {
      float d[8];
      load8<T>((const T *)a.dy + m * a.ys + col, n, d);
      if (a.act != SPLAT_ACT_NONE) {
        float z[8];
        load8<T>((const T *)a.z + m * a.N + col, n, z);
        slope_times<T>(d, z, a.act);
      }
      if (a.draw) drop8<false>(d, m * a.N + col, a.drop, key);
      if (a.dz) store8<T>((T *)a.dz + m * a.N + col, n, d);
#pragma unroll
      for (int j = 0; j < 8; j++) t[j] += d[j];
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

// db: the chunks' sums in order, a wave's lanes on neighbouring columns.
template <typename T>
__global__ __launch_bounds__(LN_THREADS) void k_linear_bias(const float *sums, int64_t chunks, int64_t N, void *db, int f32) {
  const int64_t col = (int64_t)blockIdx.x * LN_THREADS + threadIdx.x;
  if (col >= N) return;
  float v = 0.0f;
  for (int64_t k = 0; k < chunks; k++) v += sums[k * N + col];
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

constexpr int TILE_SIDE = 64, ENOUGH = 512;            // workgroups that fill the chip twice

struct Split {
  int64_t ti, tj, steps, per;
  int splits;
};
Split split_of(int64_t I, int64_t J, int64_t K, int ke) {
  Split s;
  s.ti = (I + TILE_SIDE - 1) / TILE_SIDE;
  s.tj = (J + TILE_SIDE - 1) / TILE_SIDE;
  s.steps = (K + ke - 1) / ke;
  const int64_t tiles = s.ti * s.tj;
  int64_t want = tiles < ENOUGH ? ENOUGH / tiles : 1;
  if (want > s.steps / 8) want = s.steps / 8;          // at least eight stages each
  if (want < 1) want = 1;
  s.per = (s.steps + want - 1) / want;
  if (s.per < 1) s.per = 1;
  s.splits = (int)((s.steps + s.per - 1) / s.per);
  if (s.splits < 1) s.splits = 1;
  return s;
}
int ke_of(int dtype) { return dtype == SPLAT_F32 ? 16 : 32; }
size_t part_bytes(int64_t I, int64_t J, int64_t K, int dtype) {
  if (I == 0 || J == 0) return 0;
  const Split s = split_of(I, J, K, ke_of(dtype));
  return s.splits > 1 ? ws_align(sizeof(float) * (size_t)s.splits * I * J) : 0;
}

unsigned blocks_for(int64_t items) {
  const int64_t b = (items + LN_THREADS - 1) / LN_THREADS;
  return (unsigned)(b < 1 ? 1 : b < 65536 ? b : 65536);
}

template <typename T, bool QT, bool PT, int OUT>
int run_product(ProductArgs a, hipStream_t stream) {
  const Split s = split_of(a.I, a.J, a.K, ke_of(sizeof(T) == 4 ? SPLAT_F32 : SPLAT_F16));
  a.ti = s.ti;
  a.tj = s.tj;
  a.steps = s.steps;
  a.per = s.per;
  const dim3 grid((unsigned)(s.ti * s.tj), (unsigned)s.splits);
  if (s.splits == 1) {
    hipLaunchKernelGGL((k_product<T, TILE_SIDE, TILE_SIDE, QT, PT, OUT>), grid, dim3(LN_THREADS), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  hipLaunchKernelGGL((k_product<T, TILE_SIDE, TILE_SIDE, QT, PT, OUT_PART>), grid, dim3(LN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  hipLaunchKernelGGL((k_product_join<T, OUT>), dim3(blocks_for(a.I * ((a.J + 7) / 8))), dim3(LN_THREADS), 0, stream, a,
                     s.splits);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

int64_t slope_chunks(int64_t M, int64_t N) {
  const int64_t cols = (N + SL_COLS - 1) / SL_COLS;
  int64_t chunks = (2048 + cols - 1) / cols, most = (M + 63) / 64;
  if (chunks > most) chunks = most;
  return chunks < 1 ? 1 : chunks;
}

// W as [in][out], `out` contiguous, or its transpose.
bool w_by_out(int64_t si, int64_t so) { return so == 1 && si != 1; }

struct Plan {
  size_t pre, dz, sums, part, total;
};
Plan plan_of(const splat_dense *d, bool bwd) {
  Plan p = {};
  const int64_t M = d->rows, N = d->out, K = d->in;
  if (M == 0 || N == 0) return p;
  auto most = [&](size_t v) { if (v > p.part) p.part = v; };
  most(part_bytes(M, N, K, d->dtype));
  if (bwd) {
    const size_t e = dtype_bytes(d->dtype);
    if (d->act != SPLAT_ACT_NONE) p.pre = ws_align((size_t)M * N * e);
    if (d->act != SPLAT_ACT_NONE || d->drop.p > 0.0) p.dz = ws_align((size_t)M * N * e);
    p.sums = ws_align(sizeof(float) * (size_t)slope_chunks(M, N) * N);
    most(part_bytes(M, K, N, d->dtype));
    most(part_bytes(K, N, M, d->dtype));
    most(part_bytes(N, K, M, d->dtype));
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
  a.q = {x, d->x_stride};
  a.c = y;
  a.cs = ys;
  a.part = part;
  a.layer = l;
  if (w_by_out(d->w_in_stride, d->w_out_stride)) {
    a.p = {w, d->w_in_stride};
    return run_product<T, false, true, OUT_LAYER>(a, stream);
  }
  a.p = {w, d->w_out_stride};
  return run_product<T, false, false, OUT_LAYER>(a, stream);
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
    s.sums = db ? sums : nullptr;
    s.M = M;
    s.N = N;
    s.ys = d->y_stride;
    s.act = d->act;
    s.draw = draw;
    s.drop = drop_args(&d->drop);
    const int64_t chunks = slope_chunks(M, N);
    s.chunk = (M + chunks - 1) / chunks;
    const dim3 grid((unsigned)((N + SL_COLS - 1) / SL_COLS), (unsigned)((M + s.chunk - 1) / s.chunk));
    hipLaunchKernelGGL(k_linear_slope<T>, grid, dim3(LN_THREADS), 0, stream, s);
    SPLAT_LAUNCH_CHECK();
    if (db) {
      hipLaunchKernelGGL(k_linear_bias<T>, dim3((unsigned)((N + LN_THREADS - 1) / LN_THREADS)), dim3(LN_THREADS), 0, stream,
                         (const float *)sums, (int64_t)grid.y, N, db, d->bias_dtype == SPLAT_F32);
      SPLAT_LAUNCH_CHECK();
    }
  }
  const Operand z = shaped ? Operand{dz, N} : Operand{dy, d->y_stride};
  if (dx && K > 0) {
    ProductArgs a = {};
    a.I = M;
    a.J = K;
    a.K = N;
    a.q = z;
    a.c = dx;
    a.cs = d->dx_stride;
    a.part = part;
    if (w_by_out(d->w_in_stride, d->w_out_stride)) {
      a.p = {w, d->w_in_stride};
      st = run_product<T, false, false, OUT_STORE>(a, stream);
    } else {
      a.p = {w, d->w_out_stride};
      st = run_product<T, false, true, OUT_STORE>(a, stream);
    }
    if (st) return st;
  }
  if (dw && K > 0) {
    ProductArgs a = {};
    const Operand xo = {x, d->x_stride};
    a.I = by_out ? K : N;
    a.J = by_out ? N : K;
    a.K = M;
    a.q = by_out ? xo : z;
    a.p = by_out ? z : xo;
    a.c = dw;
    a.cs = dws;
    a.part = part;
    return run_product<T, true, true, OUT_STORE>(a, stream);
  }
  return SPLAT_OK;
}

}  // namespace

bool linear_saves(const splat_dense *d) { return d->act != SPLAT_ACT_NONE && !linear_by_rows(d); }

size_t linear_workspace_bytes(const splat_dense *d, bool bwd) {
  if (d->rows == 0 || d->out == 0) return 0;
  if (linear_by_rows(d)) return bwd ? linear_rows_workspace_bytes(d) : 0;
  return plan_of(d, bwd).total;
}

int launch_linear(const splat_dense *d, const void *x, const void *w, const void *bias, const void *res, void *y,
                  void *pre, void *ws, hipStream_t stream) {
  LayerArgs l = {bias, res, pre, d->residual_stride, d->bias_dtype == SPLAT_F32, d->act, d->drop.p > 0.0, drop_args(&d->drop)};
  if (linear_by_rows(d) && !pre) {
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
    const LayerArgs l = {bias, nullptr, nullptr, 0, d->bias_dtype == SPLAT_F32, d->act, d->drop.p > 0.0, drop_args(&d->drop)};
    if (d->dtype == SPLAT_F32) return launch_linear_rows_bwd_f32(d, dy, x, w, l, dx, dw, db, ws, stream);
    if (d->dtype == SPLAT_F16) return launch_linear_rows_bwd_f16(d, dy, x, w, l, dx, dw, db, ws, stream);
    return launch_linear_rows_bwd_bf16(d, dy, x, w, l, dx, dw, db, ws, stream);
  }
  if (d->dtype == SPLAT_F32) return backward<float>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
  if (d->dtype == SPLAT_F16) return backward<f16_t>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
  return backward<bf16_t>(d, dy, x, w, bias, pre, dx, dw, db, ws, stream);
}
