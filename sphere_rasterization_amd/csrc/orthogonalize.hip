// Orthogonalised updates: an odd quintic applied to a matrix's singular values by
// products alone (Newton-Schulz iteration), as in momentum optimisers for weight
// matrices.
//
//   X = G / (|G|_F + eps), transposed if it has more rows than columns (m <= n);
//   steps times: A = X X^T, B = a I + b A + c A A, X <- B X;  output = scale X.
//
// Bound by the matrix cores: m^2 n / 2 + m^3 / 2 + m^2 n multiply-adds a step with the
// symmetric products' halves counted once (only tiles on or below the diagonal are
// computed; each is written to both places).
//
// Precision. Directions with small singular values grow by up to a^steps (about 485
// for the usual coefficients), and the rounding of the operands grows with them, so
// one 11-bit operand per factor is not enough. Every operand is kept as two fp16
// parts, v S = hi + lo (22 bits and more; S a power of two from a bound on the
// singular values, so that neither part leaves fp16's range), and a product is
// hi hi + hi lo + lo hi on the matrix cores with fp32 sums (with few rows also lo lo, which is
// below 2^-22 of the product). Three fp16 products still run several times faster
// than one in fp32, whose matrix rate on gfx950 is 1/16 of fp16's.
//
// Layout. A factor is stored in panels of 64 rows, a panel in blocks of 16 values of the
// summed axis, and in a block each row's 16 hi then 16 lo parts: 64 bytes. So a block is
// a contiguous 4 KB, loaded straight into LDS, and the two parts travel together. X is
// kept both by rows and transposed, because X X^T sums over columns and B X over rows.
#include <math.h>

#include "learn_common.h"

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int KB = 16;                 // values per block of the summed axis
constexpr int BLOCK = 64 * 2 * KB;     // halves per block of a panel
constexpr int OR_THREADS = 256;
constexpr int NORM_BLOCKS = 1024;

enum { EPI_GRAM, EPI_POLY, EPI_NEXT, EPI_LAST };

struct OrthoArgs {
  const void *g;
  void *out;
  int64_t gb, gr, ob, orow;            // batch and row strides of the input and the output
  int dtype, rows, cols, tall;
  int m, n, mp, np;                    // m <= n, and padded to multiples of the tile
  int tile;
  float *part;                         // sums of shared-out products
  double *norms;                       // [batch][NORM_BLOCKS] partial sums of squares
  _Float16 *x, *y, *y2, *a, *b;        // packed factors: X, X^T (two), A, B; per matrix strides below
  int64_t sx, sa;                      // halves per matrix of x / y, and of a / b
  float eps, s0;                       // s0: scale of X before the first step
};

struct GemmArgs {
  const _Float16 *p, *q;               // factors by rows [I][K], [J][K], packed
  int64_t pb, qb;                      // halves per matrix
  int K;                               // padded length of the summed axis
  int ti;                              // tiles along I
  int tiles;                           // tiles per matrix
  // shared-out products: the sums of piece (run w, tile t) lie at part[w + t]
  float *part;
  int64_t units;                       // double steps of all tiles of all matrices
  float mul;                           // product of the stored sums to the stored result's scale
  // EPI_POLY: result = ca I + cb A + mul acc with A read from `a` (stored scale folded in)
  const _Float16 *a;
  float ca, cb;
  _Float16 *d0, *d1;                   // result by rows [I][J] and transposed [J][I], packed
  int64_t db;
  int ld0, ld1;                        // padded row lengths of d0 and d1, in values
  // EPI_LAST
  void *out;
  int64_t ob, orow;
  int dtype, tall, m, n;
};

__device__ __forceinline__ float read_as_f32(const void *p, int64_t i, int dtype) {
  if (dtype == SPLAT_F32) return ((const float *)p)[i];
  if (dtype == SPLAT_F16) return (float)((const f16_t *)p)[i];
  return (float)((const bf16_t *)p)[i];
}
__device__ __forceinline__ void write_from_f32(void *p, int64_t i, int dtype, float v) {
  if (dtype == SPLAT_F32) ((float *)p)[i] = v;
  else if (dtype == SPLAT_F16) ((f16_t *)p)[i] = (f16_t)v;
  else ((bf16_t *)p)[i] = (bf16_t)v;
}

// What brings G to X S: G times pre times inv, inv = s0 / (norm + eps) / pre. The power of
// two pre keeps inv within fp32 where the norm alone would not (below 1e-34 with eps = 0);
// it is exact, and one in between.
__device__ __forceinline__ void unit_scale(double sum_of_squares, float eps, float s0, float &pre, float &inv) {
  const double d = sqrt(sum_of_squares) + (double)eps;
  pre = d < 0x1p-64 ? 0x1p64f : d > 0x1p64 ? 0x1p-64f : 1.0f;
  inv = (float)((double)s0 / d / (double)pre);
}

// Place of the hi part of value k of row r, for rows of K values; lo lies KB further.
__device__ __forceinline__ int64_t packed(int r, int k, int K) {
  return ((int64_t)(r >> 6) * (K / KB) + k / KB) * BLOCK + (r & 63) * (2 * KB) + k % KB;
}

// Sums of squares in fp64: no square over- or underflows and the norm is exact to fp32.
// Rows in turn; a thread has 8 independent loads in flight.
__global__ __launch_bounds__(OR_THREADS) void k_ortho_norm(OrthoArgs o) {
  __shared__ double s[OR_THREADS / WAVE];
  const int64_t mat = blockIdx.y;
  const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
  double t = 0.0;
  const int64_t per = 8 * OR_THREADS;                     // values of a row per piece
  const int64_t pieces = (o.cols + per - 1) / per;
  for (int64_t i = blockIdx.x; i < pieces * o.rows; i += gridDim.x) {
    const int64_t r = i / pieces, c0 = (i - r * pieces) * per + threadIdx.x;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int64_t c = c0 + k * OR_THREADS;
      v[k] = c < o.cols ? read_as_f32(g, r * o.gr + c, o.dtype) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; k++) t = __builtin_fma((double)v[k], (double)v[k], t);
  }
  t = wave_sum_f64(t);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) o.norms[mat * NORM_BLOCKS + blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// X S and its transpose, packed, zero beyond the matrix. A workgroup takes 32 x 32
// values of G; `norm_blocks` partial sums give the norm.
__global__ __launch_bounds__(OR_THREADS) void k_ortho_pack(OrthoArgs o, int norm_blocks) {
  __shared__ float t[32][33];
  __shared__ double s[OR_THREADS / WAVE];
  const int64_t mat = blockIdx.z;
  double q = 0.0;
  for (int k = threadIdx.x; k < norm_blocks; k += OR_THREADS) q += o.norms[mat * NORM_BLOCKS + k];
  q = wave_sum_f64(q);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = q;
  __syncthreads();
  float pre, inv;
  unit_scale((s[0] + s[1]) + (s[2] + s[3]), o.eps, o.s0, pre, inv);
  const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
  // direct image: rows of G; cross image: its columns
  _Float16 *direct = (o.tall ? o.y : o.x) + mat * o.sx, *cross = (o.tall ? o.x : o.y) + mat * o.sx;
  const int dlen = o.tall ? o.mp : o.np, clen = o.tall ? o.np : o.mp;
  const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int r = r0 + ty + k, c = c0 + tx;
    const float v = r < o.rows && c < o.cols ? read_as_f32(g, r * o.gr + c, o.dtype) * pre * inv : 0.0f;
    t[ty + k][tx] = v;
    const _Float16 hi = (_Float16)v;
    _Float16 *d = direct + packed(r, c, dlen);
    d[0] = hi;
    d[KB] = (_Float16)(v - (float)hi);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int r = r0 + tx, c = c0 + ty + k;
    const float v = t[tx][ty + k];
    const _Float16 hi = (_Float16)v;
    _Float16 *d = cross + packed(c, r, clen);
    d[0] = hi;
    d[KB] = (_Float16)(v - (float)hi);
  }
}

// TL x TL tile (it, jt) of D = P Q^T, steps [k0, k1) of the summed axis, by four waves, a
// quarter each. A stage holds SUB blocks of the tile's rows of P and Q; NST stages form a
// ring in LDS, filled by loads that go straight there. In step k, after the wait for
// stage k + 1 and a barrier, stage k (already in registers) is free for stage k + NST,
// the fragments of stage k + 1 are read, and those of stage k are multiplied: loads have
// NST - 1 steps to arrive, and fragment reads a step.
//
// In a block the 16-byte chunk c of row r lies at c ^ ((r >> 2) & 3): a fragment read
// serves 16 rows in a cycle from 64 banks, four rows to a line of banks, and so meets no
// bank twice (with an exchange by r & 3 the bank conflict counter shows twice the cycles).
template <int TL, int SUB, int NST>
struct Tile {
  static constexpr int F = TL / 64;                  // 32 x 32 fragments per side of a wave's quarter, and panels
  static constexpr int LOADS = SUB * 2 * F;          // loads per thread and stage, 16 bytes each
  static constexpr int BLK = BLOCK / 8;              // 16-byte chunks per block
  static constexpr int RING = NST * SUB * 2 * F * BLK;
  static constexpr int PATCH = F * 2 * (32 * 40 + 16) / 8;   // 16-byte chunks of a wave's patch in the epilogue
  static constexpr int LDS = RING > 4 * PATCH ? RING : 4 * PATCH;

  static __device__ __forceinline__ void product(const _Float16 *p0, const _Float16 *q0, int K, int it, int jt,
                                                 int k0, int k1, bool one_tile, half8 *lds,
                                                 float16v (&acc)[F][F]) {
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = (w & 1) * (TL / 2), wj = (w >> 1) * (TL / 2);
    const int64_t panel = (int64_t)(K / KB) * BLOCK;
    // chunk tid of a block, in the order in which LDS holds them
    const int src = ((tid >> 2) * 4 + ((tid & 3) ^ ((tid >> 4) & 3))) * 8;
    const _Float16 *p = p0 + (int64_t)it * F * panel + src, *q = q0 + (int64_t)jt * F * panel + src;
    typedef const __attribute__((address_space(1))) void *gptr;
    typedef __attribute__((address_space(3))) void *lptr;
    // stages past the end load the last one again, so that the count of loads in flight
    // stays a constant
    auto fetch = [&](int k, int slot) {
      const int64_t at = (int64_t)(k < k1 ? k : k1 - 1) * (SUB * BLOCK);
#pragma unroll
      for (int u = 0; u < SUB; u++)
#pragma unroll
        for (int f = 0; f < F; f++) {
          half8 *d = &lds[(slot * SUB + u) * (2 * F * BLK) + f * BLK + w * 64];
          __builtin_amdgcn_global_load_lds((gptr)(p + at + u * BLOCK + f * panel), (lptr)d, 16, 0, 0);
          __builtin_amdgcn_global_load_lds((gptr)(q + at + u * BLOCK + f * panel), (lptr)(d + F * BLK), 16, 0, 0);
        }
    };
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
      for (int j = 0; j < F; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    const int fr = lane & 31, fk = lane >> 5;
    // a fragment's chunk: row fr of its 32, hi chunk fk, lo chunk fk + 2
    const int sw = (fr >> 2) & 3, hi_at = fr * 4 + (fk ^ sw), lo_at = fr * 4 + ((fk + 2) ^ sw);
    half8 ph[2][SUB][F], pl[2][SUB][F], qh[2][SUB][F], ql[2][SUB][F];
    auto read = [&](int slot, int set) {
#pragma unroll
      for (int u = 0; u < SUB; u++) {
        const half8 *l = &lds[(slot * SUB + u) * (2 * F * BLK)];
#pragma unroll
        for (int i = 0; i < F; i++) {
          const half8 *a = l + (wi + i * 32) * 4, *b = l + F * BLK + (wj + i * 32) * 4;
          pl[set][u][i] = a[lo_at];
          qh[set][u][i] = b[hi_at];
          ph[set][u][i] = a[hi_at];
          ql[set][u][i] = b[lo_at];
        }
      }
    };
    // 64 x 64 tiles wait for memory rather than for the matrix cores and can afford sums of
    // their own for the small products. Where one tile holds all rows, lo lo is among them:
    // with few rows and long sums it is a good part of the error (8 x 2048 fp32: 1.9 times
    // that of fp32 products without, 1.2 with; all tiles with it: 1000 x 777 bf16 from 165
    // to 177 us).
    float16v small[F][F];
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
      for (int j = 0; j < F; j++) small[i][j] = acc[i][j];
    auto multiply = [&](int set) {
#pragma unroll
      for (int u = 0; u < SUB; u++) {
        if constexpr (F == 1) {
          if (one_tile)
            small[0][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[set][u][0], ql[set][u][0], small[0][0], 0, 0, 0);
          acc[0][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[set][u][0], qh[set][u][0], acc[0][0], 0, 0, 0);
          small[0][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[set][u][0], qh[set][u][0], small[0][0], 0, 0, 0);
          small[0][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[set][u][0], ql[set][u][0], small[0][0], 0, 0, 0);
          continue;
        }
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
          for (int j = 0; j < F; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[set][u][i], qh[set][u][j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
          for (int j = 0; j < F; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[set][u][i], ql[set][u][j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
          for (int j = 0; j < F; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[set][u][i], qh[set][u][j], acc[i][j], 0, 0, 0);
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
      __builtin_amdgcn_sched_barrier(0);
      multiply(set);
      __builtin_amdgcn_sched_barrier(0);
      slot = next;
    };
    // The matrix cores' running sums lose bits as they grow: every 256 values they are
    // added to the total and start again.
    float16v total[F][F];
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
      for (int j = 0; j < F; j++) total[i][j] = acc[i][j];
    constexpr int FLUSH = 256 / (KB * SUB);
    for (int k = k0; k < k1; k += 2) {               // an even number of steps
      step(k, 0);
      step(k + 1, 1);
      if ((k - k0) % FLUSH == FLUSH - 2) {
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
          for (int j = 0; j < F; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) {
              total[i][j][e] += acc[i][j][e];
              acc[i][j][e] = 0.0f;
            }
      }
    }
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
      for (int j = 0; j < F; j++) acc[i][j] += total[i][j] + small[i][j];
    // nothing may land in LDS after this
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }

  // Writes row i of fragments of a wave's quarter. A lane holds column fr and rows 8 (e / 4) + 4 fk +
  // e % 4 of each fragment. Packed results go through LDS by patches of 32 rows of the
  // wave's quarter, rows padded to 40 halves, so that memory sees whole 16-byte chunks of
  // consecutive rows.
  template <int EPI>
  static __device__ __forceinline__ void finish(const GemmArgs &g, int64_t mat, int it, int jt, int w,
                                                int i, _Float16 *patch, const float16v (&acc)[F]) {
    const int lane = threadIdx.x & 63, fr = lane & 31, fk = lane >> 5;
    const int wi = (w & 1) * (TL / 2), wj = (w >> 1) * (TL / 2);
    const int I = it * TL + wi + i * 32, Jw = jt * TL + wj;
    half4 hi[F][4], lo[F][4];
#pragma unroll
    for (int j = 0; j < F; j++) {
      const int J = Jw + j * 32 + fr;
#pragma unroll
      for (int e4 = 0; e4 < 4; e4++) {
        const int I0 = I + e4 * 8 + fk * 4;
        half4 ah, al;                                  // A (symmetric) at row J, values I0 .. I0 + 3
        if constexpr (EPI == EPI_POLY) {
          const _Float16 *a = g.a + mat * g.db + packed(J, I0, g.ld0);
          ah = *reinterpret_cast<const half4 *>(a);
          al = *reinterpret_cast<const half4 *>(a + KB);
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float v = acc[j][e4 * 4 + e] * g.mul;
          if constexpr (EPI == EPI_POLY) {
            v = __builtin_fmaf(g.cb, (float)ah[e] + (float)al[e], v);
            if (I0 + e == J) v += g.ca;
          }
          if constexpr (EPI == EPI_LAST) {
            if (I0 + e < g.m && J < g.n)
              write_from_f32(g.out, mat * g.ob + (g.tall ? J * g.orow + I0 + e : (I0 + e) * g.orow + J), g.dtype, v);
          } else {
            hi[j][e4][e] = (_Float16)v;
            lo[j][e4][e] = (_Float16)(v - (float)hi[j][e4][e]);
          }
        }
      }
    }
    if constexpr (EPI != EPI_LAST) {
      // by rows: 2 F blocks of 32 rows
      constexpr int B0 = 32 * 40 + 16, B1 = F * 32 * 40 + 16;
#pragma unroll
      for (int j = 0; j < F; j++)
#pragma unroll
        for (int e4 = 0; e4 < 4; e4++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            _Float16 *d = patch + (j * 2 + (fr >> 4)) * B0 + (e4 * 8 + fk * 4 + e) * 40 + (fr & 15);
            d[0] = hi[j][e4][e];
            d[KB] = lo[j][e4][e];
          }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < F * 4; u++) {
        const int c = u * 64 + lane, blk = c >> 7, r = (c >> 2) & 31, k = c & 3;
        const half8 v = *reinterpret_cast<const half8 *>(patch + blk * B0 + r * 40 + k * 8);
        *reinterpret_cast<half8 *>(g.d0 + mat * g.db + packed(I + r, Jw + blk * KB, g.ld0) + k * 8) = v;
      }
      // transposed (of a symmetric result: the tile above the diagonal): 2 blocks of 32 F rows
      if (EPI == EPI_NEXT || it != jt) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
          for (int e4 = 0; e4 < 4; e4++) {
            _Float16 *d = patch + (e4 >> 1) * B1 + (j * 32 + fr) * 40 + (e4 & 1) * 8 + fk * 4;
            *reinterpret_cast<half4 *>(d) = hi[j][e4];
            *reinterpret_cast<half4 *>(d + KB) = lo[j][e4];
          }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < F * 4; u++) {
          const int c = u * 64 + lane, blk = c / (F * 128), r = (c >> 2) % (F * 32), k = c & 3;
          const half8 v = *reinterpret_cast<const half8 *>(patch + blk * B1 + r * 40 + k * 8);
          *reinterpret_cast<half8 *>(g.d1 + mat * g.db + packed(Jw + r, I + blk * KB, g.ld1) + k * 8) = v;
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
};

// Tile t of the lower triangle, by rows.
__device__ __forceinline__ void lower_tile(int t, int &it, int &jt) {
  it = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((it + 1) * (it + 2) / 2 <= t) it++;
  while (it * (it + 1) / 2 > t) it--;
  jt = t - it * (it + 1) / 2;
}

// Workgroups go to the eight XCDs in turn. Work item of workgroup b out of n such that
// each XCD takes a run of neighbouring items, whose panels its own L2 then holds.
__device__ __forceinline__ int by_xcd(int b, int n) {
  const int x = b & 7, each = n >> 3, more = n & 7;
  return x * each + (x < more ? x : more) + (b >> 3);
}

// A whole tile per workgroup. B X of 2048 x 4096, 103 GFLOP of fp16 products: 108 to 120
// us, 0.86 to 0.95 PFLOP/s, where a plain fp16 library product reaches 1.2 to 1.3; the
// matrix cores are busy for 57 % of the time in which CUs have work, and the launch and
// its write-back of 67 MB take a sixth. 777 x 1000: 10 us, 0.2 us a step of 32: two
// 8 KB blocks per CU and step through its 64 bytes a cycle of cache bandwidth.
template <int EPI, int TL, int SUB, int NST>
__global__ __launch_bounds__(OR_THREADS, 2) void k_ortho_gemm(GemmArgs g) {
  typedef Tile<TL, SUB, NST> Tl;
  __shared__ half8 lds[Tl::LDS];
  const int64_t mat = blockIdx.y;
  int it, jt;
  if constexpr (EPI == EPI_GRAM || EPI == EPI_POLY) {
    lower_tile(blockIdx.x, it, jt);
  } else {
    it = blockIdx.x % g.ti;
    jt = blockIdx.x / g.ti;
  }
  float16v acc[Tl::F][Tl::F];
  Tl::product(g.p + mat * g.pb, g.q + mat * g.qb, g.K, it, jt, 0, g.K / (KB * SUB), g.ti == 1, lds, acc);
  const int w = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < Tl::F; i++)
    Tl::template finish<EPI>(g, mat, it, jt, w, i, reinterpret_cast<_Float16 *>(lds + w * Tl::PATCH), acc[i]);
}

// Symmetric products with too few tiles to fill the chip evenly: the steps of all tiles,
// laid end to end, are cut into equal runs, one per workgroup, and a second kernel adds
// the pieces of each tile in order.
template <int TL, int SUB, int NST>
__global__ __launch_bounds__(OR_THREADS, 2) void k_ortho_pieces(GemmArgs g) {
  typedef Tile<TL, SUB, NST> Tl;
  __shared__ half8 lds[Tl::LDS];
  const int per = g.K / (KB * SUB) / 2;              // double steps per tile
  const int run = by_xcd(blockIdx.x, gridDim.x);
  int64_t u = g.units * run / gridDim.x;
  const int64_t end = g.units * (run + 1) / gridDim.x;
  while (u < end) {
    const int t = (int)(u / per), from = (int)(u - (int64_t)t * per);
    const int to = end - u < per - from ? from + (int)(end - u) : per;
    const int64_t mat = t / g.tiles;
    int it, jt;
    lower_tile((int)(t - mat * g.tiles), it, jt);
    float16v acc[Tl::F][Tl::F];
    Tl::product(g.p + mat * g.pb, g.q + mat * g.qb, g.K, it, jt, 2 * from, 2 * to, g.ti == 1, lds, acc);
    float4 *o = reinterpret_cast<float4 *>(g.part + ((int64_t)run + t) * TL * TL) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < Tl::F; i++)
#pragma unroll
      for (int j = 0; j < Tl::F; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          o[((i * Tl::F + j) * 4 + e) * OR_THREADS] =
              make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
    u += to - from;
  }
}

// A workgroup per row of fragments of a tile's quarter: each wave adds every fourth piece,
// first to last, and the first wave adds the four sums and writes the result.
template <int EPI, int TL, int SUB, int NST>
__global__ __launch_bounds__(OR_THREADS) void k_ortho_join(GemmArgs g, int groups) {
  typedef Tile<TL, SUB, NST> Tl;
  constexpr int F = Tl::F;
  __shared__ float4 sums[3][F * 4][WAVE];
  __shared__ half8 lds[Tl::PATCH];
  const int per = g.K / (KB * SUB) / 2;
  const int i = blockIdx.x % F, w = blockIdx.x / F & 3, t = blockIdx.x / (F * 4);
  const int64_t mat = t / g.tiles;
  int it, jt;
  lower_tile((int)(t - mat * g.tiles), it, jt);
  // the first and the last run [units r / groups, units (r + 1) / groups) that meets the
  // tile's [t per, (t + 1) per)
  const int64_t lo = (int64_t)t * per, hi = lo + per;
  int first = (int)(lo * groups / g.units), last = (int)((hi - 1) * groups / g.units);
  while (g.units * (first + 1) / groups <= lo) first++;
  while (g.units * (last + 1) / groups < hi) last++;
  const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  float4 a[F * 4];
#pragma unroll
  for (int e = 0; e < F * 4; e++) a[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int r = first + part; r <= last; r += 4) {
    const float4 *o = reinterpret_cast<const float4 *>(g.part + ((int64_t)r + t) * TL * TL) +
                      i * F * 4 * OR_THREADS + w * WAVE + lane;
#pragma unroll
    for (int e = 0; e < F * 4; e++) {
      const float4 x = o[e * OR_THREADS];
      a[e].x += x.x; a[e].y += x.y; a[e].z += x.z; a[e].w += x.w;
    }
  }
  if (part > 0) {
#pragma unroll
    for (int e = 0; e < F * 4; e++) sums[part - 1][e][lane] = a[e];
  }
  __syncthreads();
  if (part > 0) return;
  float16v acc[F];
#pragma unroll
  for (int j = 0; j < F; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      float4 x = a[j * 4 + e];
#pragma unroll
      for (int k = 0; k < 3; k++) {
        const float4 y = sums[k][j * 4 + e][lane];
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      acc[j][4 * e] = x.x;
      acc[j][4 * e + 1] = x.y;
      acc[j][4 * e + 2] = x.z;
      acc[j][4 * e + 3] = x.w;
    }
  Tl::template finish<EPI>(g, mat, it, jt, w, i, reinterpret_cast<_Float16 *>(lds), acc);
}

// ---- small matrices ---------------------------------------------------------------------
// All steps of one matrix by one workgroup, X, X^T, A and B in LDS, padded to multiples
// of 32: a step is three short products and as many barriers instead of three launches.
// What bounds it is the length of one wave's instruction stream per product (a 32 x 32
// tile's 16 values per lane to split and store took 0.8 us), so tiles are 16 x 16 and 16
// waves share them. Symmetric results are written transposed only, four values to a
// store. A block of a factor holds 32 values of the summed axis: 32 hi, then 32 lo, 128
// bytes a row; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7), which meets no bank
// twice in a fragment read.
constexpr int SM_THREADS = 1024, SM_WAVES = SM_THREADS / WAVE;
constexpr int SM_TILES = 6;                        // 16 x 16 tiles of X per wave, at most
typedef float float4v __attribute__((ext_vector_type(4)));

struct SmallArgs {
  const void *g;
  void *out;
  int64_t gb, gr, ob, orow;
  int dtype, rows, cols, tall, m, n, mp, np, steps;
  float eps, s0;
  struct {
    float mul_a, mul_p, ca, cb, mul_x, pad[3];     // scales of A, B and X, folded in
  } step[64];
};

// Chunk `c` (hi 0 .. 3, lo 4 .. 7) of row r in block b of a factor of R rows, in halves.
__device__ __forceinline__ int small_at(int R, int b, int r, int c) { return (b * R + r) * 64 + ((c ^ ((r >> 1) & 7)) << 3); }

// 16 x 16 tile (it, jt) of P Q^T, factors of RP and RQ rows, summed over kb blocks.
__device__ __forceinline__ float4v small_product(const _Float16 *p, int RP, int it, const _Float16 *q, int RQ, int jt,
                                                 int kb, int lane) {
  const int fr = lane & 15, fk = lane >> 4, ri = it * 16 + fr, rj = jt * 16 + fr;
  float4v acc = {0.0f, 0.0f, 0.0f, 0.0f}, cross = acc;
#pragma unroll 1
  for (int b = 0; b < kb; b++) {
    const half8 pl = *reinterpret_cast<const half8 *>(p + small_at(RP, b, ri, fk + 4));
    const half8 qh = *reinterpret_cast<const half8 *>(q + small_at(RQ, b, rj, fk));
    const half8 ph = *reinterpret_cast<const half8 *>(p + small_at(RP, b, ri, fk));
    const half8 ql = *reinterpret_cast<const half8 *>(q + small_at(RQ, b, rj, fk + 4));
    cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, ql, cross, 0, 0, 0);
    cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh, cross, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh, acc, 0, 0, 0);
    cross = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql, cross, 0, 0, 0);
  }
  return acc + cross;
}

// Writes v as element k of row r of a factor of R rows.
__device__ __forceinline__ void small_put(_Float16 *d, int R, int r, int k, float v) {
  const int at = k & 7, c = (k >> 3) & 3;
  const _Float16 hi = (_Float16)v;
  d[small_at(R, k >> 5, r, c) + at] = hi;
  d[small_at(R, k >> 5, r, c + 4) + at] = (_Float16)(v - (float)hi);
}
// Four consecutive elements from k, a multiple of four.
__device__ __forceinline__ void small_put4(_Float16 *d, int R, int r, int k, float4v v) {
  const int at = k & 7, c = (k >> 3) & 3;
  half4 hi, lo;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    hi[e] = (_Float16)v[e];
    lo[e] = (_Float16)(v[e] - (float)hi[e]);
  }
  *reinterpret_cast<half4 *>(d + small_at(R, k >> 5, r, c) + at) = hi;
  *reinterpret_cast<half4 *>(d + small_at(R, k >> 5, r, c + 4) + at) = lo;
}

template <int LDS_BYTES>
__global__ __launch_bounds__(SM_THREADS) void k_ortho_small(SmallArgs o) {
  constexpr int SUMS = SM_WAVES * sizeof(double);
  __shared__ __align__(16) char lds[LDS_BYTES];
  double *sums = reinterpret_cast<double *>(lds);
  float *result = reinterpret_cast<float *>(lds + SUMS);   // in X's and X^T's place at the end, rows padded by one
  _Float16 *x = reinterpret_cast<_Float16 *>(lds + SUMS), *y = x + 2 * o.mp * o.np, *a = y + 2 * o.mp * o.np,
           *b = a + 2 * o.mp * o.mp;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63;
  const int64_t mat = blockIdx.x;
  const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
  const int count = o.rows * o.cols;
  double t = 0.0;
  for (int i = tid; i < count; i += SM_THREADS) {
    const int r = i / o.cols, c = i - r * o.cols;
    const double v = (double)read_as_f32(g, r * o.gr + c, o.dtype);
    t = __builtin_fma(v, v, t);
  }
  t = wave_sum_f64(t);
  if (lane == 0) sums[w] = t;
  __syncthreads();
  double all = 0.0;
#pragma unroll
  for (int k = 0; k < SM_WAVES; k++) all += sums[k];
  float pre, inv;
  unit_scale(all, o.eps, o.s0, pre, inv);
  for (int i = tid; i < o.mp * o.np; i += SM_THREADS) {
    const int r = i / o.np, c = i - r * o.np;     // of X
    float v = 0.0f;
    if (r < o.m && c < o.n) v = read_as_f32(g, o.tall ? c * o.gr + r : r * o.gr + c, o.dtype) * pre * inv;
    small_put(x, o.mp, r, c, v);
    small_put(y, o.np, c, r, v);
  }
  __syncthreads();
  const int tm = o.mp / 16, tn = o.np / 16;
  // k / tm for k below 6 x 16 tiles, exactly: tm is at most 9
  const int recip = (65536 + tm - 1) / tm;
  auto div_tm = [&](int k) { return (k * recip) >> 16; };
  for (int s = 0; s < o.steps; s++) {
    const auto st = o.step[s];
    // the lane as a new value in each step: addresses made from it are formed where they
    // are used, not kept (and spilled) across steps
    asm volatile("" : "+v"(lane));
    const int fr = lane & 15, fk = lane >> 4;
#pragma unroll 1
    for (int k = w; k < tm * tm; k += SM_WAVES) {  // A
      const int it = div_tm(k), jt = k - it * tm;
      const float4v v = small_product(x, o.mp, it, x, o.mp, jt, o.np / 32, lane);
      small_put4(a, o.mp, jt * 16 + fr, it * 16 + fk * 4, v * st.mul_a);
    }
    __syncthreads();
#pragma unroll 1
    for (int k = w; k < tm * tm; k += SM_WAVES) {  // B = a I + b A + c A A
      const int it = div_tm(k), jt = k - it * tm, J = jt * 16 + fr, I0 = it * 16 + fk * 4;
      const int at = I0 & 7, c = (I0 >> 3) & 3;
      const half4 hi = *reinterpret_cast<const half4 *>(a + small_at(o.mp, I0 >> 5, J, c) + at);
      const half4 lo = *reinterpret_cast<const half4 *>(a + small_at(o.mp, I0 >> 5, J, c + 4) + at);
      float4v v = small_product(a, o.mp, it, a, o.mp, jt, o.mp / 32, lane);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[e] = __builtin_fmaf(st.cb, (float)hi[e] + (float)lo[e], v[e] * st.mul_p);
        if (I0 + e == J) v[e] += st.ca;
      }
      small_put4(b, o.mp, J, I0, v);
    }
    __syncthreads();
    // X <- B X: X^T is read by every wave, so the results wait in registers
    float4v acc[SM_TILES];
#pragma unroll
    for (int u = 0; u < SM_TILES; u++) {
      const int k = w + u * SM_WAVES;
      if (k < tm * tn) acc[u] = small_product(b, o.mp, k - div_tm(k) * tm, y, o.np, div_tm(k), o.mp / 32, lane);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < SM_TILES; u++) {
      const int k = w + u * SM_WAVES;
      if (k < tm * tn) {
        const int jt = div_tm(k), I0 = (k - jt * tm) * 16 + fk * 4, J = jt * 16 + fr;
        const float4v v = acc[u] * st.mul_x;
        if (s + 1 < o.steps) {
          small_put4(y, o.np, J, I0, v);
#pragma unroll
          for (int e = 0; e < 4; e++) small_put(x, o.mp, I0 + e, J, v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++) result[o.tall ? J * (o.mp + 1) + I0 + e : (I0 + e) * (o.np + 1) + J] = v[e];
        }
      }
    }
    __syncthreads();
  }
  const int ld = (o.tall ? o.mp : o.np) + 1;
  for (int i = tid; i < count; i += SM_THREADS) {
    const int r = i / o.cols, c = i - r * o.cols;
    write_from_f32(o.out, mat * o.ob + r * o.orow + c, o.dtype, result[r * ld + c]);
  }
}

// ---- narrow matrices --------------------------------------------------------------------
// Few rows (at most 96) and a long axis: one launch per step instead of three. A
// workgroup keeps `ns` columns of X; in a step it adds the slices' shares of X X^T, which
// is small, forms B by itself, multiplies its own columns and leaves their share of the
// next X X^T. Shares alternate between two places, since other workgroups may still read
// the last ones. X^T of a slice passes from launch to launch as the image LDS holds.
constexpr int NW_ROWS = 96;                        // LDS: X, X^T (64 or 128 columns), A, B, 4 bytes a value
constexpr int NW_TILES = 2;                        // 16 x 16 tiles of a slice per wave, at most
constexpr int NW_LDS = 128 << 10;

struct NarrowArgs {
  const void *g;
  void *out;
  int64_t gb, gr, ob, orow;
  int dtype, rows, cols, tall, m, n, mp, ns, slices, last, norm_blocks;
  float eps, s0, mul_a, mul_p, ca, cb, mul_x;
  const double *norms;
  _Float16 *image;                                 // [batch][slices][2 ns mp]
  const float4 *from;                              // [batch][slices][tiles][lanes]: shares of X X^T
  float4 *to;
};

template <bool FIRST>
__global__ __launch_bounds__(SM_THREADS) void k_ortho_narrow(NarrowArgs o) {
  __shared__ __align__(16) char lds[NW_LDS];
  _Float16 *x = reinterpret_cast<_Float16 *>(lds), *y = x + 2 * o.mp * o.ns, *a = y + 2 * o.mp * o.ns,
           *b = a + 2 * o.mp * o.mp;
  float *result = reinterpret_cast<float *>(lds);  // in X's and X^T's place at the end
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, fk = lane >> 4;
  const int64_t mat = blockIdx.y;
  const int j0 = blockIdx.x * o.ns, tm = o.mp / 16, tn = o.ns / 16, mm = tm * tm;
  const int64_t slice = mat * o.slices + blockIdx.x;
  half8 *image = reinterpret_cast<half8 *>(o.image + slice * 2 * o.mp * o.ns);
  const int chunks = o.mp * o.ns / 4;              // of 16 bytes in a slice's image
  if constexpr (FIRST) {
    double *sums = reinterpret_cast<double *>(b);
    double t = 0.0;
    for (int k = tid; k < o.norm_blocks; k += SM_THREADS) t += o.norms[mat * NORM_BLOCKS + k];
    t = wave_sum_f64(t);
    if (lane == 0) sums[w] = t;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int k = 0; k < SM_WAVES; k++) all += sums[k];
    float pre, inv;
    unit_scale(all, o.eps, o.s0, pre, inv);
    const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
    const int fast = o.tall ? o.mp : o.ns;         // the axis that memory holds side by side
    for (int i = tid; i < o.mp * o.ns; i += SM_THREADS) {
      const int q = i / fast, f = i - q * fast, r = o.tall ? f : q, c = o.tall ? q : f;
      float v = 0.0f;
      if (r < o.m && j0 + c < o.n)
        v = read_as_f32(g, o.tall ? (j0 + c) * o.gr + r : r * o.gr + j0 + c, o.dtype) * pre * inv;
      small_put(x, o.mp, r, c, v);
      small_put(y, o.ns, c, r, v);
    }
    __syncthreads();
  } else {
    for (int i = tid; i < chunks; i += SM_THREADS) reinterpret_cast<half8 *>(y)[i] = image[i];
    // A: the slices' shares, first to last
    for (int k = w; k < mm; k += SM_WAVES) {
      const int it = k / tm, jt = k - it * tm;
      const float4 *f = o.from + ((mat * o.slices) * mm + k) * WAVE + lane;
      float4v v = {0.0f, 0.0f, 0.0f, 0.0f};
      int s = 0;
      for (; s + 8 <= o.slices; s += 8) {
        float4 t[8];
#pragma unroll
        for (int u = 0; u < 8; u++) t[u] = f[(int64_t)(s + u) * mm * WAVE];
#pragma unroll
        for (int u = 0; u < 8; u++) v += float4v{t[u].x, t[u].y, t[u].z, t[u].w};
      }
      for (; s < o.slices; s++) {
        const float4 t = f[(int64_t)s * mm * WAVE];
        v += float4v{t.x, t.y, t.z, t.w};
      }
      small_put4(a, o.mp, jt * 16 + fr, it * 16 + fk * 4, v * o.mul_a);
    }
    __syncthreads();
    for (int k = w; k < mm; k += SM_WAVES) {       // B = a I + b A + c A A
      const int it = k / tm, jt = k - it * tm, J = jt * 16 + fr, I0 = it * 16 + fk * 4, at = I0 & 7, c = (I0 >> 3) & 3;
      const half4 hi = *reinterpret_cast<const half4 *>(a + small_at(o.mp, I0 >> 5, J, c) + at);
      const half4 lo = *reinterpret_cast<const half4 *>(a + small_at(o.mp, I0 >> 5, J, c + 4) + at);
      float4v v = small_product(a, o.mp, it, a, o.mp, jt, o.mp / 32, lane);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[e] = __builtin_fmaf(o.cb, (float)hi[e] + (float)lo[e], v[e] * o.mul_p);
        if (I0 + e == J) v[e] += o.ca;
      }
      small_put4(b, o.mp, J, I0, v);
    }
    __syncthreads();
    float4v acc[NW_TILES];                         // X <- B X, held until X^T has been read
#pragma unroll
    for (int u = 0; u < NW_TILES; u++) {
      const int k = w + u * SM_WAVES;
      if (k < tm * tn) acc[u] = small_product(b, o.mp, k % tm, y, o.ns, k / tm, o.mp / 32, lane) * o.mul_x;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NW_TILES; u++) {
      const int k = w + u * SM_WAVES;
      if (k < tm * tn) {
        const int I0 = k % tm * 16 + fk * 4, J = k / tm * 16 + fr;
        if (!o.last) {
          small_put4(y, o.ns, J, I0, acc[u]);
#pragma unroll
          for (int e = 0; e < 4; e++) small_put(x, o.mp, I0 + e, J, acc[u][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++) result[o.tall ? J * (o.mp + 1) + I0 + e : (I0 + e) * (o.ns + 1) + J] = acc[u][e];
        }
      }
    }
    __syncthreads();
  }
  if (FIRST || !o.last) {
    for (int i = tid; i < chunks; i += SM_THREADS) image[i] = reinterpret_cast<const half8 *>(y)[i];
    for (int k = w; k < mm; k += SM_WAVES) {
      const int it = k / tm;
      const float4v v = small_product(x, o.mp, it, x, o.mp, k - it * tm, o.ns / 32, lane);
      o.to[(slice * mm + k) * WAVE + lane] = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
    const int fast = o.tall ? o.m : (o.n - j0 < o.ns ? o.n - j0 : o.ns), slow = o.tall ? (o.n - j0 < o.ns ? o.n - j0 : o.ns) : o.m;
    const int ld = (o.tall ? o.mp : o.ns) + 1;
    for (int i = tid; i < fast * slow; i += SM_THREADS) {
      const int q = i / fast, f = i - q * fast;
      const int64_t at = o.tall ? (int64_t)(j0 + q) * o.orow + f : q * o.orow + j0 + f;
      write_from_f32(o.out, mat * o.ob + at, o.dtype, result[q * ld + f]);
    }
  }
}

// ---- host -----------------------------------------------------------------------------
// Largest |a x + b x^3 + c x^5| for 0 <= x <= u.
double sup_quintic(double a, double b, double c, double u) {
  auto f = [&](double x) { return fabs(x * (a + x * x * (b + c * x * x))); };
  double best = f(u);
  // stationary points: a + 3 b s + 5 c s^2 = 0 in s = x^2
  double r[2];
  int k = 0;
  const double A = 5 * c, B = 3 * b, D = B * B - 4 * A * a;
  if (A == 0.0) {
    if (B != 0.0) r[k++] = -a / B;
  } else if (D >= 0.0) {
    r[k++] = (-B + sqrt(D)) / (2 * A);
    r[k++] = (-B - sqrt(D)) / (2 * A);
  }
  for (int i = 0; i < k; i++)
    if (r[i] > 0.0 && r[i] < u * u) best = fmax(best, f(sqrt(r[i])));
  return best;
}

// Largest |a + b s + c s^2| for 0 <= s <= t.
double sup_quadratic(double a, double b, double c, double t) {
  auto f = [&](double s) { return fabs(a + s * (b + c * s)); };
  double best = fmax(f(0.0), f(t));
  if (c != 0.0 && -b / (2 * c) > 0.0 && -b / (2 * c) < t) best = fmax(best, f(-b / (2 * c)));
  return best;
}

// Exponent of the largest power of two S with 1.02 bound S within fp16's range.
int scale_exp(double bound) {
  if (bound < 1e-6) bound = 1e-6;
  int e;
  frexp(65504.0 / (1.02 * bound), &e);
  return e - 1;
}

constexpr int GROUPS = 512;               // workgroups that the chip holds at once, two per CU

int64_t lower_tiles(int len, int tl) { return (int64_t)(len / tl) * (len / tl + 1) / 2; }

int round_up(int x, int k) { return (x + k - 1) / k * k; }

// LDS bytes of the one-workgroup form; 0 if the matrix is too large for it. It is taken
// wherever it fits. us in this form, in the narrow one and in 3 launches a step: 32 x 32 13,
// 29, 59; 32 x 200 24, 32, 68; 64 x 64 22, 37, 59; 64 x 128 32, 39, 63; 64 x 192 42, 41, 66;
// 96 x 96 44, 58, 70; eight of 64 x 192 42, 43, 69; 300 of 96 x 96 93 and 270 (too many
// workgroups for the narrow form). The loss is on few rows and a long axis: 32 x 500 45, 31,
// 78, eight of them 45, 32, 83.
constexpr int SMALL_LDS = 64 << 10, LARGE_LDS = 160 << 10;
int small_lds(int rows, int cols) {
  const int64_t m = round_up(rows < cols ? rows : cols, 32), n = round_up(rows < cols ? cols : rows, 32);
  const int64_t bytes = 8 * SM_WAVES + 4 * (2 * m * n + 2 * m * m);
  return (m / 16) * (n / 16) <= SM_TILES * SM_WAVES && bytes <= LARGE_LDS ? (int)bytes : 0;
}

// Whether a symmetric product's tiles are shared out over all workgroups: few tiles with
// long sums, since the second launch and the pieces' traffic have to be won back. Whole
// calls with and without, us: 64 x 8192 105 and 376, 64 x 1024 87 and 97, 300 x 1024 124 and
// 130, 777 x 1000 203 and 165, 777 x 2048 237 and 239 (all 64 x 64 tiles); 512 x 8192 311 and
// 489, 1024 x 8192 702 and 1252, 2048 x 4096 1197 and 1221 (128 x 128).
bool share_out(int64_t tiles, int tl, int K) {
  return tiles < GROUPS && (tl == 128 ? K >= 512 : K >= 1024 && K >= 22 * tiles);
}

// Columns per workgroup of the narrow form; 0 where three launches a step are faster. Whole
// calls in this form and in that, us: 9 x 1000 32 and 86, 64 x 300 44 and 72, 64 x 1024 48
// and 88, 64 x 8192 93 and 105, eight of 64 x 1024 61 and 96, 96 x 1024 80 and 95; but 96 x
// 4096 158 and 111 (every workgroup adds up every slice's 36 KB), and 64 of 64 x 512 132
// and 120 (more workgroups than CUs).
int narrow_cols(int64_t batch, int rows, int cols) {
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (m > NW_ROWS || n > (m <= 64 ? 8192 : 1536)) return 0;
  const int ns = n > 2048 ? 128 : 64;
  return batch * ((n + ns - 1) / ns) <= 256 ? ns : 0;
}

struct NarrowLayout {
  int mp, ns, slices;
  double *norms;
  _Float16 *image;
  float4 *part[2];
  size_t bytes;
};

NarrowLayout narrow_layout(void *base, int64_t batch, int rows, int cols) {
  NarrowLayout L;
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  L.mp = round_up(m, 32);
  L.ns = narrow_cols(batch, rows, cols);
  L.slices = (n + L.ns - 1) / L.ns;
  char *p = (char *)base;
  auto take = [&](size_t b) {
    char *q = p;
    p += ws_align(b);
    return q;
  };
  const size_t all = (size_t)batch * L.slices;
  L.norms = (double *)take(sizeof(double) * NORM_BLOCKS * (size_t)batch);
  L.image = (_Float16 *)take(4 * all * L.mp * L.ns);
  for (int k = 0; k < 2; k++) L.part[k] = (float4 *)take(4 * all * L.mp * L.mp);
  L.bytes = (size_t)(p - (char *)base);
  return L;
}

OrthoArgs ortho_layout(void *base, int64_t batch, int rows, int cols, size_t *bytes) {
  OrthoArgs o = {};
  o.rows = rows;
  o.cols = cols;
  o.tall = rows > cols;
  o.m = o.tall ? cols : rows;
  o.n = o.tall ? rows : cols;
  // 128 x 128 tiles move half the bytes per product of 64 x 64 ones, which serve where
  // they would leave CUs without work. Whole calls with 64 and 128, us: 777 x 1000 167 and
  // 307, 1500 x 1500 443 and 525, 1024 x 4096 429 and 469, 2048 x 2048 848 and 809, 2048 x
  // 4096 1376 and 1194.
  o.tile = (int64_t)(round_up(o.m, 128) / 128) * (round_up(o.n, 128) / 128) * batch >= GROUPS ? 128 : 64;
  o.mp = round_up(o.m, o.tile);
  o.np = round_up(o.n, o.tile);
  o.sx = 2 * (int64_t)o.mp * o.np;
  o.sa = 2 * (int64_t)o.mp * o.mp;
  char *p = (char *)base;
  auto take = [&](size_t b) {
    char *q = p;
    p += ws_align(b);
    return q;
  };
  o.norms = (double *)take(sizeof(double) * NORM_BLOCKS * (size_t)batch);
  o.x = (_Float16 *)take(2 * (size_t)o.sx * batch);
  o.y = (_Float16 *)take(2 * (size_t)o.sx * batch);
  o.y2 = (_Float16 *)take(2 * (size_t)o.sx * batch);
  o.a = (_Float16 *)take(2 * (size_t)o.sa * batch);
  o.b = (_Float16 *)take(2 * (size_t)o.sa * batch);
  const int64_t lower = lower_tiles(o.mp, o.tile) * batch;
  const size_t pieces = share_out(lower, o.tile, o.np) || share_out(lower, o.tile, o.mp) ? (size_t)(lower + GROUPS) : 0;
  o.part = (float *)take(sizeof(float) * o.tile * o.tile * pieces);
  *bytes = (size_t)(p - (char *)base);
  return o;
}

// One product over the padded sizes I x J.
template <int EPI, int TL, int SUB, int NST>
int run_tiles(GemmArgs q, int I, int J, int64_t batch, hipStream_t stream) {
  constexpr bool sym = EPI == EPI_GRAM || EPI == EPI_POLY;
  q.ti = I / TL;
  const int64_t tiles = sym ? lower_tiles(I, TL) : (int64_t)(I / TL) * (J / TL);
  if constexpr (sym) {
    if (share_out(tiles * batch, TL, q.K)) {
      q.tiles = (int)tiles;
      q.units = tiles * batch * (q.K / (KB * SUB) / 2);
      const int64_t most = q.units / 4;              // at least eight steps each
      const int groups = (int)(most < GROUPS ? most : GROUPS);
      hipLaunchKernelGGL((k_ortho_pieces<TL, SUB, NST>), dim3(groups), dim3(OR_THREADS), 0, stream, q);
      SPLAT_LAUNCH_CHECK();
      hipLaunchKernelGGL((k_ortho_join<EPI, TL, SUB, NST>), dim3((unsigned)(tiles * batch * 4 * (TL / 64))),
                         dim3(OR_THREADS), 0, stream, q, groups);
      SPLAT_LAUNCH_CHECK();
      return SPLAT_OK;
    }
  }
  hipLaunchKernelGGL((k_ortho_gemm<EPI, TL, SUB, NST>), dim3((unsigned)tiles, (unsigned)batch), dim3(OR_THREADS), 0,
                     stream, q);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <int EPI>
int run_gemm(const GemmArgs &q, int tile, int I, int J, int64_t batch, hipStream_t stream) {
  return tile == 128 ? run_tiles<EPI, 128, 1, 5>(q, I, J, batch, stream) : run_tiles<EPI, 64, 2, 4>(q, I, J, batch, stream);
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int rows, int cols) {
  if (small_lds(rows, cols)) return 0;
  if (narrow_cols(batch, rows, cols)) return narrow_layout(nullptr, batch, rows, cols).bytes;
  size_t bytes = 0;
  ortho_layout(nullptr, batch, rows, cols, &bytes);
  return bytes;
}

namespace {

// Partial sums of squares of every matrix into o.norms; *blocks per matrix.
int run_norm(const OrthoArgs &o, int64_t batch, int *blocks, hipStream_t stream) {
  const int64_t pieces = (int64_t)o.rows * ((o.cols + 8 * OR_THREADS - 1) / (8 * OR_THREADS));
  *blocks = pieces < NORM_BLOCKS ? (int)pieces : NORM_BLOCKS;
  hipLaunchKernelGGL(k_ortho_norm, dim3(*blocks, (unsigned)batch), dim3(OR_THREADS), 0, stream, o);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

}  // namespace

// Whether every step's singular values stay within a range that the scales can serve.
int orthogonalize_bounds(int steps, float a, float b, float c) {
  double u = 1.0;
  for (int k = 0; k < steps; k++) {
    const double p = sup_quadratic(a, b, c, u * u);
    u = sup_quintic(a, b, c, u);
    if (!(u <= 1e4) || !(p <= 1e4)) return SPLAT_ERR_UNSUPPORTED;
  }
  return SPLAT_OK;
}

int launch_orthogonalize(const void *g, int dtype, int64_t batch, int rows, int cols, int64_t gb, int64_t gr,
                         int steps, float ca, float cb, float cc, float eps, float scale, void *out, int64_t ob,
                         int64_t orow, void *ws, hipStream_t stream) {
  if (batch == 0 || rows == 0 || cols == 0) return SPLAT_OK;
  if (const int lds = small_lds(rows, cols)) {
    SmallArgs o = {};
    o.g = g;
    o.out = out;
    o.gb = gb;
    o.gr = gr;
    o.ob = ob;
    o.orow = orow;
    o.dtype = dtype;
    o.rows = rows;
    o.cols = cols;
    o.tall = rows > cols;
    o.m = o.tall ? cols : rows;
    o.n = o.tall ? rows : cols;
    o.mp = round_up(o.m, 32);
    o.np = round_up(o.n, 32);
    o.steps = steps;
    o.eps = eps;
    double u = 1.0;
    int ex = scale_exp(u);
    o.s0 = ldexpf(1.0f, ex);
    for (int k = 0; k < steps; k++) {
      const int ea = scale_exp(u * u), eb = scale_exp(sup_quadratic(ca, cb, cc, u * u));
      u = sup_quintic(ca, cb, cc, u);
      const int en = scale_exp(u);
      o.step[k].mul_a = ldexpf(1.0f, ea - 2 * ex);
      o.step[k].mul_p = ldexpf(cc, eb - 2 * ea);
      o.step[k].ca = ldexpf(ca, eb);
      o.step[k].cb = ldexpf(cb, eb - ea);
      o.step[k].mul_x = k + 1 == steps ? ldexpf(scale, -(eb + ex)) : ldexpf(1.0f, en - eb - ex);
      ex = en;
    }
    if (lds <= SMALL_LDS)
      hipLaunchKernelGGL(k_ortho_small<SMALL_LDS>, dim3((unsigned)batch), dim3(SM_THREADS), 0, stream, o);
    else
      hipLaunchKernelGGL(k_ortho_small<LARGE_LDS>, dim3((unsigned)batch), dim3(SM_THREADS), 0, stream, o);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  if (narrow_cols(batch, rows, cols)) {
    const NarrowLayout L = narrow_layout(ws, batch, rows, cols);
    OrthoArgs q = {};
    q.g = g;
    q.dtype = dtype;
    q.gb = gb;
    q.gr = gr;
    q.rows = rows;
    q.cols = cols;
    q.norms = L.norms;
    NarrowArgs o = {};
    int st = run_norm(q, batch, &o.norm_blocks, stream);
    if (st) return st;
    o.g = g;
    o.out = out;
    o.gb = gb;
    o.gr = gr;
    o.ob = ob;
    o.orow = orow;
    o.dtype = dtype;
    o.rows = rows;
    o.cols = cols;
    o.tall = rows > cols;
    o.m = o.tall ? cols : rows;
    o.n = o.tall ? rows : cols;
    o.mp = L.mp;
    o.ns = L.ns;
    o.slices = L.slices;
    o.eps = eps;
    o.norms = L.norms;
    o.image = L.image;
    double u = 1.0;
    int ex = scale_exp(u);
    o.s0 = ldexpf(1.0f, ex);
    o.to = L.part[0];
    const dim3 grid((unsigned)L.slices, (unsigned)batch);
    hipLaunchKernelGGL(k_ortho_narrow<true>, grid, dim3(SM_THREADS), 0, stream, o);
    SPLAT_LAUNCH_CHECK();
    for (int k = 0; k < steps; k++) {
      const int ea = scale_exp(u * u), eb = scale_exp(sup_quadratic(ca, cb, cc, u * u));
      u = sup_quintic(ca, cb, cc, u);
      const int en = scale_exp(u);
      o.last = k + 1 == steps;
      o.mul_a = ldexpf(1.0f, ea - 2 * ex);
      o.mul_p = ldexpf(cc, eb - 2 * ea);
      o.ca = ldexpf(ca, eb);
      o.cb = ldexpf(cb, eb - ea);
      o.mul_x = o.last ? ldexpf(scale, -(eb + ex)) : ldexpf(1.0f, en - eb - ex);
      o.from = L.part[k & 1];
      o.to = L.part[(k + 1) & 1];
      ex = en;
      hipLaunchKernelGGL(k_ortho_narrow<false>, grid, dim3(SM_THREADS), 0, stream, o);
      SPLAT_LAUNCH_CHECK();
    }
    return SPLAT_OK;
  }
  size_t bytes;
  OrthoArgs o = ortho_layout(ws, batch, rows, cols, &bytes);
  o.g = g;
  o.dtype = dtype;
  o.gb = gb;
  o.gr = gr;
  o.eps = eps;
  double u = 1.0;
  int ex = scale_exp(u);
  o.s0 = ldexpf(1.0f, ex);
  int nb, st0 = run_norm(o, batch, &nb, stream);
  if (st0) return st0;
  const int pr = o.tall ? o.np : o.mp, pc = o.tall ? o.mp : o.np;
  hipLaunchKernelGGL(k_ortho_pack, dim3(pc / 32, pr / 32, (unsigned)batch), dim3(OR_THREADS), 0, stream, o, nb);
  SPLAT_LAUNCH_CHECK();
  for (int k = 0; k < steps; k++) {
    const int ea = scale_exp(u * u), eb = scale_exp(sup_quadratic(ca, cb, cc, u * u));
    const double un = sup_quintic(ca, cb, cc, u);
    const int en = scale_exp(un);
    const bool last = k + 1 == steps;
    GemmArgs q = {};
    q.part = o.part;
    q.p = q.q = o.x;
    q.pb = q.qb = o.sx;
    q.K = o.np;
    q.mul = ldexpf(1.0f, ea - 2 * ex);
    q.d0 = q.d1 = o.a;
    q.db = o.sa;
    q.ld0 = q.ld1 = o.mp;
    int st = run_gemm<EPI_GRAM>(q, o.tile, o.mp, o.mp, batch, stream);
    if (st) return st;
    q.p = q.q = o.a;
    q.pb = q.qb = o.sa;
    q.K = o.mp;
    q.mul = ldexpf(cc, eb - 2 * ea);
    q.a = o.a;
    q.ca = ldexpf(ca, eb);
    q.cb = ldexpf(cb, eb - ea);
    q.d0 = q.d1 = o.b;
    if ((st = run_gemm<EPI_POLY>(q, o.tile, o.mp, o.mp, batch, stream))) return st;
    q.p = o.b;
    q.q = o.y;
    q.pb = o.sa;
    q.qb = o.sx;
    q.mul = last ? ldexpf(scale, -(eb + ex)) : ldexpf(1.0f, en - eb - ex);
    q.d0 = o.x;
    q.d1 = o.y2;
    q.db = o.sx;
    q.ld0 = o.np;
    q.ld1 = o.mp;
    q.out = out;
    q.ob = ob;
    q.orow = orow;
    q.dtype = dtype;
    q.tall = o.tall;
    q.m = o.m;
    q.n = o.n;
    st = last ? run_gemm<EPI_LAST>(q, o.tile, o.mp, o.np, batch, stream) : run_gemm<EPI_NEXT>(q, o.tile, o.mp, o.np, batch, stream);
    if (st) return st;
    _Float16 *t = o.y;
    o.y = o.y2;
    o.y2 = t;
    u = un;
    ex = en;
  }
  return SPLAT_OK;
}
