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
#include "linear_common.h"
#include "linear_rows.h"

namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

struct RowsArgs {
  const void *x, *w, *bias, *dy;
  void *y, *dx;
  int64_t M, xs, ys, dxs, wi, wo;    // rows; strides of x, y or dy, dx; of W along in and out
  int K, N;
  int want_x, want_w;                // want_w: dW or db
  float *part;                       // [workgroups][K + 1][N]: sums of dW, then of db
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

// Values at .. of a row of `len`, zeros beyond: any alignment.
template <typename T>
__device__ __forceinline__ word4 load_chunk(const T *row, int at, int len, bool ok) {
  constexpr int E = 16 / sizeof(T);
  word4 v = {0, 0, 0, 0};
  if (ok && at + E <= len) {
    v = *reinterpret_cast<const typename Loose<T, E>::type *>(row + at);
  } else if (ok && at < len) {
    Pack<T, E> t = __builtin_bit_cast(Pack<T, E>, v);
#pragma unroll
    for (int j = 0; j < E; j++)
      if (at + j < len) t.v[j] = row[at + j];
    v = __builtin_bit_cast(word4, t);
  }
  return v;
}

template <typename T, int KP, int NP>
struct Rows {
  static constexpr int E = 16 / sizeof(T);            // values per chunk
  static constexpr int KC = KP * 32 / (4 * E);        // chunks of a row of x per lane
  static constexpr int DC = 8 / E;                    // chunks of eight values
  static constexpr int WP = NP * 32 + 2;              // pitch of W in LDS
  static constexpr int W_BYTES = KP * 32 * WP * sizeof(T);
  // Row pitches of the tiles that are read turned around. 16-bit: a transposing read takes
  // eight rows of 32 bytes at once, which a pitch of an odd multiple of 32 bytes spreads over
  // all banks; fp32: four rows of 64 bytes, and a pitch of 64 more than a multiple of 128.
  static constexpr int XP = KP * 32 * sizeof(T) + 16 * sizeof(T), ZP = NP * 32 * sizeof(T) + 16 * sizeof(T);
  static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;   // of dz
  static constexpr int WAVE_BYTES = 32 * (XP + PARTS * ZP);
  static constexpr int SUM_BYTES = (KP * 32 * NP * 32 + NP * 32) * 4;

  // W as [in][out] in LDS, zeros beyond it.
  static __device__ __forceinline__ void stage_w(const RowsArgs &a, T *l) {
    for (int t = threadIdx.x; t < KP * 32 * NP * 32; t += LN_THREADS) {
      // neighbouring threads read neighbouring values
      const int k = a.wo == 1 ? t / (NP * 32) : t % (KP * 32), n = a.wo == 1 ? t % (NP * 32) : t / (KP * 32);
      l[k * WP + n] = k < a.K && n < a.N ? ((const T *)a.w)[k * a.wi + n * a.wo] : (T)0.0f;
    }
  }

  // Operands of z: row i of fragment t of 32 outputs p stands for output 32 p + 8 (i / 4) + 4 t + i % 4.
  static __device__ __forceinline__ void fragments(const T *l, word4 (&f)[NP][2][KC]) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int p = 0; p < NP; p++)
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int c = 0; c < KC; c++) {
          Pack<T, E> v;
#pragma unroll
          for (int e = 0; e < E; e++) v.v[e] = l[((c * 4 + g) * E + e) * WP + 32 * p + 8 * (i >> 2) + 4 * t + (i & 3)];
          f[p][t][c] = __builtin_bit_cast(word4, v);
        }
  }

  // Operands of dx, the same with inputs for outputs: eight neighbouring outputs 32 p + 8 g of
  // input row i in DC chunks.
  static __device__ __forceinline__ void fragments_t(const T *l, word4 (&f)[KP][2][NP][DC]) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int q = 0; q < KP; q++)
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
          for (int c = 0; c < DC; c++) {
            Pack<T, E> v;
#pragma unroll
            for (int e = 0; e < E; e++)
              v.v[e] = l[(32 * q + 8 * (i >> 2) + 4 * t + (i & 3)) * WP + 32 * p + 8 * g + c * E + e];
            f[q][t][p][c] = __builtin_bit_cast(word4, v);
          }
  }

  static __device__ __forceinline__ void load_x(const RowsArgs &a, int64_t base, word4 (&x)[2][KC]) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t m = base + 16 * h + i;
#pragma unroll
      for (int c = 0; c < KC; c++)
        x[h][c] = load_chunk<T>((const T *)a.x + m * a.xs, (c * 4 + g) * E, a.K, m < a.M);
    }
  }

  // Eight values of each lane's rows and outputs.
  static __device__ __forceinline__ void load_out(const void *p, int64_t stride, const RowsArgs &a, int64_t base,
                                                  word4 (&d)[2][NP][DC]) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t m = base + 16 * h + i;
#pragma unroll
      for (int q = 0; q < NP; q++)
#pragma unroll
        for (int c = 0; c < DC; c++)
          d[h][q][c] = load_chunk<T>((const T *)p + m * stride, 32 * q + 8 * g + c * E, a.N, m < a.M);
    }
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

  // Fragment of 16 columns from `col` of a tile, summed over its 32 rows: 16-bit values, lane
  // i holds column i, rows 16 h + 4 g + e. Two tiles read alike agree on the rows' order.
  static __device__ __forceinline__ word4 turned(const char *tile, int pitch, int col) {
    typedef __attribute__((address_space(3))) short4v *lds4;
    const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
    word4 v;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const char *at = tile + (16 * h + 4 * g + (j >> 2)) * pitch + (col + (j & 3) * 4) * 2;
      const uint2 w = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(short4v *)const_cast<char *>(at)));
      v[2 * h] = w.x;
      v[2 * h + 1] = w.y;
    }
    return v;
  }
};

// Orders a wave's own LDS accesses: the hardware keeps them in program order.
__device__ __forceinline__ void wave_lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

template <typename T, int KP, int NP>
__global__ __launch_bounds__(LN_THREADS) void k_rows(RowsArgs a) {
  typedef Rows<T, KP, NP> R;
  __shared__ T lw[KP * 32 * R::WP];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t step = (int64_t)gridDim.x * (LN_THREADS / WAVE) * 32;
  int64_t base = ((int64_t)blockIdx.x * (LN_THREADS / WAVE) + (threadIdx.x >> 6)) * 32;
  word4 next[2][R::KC];
  R::load_x(a, base, next);
  R::stage_w(a, lw);
  __syncthreads();
  word4 f[NP][2][R::KC];
  R::fragments(lw, f);
  float b[NP][8];
  int n[NP];
#pragma unroll
  for (int p = 0; p < NP; p++) {
    n[p] = a.N - (32 * p + 8 * g);
    n[p] = n[p] < 0 ? 0 : n[p] > 8 ? 8 : n[p];
    load_bias<T>(a.layer, 32 * p + 8 * g, n[p], b[p]);
  }
  DropKey key = {};
  if (a.layer.draw) key = drop_key(a.layer.drop);
  for (; base < a.M; base += step) {
    word4 x[2][R::KC], r[2][NP][R::DC];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int c = 0; c < R::KC; c++) x[h][c] = next[h][c];
    if (a.layer.res) R::load_out(a.layer.res, a.layer.rs, a, base, r);
    R::load_x(a, base + step, next);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t m = base + 16 * h + i;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        float v[8];
        R::product(f, x[h], p, v);
        if (m < a.M && n[p] > 0) {
          const int64_t col = 32 * p + 8 * g;
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] += b[p][j];
          if (a.layer.pre) store8<T>((T *)a.layer.pre + m * a.N + col, n[p], v);
          activate<T>(v, a.layer.act);
          if (a.layer.draw) {
            const uint32_t keep = keeps_from(m * a.N + col, a.layer.drop, key);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = keep >> j & 1 ? v[j] * a.layer.drop.scale : 0.0f;
          }
          if (a.layer.res) {
            float q[8];
            R::widen(r[h][p], q);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += q[j];
          }
          store8<T>((T *)a.y + m * a.ys + col, n[p], v);
        }
      }
    }
  }
}

// dz in one or two parts of T: two of 16-bit types hold it to 16 bits and more, where one
// would add as much error to dx and dW as their own rounding does. The second part of an
// infinity is zero.
template <typename T>
__device__ __forceinline__ void split8(const float (&d)[8], word4 &hi, word4 &lo) {
  Pack<T, 8> h, l;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    h.v[j] = (T)d[j];
    const float f = (float)h.v[j];
    l.v[j] = (T)(fabsf(f) < INFINITY ? d[j] - f : 0.0f);
  }
  hi = __builtin_bit_cast(word4, h);
  lo = __builtin_bit_cast(word4, l);
}

template <typename T, int KP, int NP>
__global__ __launch_bounds__(LN_THREADS, 2) void k_rows_bwd(RowsArgs a) {
  typedef Rows<T, KP, NP> R;
  constexpr int WAVES = LN_THREADS / WAVE;
  constexpr int A = R::W_BYTES > R::SUM_BYTES ? R::W_BYTES : R::SUM_BYTES;
  constexpr int LDS = WAVES * R::WAVE_BYTES > A ? WAVES * R::WAVE_BYTES : A;
  __shared__ __attribute__((aligned(16))) char lds[LDS];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, w = threadIdx.x >> 6;
  const int64_t step = (int64_t)gridDim.x * WAVES * 32;
  int64_t base = ((int64_t)blockIdx.x * WAVES + w) * 32;
  const bool shaped = a.layer.act != SPLAT_ACT_NONE || a.layer.draw, slope = a.layer.act != SPLAT_ACT_NONE;
  word4 nx[2][R::KC], nd[2][NP][R::DC];
  R::load_x(a, base, nx);
  R::load_out(a.dy, a.ys, a, base, nd);
  R::stage_w(a, reinterpret_cast<T *>(lds));
  __syncthreads();
  word4 f[NP][2][R::KC], ft[KP][2][NP][R::DC];
  R::fragments(reinterpret_cast<const T *>(lds), f);
  R::fragments_t(reinterpret_cast<const T *>(lds), ft);
  __syncthreads();
  char *xt = lds + w * R::WAVE_BYTES, *zt = xt + 32 * R::XP, *zt2 = zt + 32 * R::ZP;
  float b[NP][8];
  int n[NP];
#pragma unroll
  for (int p = 0; p < NP; p++) {
    n[p] = a.N - (32 * p + 8 * g);
    n[p] = n[p] < 0 ? 0 : n[p] > 8 ? 8 : n[p];
    load_bias<T>(a.layer, 32 * p + 8 * g, n[p], b[p]);
  }
  DropKey key = {};
  if (a.layer.draw) key = drop_key(a.layer.drop);
  float4v dw[2 * KP][2 * NP];
  float db[NP][8];
#pragma unroll
  for (int k = 0; k < 2 * KP; k++)
#pragma unroll
    for (int q = 0; q < 2 * NP; q++) dw[k][q] = float4v{0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < NP; p++)
#pragma unroll
    for (int j = 0; j < 8; j++) db[p][j] = 0.0f;
  for (; base < a.M; base += step) {
    word4 x[2][R::KC], dy[2][NP][R::DC];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int c = 0; c < R::KC; c++) x[h][c] = nx[h][c];
#pragma unroll
      for (int p = 0; p < NP; p++)
#pragma unroll
        for (int c = 0; c < R::DC; c++) dy[h][p][c] = nd[h][p][c];
    }
    R::load_x(a, base + step, nx);
    R::load_out(a.dy, a.ys, a, base + step, nd);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int64_t m = base + 16 * h + i;
      word4 dz[NP][R::DC], dz2[NP];
#pragma unroll
      for (int p = 0; p < NP; p++) {
        float d[8];
        R::widen(dy[h][p], d);
        if (slope) {
          float z[8];
          R::product(f, x[h], p, z);
#pragma unroll
          for (int j = 0; j < 8; j++) z[j] += b[p][j];
          slope_times<T>(d, z, a.layer.act);
        }
        if (a.layer.draw) {
          const uint32_t keep = keeps_from(m * a.N + 32 * p + 8 * g, a.layer.drop, key);
#pragma unroll
          for (int j = 0; j < 8; j++) d[j] = keep >> j & 1 ? d[j] * a.layer.drop.scale : 0.0f;
        }
        if (shaped && m >= a.M) {
#pragma unroll
          for (int j = 0; j < 8; j++) d[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) db[p][j] += d[j];
        if constexpr (sizeof(T) == 2) {
          if (shaped) split8<T>(d, dz[p][0], dz2[p]);
          else dz[p][0] = dy[h][p][0];
          *reinterpret_cast<word4 *>(zt + (16 * h + i) * R::ZP + p * 64 + g * 16) = dz[p][0];
          if (shaped) *reinterpret_cast<word4 *>(zt2 + (16 * h + i) * R::ZP + p * 64 + g * 16) = dz2[p];
        } else {
#pragma unroll
          for (int c = 0; c < R::DC; c++) {
            dz[p][c] = __builtin_bit_cast(word4, make_float4(d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]));
            *reinterpret_cast<word4 *>(zt + (16 * h + i) * R::ZP + p * 128 + g * 32 + c * 16) = dz[p][c];
          }
        }
      }
#pragma unroll
      for (int c = 0; c < R::KC; c++) *reinterpret_cast<word4 *>(xt + (16 * h + i) * R::XP + c * 64 + g * 16) = x[h][c];
      if (a.want_x) {
#pragma unroll
        for (int q = 0; q < KP; q++) {
          float4v lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
          for (int p = 0; p < NP; p++) {
#pragma unroll
            for (int c = 0; c < R::DC; c++) {
              lo = mul16<T>(ft[q][0][p][c], dz[p][c], lo);
              hi = mul16<T>(ft[q][1][p][c], dz[p][c], hi);
            }
            if constexpr (sizeof(T) == 2) {
              if (shaped) {
                lo = mul16<T>(ft[q][0][p][0], dz2[p], lo);
                hi = mul16<T>(ft[q][1][p][0], dz2[p], hi);
              }
            }
          }
          const int col = 32 * q + 8 * g, left = a.K - col;
          if (m < a.M && left > 0) {
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            store8<T>((T *)a.dx + m * a.dxs + col, left < 8 ? left : 8, v);
          }
        }
      }
    }
    if (a.want_w) {
      wave_lds_order();
      if constexpr (sizeof(T) == 2) {
        word4 xf[2 * KP];
#pragma unroll
        for (int k = 0; k < 2 * KP; k++) xf[k] = R::turned(xt, R::XP, 16 * k);
#pragma unroll
        for (int q = 0; q < 2 * NP; q++) {
          const word4 zf = R::turned(zt, R::ZP, 16 * q);
#pragma unroll
          for (int k = 0; k < 2 * KP; k++) dw[k][q] = mul16<T>(xf[k], zf, dw[k][q]);
        }
        if (shaped) {
#pragma unroll
          for (int q = 0; q < 2 * NP; q++) {
            const word4 zf = R::turned(zt2, R::ZP, 16 * q);
#pragma unroll
            for (int k = 0; k < 2 * KP; k++) dw[k][q] = mul16<T>(xf[k], zf, dw[k][q]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; s++) {
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
  }
  if (!a.want_w) return;
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

// The workgroups' sums in order: 32 values by 32 slices of the workgroups per workgroup.
template <typename T>
__global__ __launch_bounds__(1024) void k_rows_join(const float *part, int groups, int K, int N, T *dw, int64_t di, int64_t dn,
                                                    void *db, int f32) {
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
    if (dw) dw[k * di + n * dn] = (T)v;
  } else if (db) {
    if (f32) ((float *)db)[n] = v;
    else ((T *)db)[n] = (T)v;
  }
}

template <typename T>
int run_rows(const RowsArgs &a, bool bwd, int groups, hipStream_t s) {
  const dim3 grid((unsigned)groups), block(LN_THREADS);
  const int kp = a.K > 32 ? 2 : 1, np = a.N > 32 ? 2 : 1;
#define ROWS(KP, NP)                                                                  \
  if (kp == KP && np == NP) {                                                         \
    if (bwd) hipLaunchKernelGGL((k_rows_bwd<T, KP, NP>), grid, block, 0, s, a);       \
    else hipLaunchKernelGGL((k_rows<T, KP, NP>), grid, block, 0, s, a);               \
  }
  ROWS(1, 1)
  ROWS(1, 2)
  ROWS(2, 1)
  ROWS(2, 2)
#undef ROWS
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

int by_type(const RowsArgs &a, int dtype, bool bwd, int groups, hipStream_t s) {
  if (dtype == SPLAT_F32) return run_rows<float>(a, bwd, groups, s);
  if (dtype == SPLAT_F16) return run_rows<f16_t>(a, bwd, groups, s);
  return run_rows<bf16_t>(a, bwd, groups, s);
}

int groups_for(int64_t M, int most) {
  const int64_t g = (M + 127) / 128;                  // four waves of 32 rows
  return (int)(g < most ? g : most);
}
constexpr int FWD_GROUPS = 2048, BWD_GROUPS = 512;

RowsArgs rows_args(const splat_dense *d, const void *x, const void *w) {
  RowsArgs a = {};
  a.x = x;
  a.w = w;
  a.M = d->rows;
  a.K = d->in;
  a.N = d->out;
  a.xs = d->x_stride;
  a.ys = d->y_stride;
  a.dxs = d->dx_stride;
  a.wi = d->w_in_stride;
  a.wo = d->w_out_stride;
  return a;
}

}  // namespace

bool linear_by_rows(const splat_dense *d) { return d->in >= 1 && d->in <= 64 && d->out <= 64; }

size_t linear_rows_workspace_bytes(const splat_dense *d) {
  return ws_align(sizeof(float) * (size_t)groups_for(d->rows, BWD_GROUPS) * (d->in + 1) * d->out);
}

int launch_linear_rows(const splat_dense *d, const void *x, const void *w, const LayerArgs &l, void *y, hipStream_t stream) {
  RowsArgs a = rows_args(d, x, w);
  a.y = y;
  a.layer = l;
  return by_type(a, d->dtype, false, groups_for(a.M, FWD_GROUPS), stream);
}

int launch_linear_rows_bwd(const splat_dense *d, const void *dy, const void *x, const void *w, const LayerArgs &l, void *dx,
                           void *dw, void *db, void *ws, hipStream_t stream) {
  RowsArgs a = rows_args(d, x, w);
  a.dy = dy;
  a.dx = dx;
  a.layer = l;
  a.want_x = dx != nullptr;
  a.want_w = dw || db;
  a.part = (float *)ws;
  const int groups = groups_for(a.M, BWD_GROUPS);
  int st = by_type(a, d->dtype, true, groups, stream);
  if (st || !a.want_w) return st;
  const dim3 grid((unsigned)(((a.K + 1) * a.N + 31) / 32)), block(1024);
  const int f32 = d->bias_dtype == SPLAT_F32;
  const int64_t di = d->dw_in_stride, dn = d->dw_out_stride;
  if (d->dtype == SPLAT_F32)
    hipLaunchKernelGGL(k_rows_join<float>, grid, block, 0, stream, a.part, groups, a.K, a.N, (float *)dw, di, dn, db, f32);
  else if (d->dtype == SPLAT_F16)
    hipLaunchKernelGGL(k_rows_join<f16_t>, grid, block, 0, stream, a.part, groups, a.K, a.N, (f16_t *)dw, di, dn, db, f32);
  else
    hipLaunchKernelGGL(k_rows_join<bf16_t>, grid, block, 0, stream, a.part, groups, a.K, a.N, (bf16_t *)dw, di, dn, db, f32);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}
