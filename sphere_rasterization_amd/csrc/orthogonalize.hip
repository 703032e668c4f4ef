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
// hi hi + hi lo + lo hi on the matrix cores with fp32 sums: the dropped lo lo is below
// 2^-23 of the product. Three fp16 products still run several times faster than one
// in fp32, whose matrix rate on gfx950 is 1/16 of fp16's.
//
// Layout. A factor is stored by rows along the summed axis in blocks of 32 values:
// 32 hi then 32 lo, 128 bytes, one cache line per row and block, so that a tile's
// step is whole lines and the two parts travel together. X is kept both by rows and
// transposed, because X X^T sums over columns and B X over rows.
#include <math.h>

#include "learn_common.h"

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int KB = 32;                 // values per block of the summed axis
constexpr int PAD = 128;               // matrices are padded to multiples of the tile
constexpr int TM = 128, TN = 128;      // tile of one workgroup: four waves of 64 x 64
constexpr int OR_THREADS = 256;
constexpr int NORM_BLOCKS = 256;

enum { EPI_GRAM, EPI_POLY, EPI_NEXT, EPI_LAST };

struct OrthoArgs {
  const void *g;
  void *out;
  int64_t gb, gr, ob, orow;            // batch and row strides of the input and the output
  int dtype, rows, cols, tall;
  int m, n, mp, np;                    // m <= n and their padded sizes
  double *norms;                       // [batch][NORM_BLOCKS] partial sums of squares
  _Float16 *x, *y, *y2, *a, *b;        // packed factors: X, X^T (two), A, B; per matrix strides below
  int64_t sx, sa;                      // halves per matrix of x / y, and of a / b
  float eps, s0;                       // s0: scale of X before the first step
};

struct GemmArgs {
  const _Float16 *p, *q;               // factors by rows [I][K], [J][K], packed
  int64_t pb, qb;                      // halves per matrix
  int K;                               // padded length of the summed axis
  int ti, tj;                          // tiles per side
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

// Place of value k in a packed row: block k / 32, hi part first.
__device__ __forceinline__ int packed(int k) { return (k >> 5) * (2 * KB) + (k & 31); }

// Sums of squares in fp64: no square over- or underflows and the norm is exact to fp32.
__global__ __launch_bounds__(OR_THREADS) void k_ortho_norm(OrthoArgs o) {
  __shared__ double s[OR_THREADS / WAVE];
  const int64_t mat = blockIdx.y;
  const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
  double t = 0.0;
  for (int r = blockIdx.x; r < o.rows; r += gridDim.x)
    for (int c = threadIdx.x; c < o.cols; c += OR_THREADS) {
      const double v = (double)read_as_f32(g, r * o.gr + c, o.dtype);
      t = __builtin_fma(v, v, t);
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
  if ((int)threadIdx.x < norm_blocks) q = o.norms[mat * NORM_BLOCKS + threadIdx.x];
  q = wave_sum_f64(q);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = q;
  __syncthreads();
  const float inv = (float)((double)o.s0 / (sqrt((s[0] + s[1]) + (s[2] + s[3])) + (double)o.eps));
  const char *g = (const char *)o.g + mat * o.gb * (o.dtype == SPLAT_F32 ? 4 : 2);
  // direct image: rows of G; cross image: its columns
  _Float16 *direct = (o.tall ? o.y : o.x) + mat * o.sx, *cross = (o.tall ? o.x : o.y) + mat * o.sx;
  const int dlen = o.tall ? o.mp : o.np, clen = o.tall ? o.np : o.mp;
  const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int r = r0 + ty + k, c = c0 + tx;
    const float v = r < o.rows && c < o.cols ? read_as_f32(g, r * o.gr + c, o.dtype) * inv : 0.0f;
    t[ty + k][tx] = v;
    const _Float16 hi = (_Float16)v;
    _Float16 *d = direct + (int64_t)r * 2 * dlen + packed(c);
    d[0] = hi;
    d[KB] = (_Float16)(v - (float)hi);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int r = r0 + tx, c = c0 + ty + k;
    const float v = t[tx][ty + k];
    const _Float16 hi = (_Float16)v;
    _Float16 *d = cross + (int64_t)c * 2 * clen + packed(r);
    d[0] = hi;
    d[KB] = (_Float16)(v - (float)hi);
  }
}

// One 128 x 128 tile of D = P Q^T. A step of 32 along K brings 256 rows of 128 bytes
// into LDS; the 16-byte chunk c of row r lies at c ^ (r & 7), so that the eight rows a
// fragment read touches at a time fall on different banks.
template <int EPI>
__global__ __launch_bounds__(OR_THREADS, 2) void k_ortho_gemm(GemmArgs g) {
  __shared__ half8 lds[2][(TM + TN) * 8];
  const int64_t mat = blockIdx.y;
  int it, jt;
  if constexpr (EPI == EPI_GRAM || EPI == EPI_POLY) {
    // tile t of the lower triangle
    const int t = blockIdx.x;
    it = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((it + 1) * (it + 2) / 2 <= t) it++;
    while (it * (it + 1) / 2 > t) it--;
    jt = t - it * (it + 1) / 2;
  } else {
    it = blockIdx.x % g.ti;
    jt = blockIdx.x / g.ti;
  }
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int wi = (w & 1) * 64, wj = (w >> 1) * 64;
  // this thread's chunks of a step: rows r0 + 32 k, chunk tid & 7
  const int lr = tid >> 3, lc = tid & 7;
  const int64_t row = 2 * (int64_t)g.K;
  const _Float16 *p = g.p + mat * g.pb + ((int64_t)it * TM + lr) * row + lc * 8;
  const _Float16 *q = g.q + mat * g.qb + ((int64_t)jt * TN + lr) * row + lc * 8;
  half8 st[8];
  auto fetch = [&](int k) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
      st[u] = *reinterpret_cast<const half8 *>(p + (int64_t)u * 32 * row + k * (2 * KB));
      st[4 + u] = *reinterpret_cast<const half8 *>(q + (int64_t)u * 32 * row + k * (2 * KB));
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < 8; u++) {
      const int r = lr + u * 32;
      lds[buf][r * 8 + (lc ^ (r & 7))] = st[u];
    }
  };
  float16v acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
  const int steps = g.K / KB;
  const int fr = lane & 31, fk = lane >> 5;
  fetch(0);
  stage(0);
  __syncthreads();
  for (int k = 0; k < steps; k++) {
    if (k + 1 < steps) fetch(k + 1);
    const half8 *l = lds[k & 1];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      half8 ph[2], pl[2], qh[2], ql[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int r = wi + i * 32 + fr, c = h * 2 + fk;
        ph[i] = l[r * 8 + (c ^ (r & 7))];
        pl[i] = l[r * 8 + ((c + 4) ^ (r & 7))];
        const int s = TM + wj + i * 32 + fr;
        qh[i] = l[s * 8 + (c ^ (s & 7))];
        ql[i] = l[s * 8 + ((c + 4) ^ (s & 7))];
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[i], qh[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[i], ql[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[i], qh[j], acc[i][j], 0, 0, 0);
        }
    }
    if (k + 1 < steps) stage((k + 1) & 1);
    __syncthreads();
  }
  // a lane holds column fr and rows 8 (e / 4) + 4 (lane / 32) + e % 4 of each 32 x 32
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int J = jt * TN + wj + j * 32 + fr;
#pragma unroll
      for (int e4 = 0; e4 < 4; e4++) {
        const int I0 = it * TM + wi + i * 32 + e4 * 8 + fk * 4;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = acc[i][j][e4 * 4 + e] * g.mul;
        if constexpr (EPI == EPI_POLY) {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const _Float16 *a = g.a + mat * g.db + (int64_t)(I0 + e) * 2 * g.ld0 + packed(J);
            v[e] = __builtin_fmaf(g.cb, (float)a[0] + (float)a[KB], v[e]);
            if (I0 + e == J) v[e] += g.ca;
          }
        }
        if constexpr (EPI == EPI_LAST) {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (I0 + e < g.m && J < g.n)
              write_from_f32(g.out, mat * g.ob + (g.tall ? J * g.orow + I0 + e : (I0 + e) * g.orow + J), g.dtype, v[e]);
        } else {
          half4 hi, lo;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            hi[e] = (_Float16)v[e];
            lo[e] = (_Float16)(v[e] - (float)hi[e]);
            _Float16 *d = g.d0 + mat * g.db + (int64_t)(I0 + e) * 2 * g.ld0 + packed(J);
            d[0] = hi[e];
            d[KB] = lo[e];
          }
          // the transposed image (of a symmetric result: the tile above the diagonal)
          if (EPI == EPI_NEXT || it != jt) {
            _Float16 *d = g.d1 + mat * g.db + (int64_t)J * 2 * g.ld1 + packed(I0);
            *reinterpret_cast<half4 *>(d) = hi;
            *reinterpret_cast<half4 *>(d + KB) = lo;
          }
        }
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

int round_up(int x, int k) { return (x + k - 1) / k * k; }

OrthoArgs ortho_layout(void *base, int64_t batch, int rows, int cols, size_t *bytes) {
  OrthoArgs o = {};
  o.rows = rows;
  o.cols = cols;
  o.tall = rows > cols;
  o.m = o.tall ? cols : rows;
  o.n = o.tall ? rows : cols;
  o.mp = round_up(o.m, PAD);
  o.np = round_up(o.n, PAD);
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
  *bytes = (size_t)(p - (char *)base);
  return o;
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int rows, int cols) {
  size_t bytes = 0;
  ortho_layout(nullptr, batch, rows, cols, &bytes);
  return bytes;
}

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
  const int nb = rows < NORM_BLOCKS ? rows : NORM_BLOCKS;
  hipLaunchKernelGGL(k_ortho_norm, dim3(nb, (unsigned)batch), dim3(OR_THREADS), 0, stream, o);
  SPLAT_LAUNCH_CHECK();
  const int pr = o.tall ? o.np : o.mp, pc = o.tall ? o.mp : o.np;
  hipLaunchKernelGGL(k_ortho_pack, dim3(pc / 32, pr / 32, (unsigned)batch), dim3(OR_THREADS), 0, stream, o, nb);
  SPLAT_LAUNCH_CHECK();
  const int tm = o.mp / TM, tn = o.np / TN;
  for (int k = 0; k < steps; k++) {
    const int ea = scale_exp(u * u), eb = scale_exp(sup_quadratic(ca, cb, cc, u * u));
    const double un = sup_quintic(ca, cb, cc, u);
    const int en = scale_exp(un);
    const bool last = k + 1 == steps;
    GemmArgs q = {};
    q.p = q.q = o.x;
    q.pb = q.qb = o.sx;
    q.K = o.np;
    q.ti = q.tj = tm;
    q.mul = ldexpf(1.0f, ea - 2 * ex);
    q.d0 = q.d1 = o.a;
    q.db = o.sa;
    q.ld0 = q.ld1 = o.mp;
    hipLaunchKernelGGL(k_ortho_gemm<EPI_GRAM>, dim3(tm * (tm + 1) / 2, (unsigned)batch), dim3(OR_THREADS), 0, stream, q);
    SPLAT_LAUNCH_CHECK();
    q.p = q.q = o.a;
    q.pb = q.qb = o.sa;
    q.K = o.mp;
    q.mul = ldexpf(cc, eb - 2 * ea);
    q.a = o.a;
    q.ca = ldexpf(ca, eb);
    q.cb = ldexpf(cb, eb - ea);
    q.d0 = q.d1 = o.b;
    hipLaunchKernelGGL(k_ortho_gemm<EPI_POLY>, dim3(tm * (tm + 1) / 2, (unsigned)batch), dim3(OR_THREADS), 0, stream, q);
    SPLAT_LAUNCH_CHECK();
    q.p = o.b;
    q.q = o.y;
    q.pb = o.sa;
    q.qb = o.sx;
    q.tj = tn;
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
    if (last)
      hipLaunchKernelGGL(k_ortho_gemm<EPI_LAST>, dim3(tm * tn, (unsigned)batch), dim3(OR_THREADS), 0, stream, q);
    else
      hipLaunchKernelGGL(k_ortho_gemm<EPI_NEXT>, dim3(tm * tn, (unsigned)batch), dim3(OR_THREADS), 0, stream, q);
    SPLAT_LAUNCH_CHECK();
    _Float16 *t = o.y;
    o.y = o.y2;
    o.y2 = t;
    u = un;
    ex = en;
  }
  return SPLAT_OK;
}
