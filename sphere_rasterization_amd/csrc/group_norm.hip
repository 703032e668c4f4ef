// Group norm with an activation over channels-last images [N][P][C], and its gradients.
//
//   mu, var over the P C/G values of (image, group); xh = (x - mu) rstd,
//   rstd = 1 / sqrt(var + eps); z = w_c xh + b_c; y = act(z).
//   dz = dy act'(z); db = sum dz, dw = sum dz xh;
//   dx = rstd (w dz - (S1 + xh S2) / m), S1 = sum w dz, S2 = sum w dz xh over the group.
//
// Bound by the bytes of x, y (and dy, dx): a few operations per value. The statistics
// need a whole group before the first output, so each direction is a pass of sums, a
// join of the sums, and a pass that writes. A thread keeps to one pack of up to 16
// bytes of channels and walks over pixels, so that its channels' constants stay in
// registers and no vector has to lie within one group; consecutive threads cover
// consecutive packs of a pixel, then the next pixel. The writing pass takes the pieces in
// reverse order, so that it finds in the last-level cache what the pass of sums read
// last, and its stores pass by that cache (forward and backward of 1024x1024x32 fp32:
// 204 us without, 186 with; of six 1280x720x24 bf16: 454 and 400).
//
// The variance is never formed as E[x^2] - mu^2: each batch of NB pixels is centred on
// its own mean in registers, and (mean, M2) pairs are joined by
//   mean = sum n_i mean_i / n,  M2 = sum (M2_i + n_i (mean_i - mean)^2),
// so values far from zero lose nothing. Every sum runs in a fixed order.
#include "activation.h"
#include "learn_common.h"

namespace {

constexpr int GN_THREADS = 256, GN_WAVES = 4;
constexpr int NB = 8;                   // pixels per batch of a thread

struct NormArgs {
  const void *x, *dy, *w, *b;
  void *y, *dx, *dw, *db;
  float *mean, *rstd;                   // [N][G]
  float2 *part;                         // statistics: [N][slices][chunks][G] (mean, M2)
  float2 *sums, *joined;                // gradient: [N][chunks][C] and [N][C] (sum dz, sum dz xh)
  int64_t xi, xp, yi, yp, di, dp;       // image and pixel strides of x, of y or dy, of dx
  int64_t N, P;
  int C, G, cg;
  int units, us, slices, TP;            // packs per pixel, per slice; slices; pixels per step of a workgroup
  int64_t chunk;                        // pixels per workgroup
  int chunks;
  int pf32;                             // w, b, dw, db are fp32 (else of x's type)
  float eps;
  int64_t items;                        // workgroups' worth of work: N x slices x chunks
};

// ---- shared pieces ----------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float param_at(const void *p, int c, int pf32, float none) {
  if (!p) return none;
  return pf32 ? ((const float *)p)[c] : (float)((const T *)p)[c];
}
// Parameters of VEC channels from c: all loads under one branch, so that they are in
// flight together (a branch per channel made each workgroup wait 16 times in a row).
template <typename T, int VEC>
__device__ __forceinline__ void params_at(const void *p, int c, int pf32, float none, float (&o)[VEC]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < VEC; j++) o[j] = none;
  } else if (pf32) {
#pragma unroll
    for (int j = 0; j < VEC; j++) o[j] = ((const float *)p)[c + j];
  } else {
    T t[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) t[j] = ((const T *)p)[c + j];
#pragma unroll
    for (int j = 0; j < VEC; j++) o[j] = (float)t[j];
  }
}

// Groups of VEC channels from c: one division.
template <int VEC>
__device__ __forceinline__ void groups_at(int c, int cg, int (&g)[VEC]) {
  g[0] = c / cg;
  int left = (g[0] + 1) * cg - c;                 // channels of this group from c on
#pragma unroll
  for (int j = 1; j < VEC; j++) {
    left--;
    g[j] = g[j - 1] + (left == 0);
    left = left == 0 ? cg : left;
  }
}

template <typename T>
__device__ __forceinline__ void param_put(void *p, int c, int pf32, float v) {
  if (!p) return;
  if (pf32) ((float *)p)[c] = v;
  else ((T *)p)[c] = (T)v;
}

// A workgroup's piece: image n, channels of one slice, pixels [p0, p1).
struct Piece {
  int64_t n, p0, p1;
  int slice, chunk;
};
__device__ __forceinline__ Piece piece_of(const NormArgs &a, int64_t item) {
  Piece q;
  const int64_t per = (int64_t)a.slices * a.chunks;
  q.n = item / per;
  const int r = (int)(item - q.n * per);
  q.slice = r / a.chunks;
  q.chunk = r - q.slice * a.chunks;
  q.p0 = q.chunk * a.chunk;
  q.p1 = q.p0 + a.chunk < a.P ? q.p0 + a.chunk : a.P;
  return q;
}

// Pixels that pixel lane l of a piece of `pixels` takes.
__device__ __forceinline__ int lane_pixels(int64_t pixels, int l, int TP) {
  return pixels > l ? (int)((pixels - l + TP - 1) / TP) : 0;
}

// ---- statistics ---------------------------------------------------------------------
// d^2 for a difference from the mean of cnt values. With none before there is nothing to
// differ from, and d is the value itself, whose square may overflow (past 1.8e19) where no
// deviation does.
__device__ __forceinline__ float square_from(float d, float cnt) { return cnt > 0.0f ? d * d : 0.0f; }

template <typename T, int VEC>
__global__ __launch_bounds__(GN_THREADS) void k_norm_stats(NormArgs a) {
  __shared__ float s_mean[GN_THREADS * VEC], s_m2[GN_THREADS * VEC];
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const Piece q = piece_of(a, item);
    const int unit = q.slice * a.us + ul;
    const bool on = pl < a.TP && unit < a.units;
    float mean[VEC], m2[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) mean[j] = m2[j] = 0.0f;
    if (on) {
      const T *x = (const T *)a.x + q.n * a.xi + (int64_t)unit * VEC;
      float cnt = 0.0f;
      int64_t p = q.p0 + pl;
      for (; p + (int64_t)(NB - 1) * a.TP < q.p1; p += (int64_t)NB * a.TP) {
        float v[NB][VEC];
#pragma unroll
        for (int k = 0; k < NB; k++) load_f32<T, VEC>(x + (p + (int64_t)k * a.TP) * a.xp, v[k]);
        const float all = cnt + NB, r = (float)NB / all, f = cnt * r;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          float s = 0.0f;
#pragma unroll
          for (int k = 0; k < NB; k++) s += v[k][j];
          const float mb = s * (1.0f / NB), d = mb - mean[j];
          float qb = 0.0f;
#pragma unroll
          for (int k = 0; k < NB; k++) {
            const float e = v[k][j] - mb;
            qb = __builtin_fmaf(e, e, qb);
          }
          mean[j] = __builtin_fmaf(d, r, mean[j]);
          m2[j] = __builtin_fmaf(square_from(d, cnt), f, m2[j] + qb);
        }
        cnt = all;
      }
      for (; p < q.p1; p += a.TP) {
        float v[VEC];
        load_f32<T, VEC>(x + p * a.xp, v);
        const float all = cnt + 1.0f, r = 1.0f / all;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          const float d = v[j] - mean[j];
          mean[j] = __builtin_fmaf(d, r, mean[j]);
          m2[j] = __builtin_fmaf(square_from(d, cnt), cnt * r, m2[j]);
        }
        cnt = all;
      }
    }
    // channel-major in LDS: [pixel lane][channel of the slice]
    if (pl < a.TP) {
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        s_mean[(pl * a.us + ul) * VEC + j] = mean[j];
        s_m2[(pl * a.us + ul) * VEC + j] = m2[j];
      }
    }
    __syncthreads();
    const int sc = a.us * VEC, c0 = q.slice * sc, c1 = c0 + sc < a.C ? c0 + sc : a.C;
    const int64_t pixels = q.p1 - q.p0;
    for (int g = c0 / a.cg + w; g * (int64_t)a.cg < c1; g += GN_WAVES) {
      const int lo = g * a.cg > c0 ? g * a.cg : c0;
      const int64_t ge = (int64_t)(g + 1) * a.cg;
      const int hi = ge < c1 ? (int)ge : c1, k = hi - lo;
      const int entries = k * a.TP;
      float s = 0.0f;
      for (int e = lane; e < entries; e += 64) {
        const int l = e / k, c = lo - c0 + (e - l * k);
        s = __builtin_fmaf((float)lane_pixels(pixels, l, a.TP), s_mean[l * sc + c], s);
      }
      const float m = wave_sum(s) / ((float)pixels * (float)k);
      float v = 0.0f;
      for (int e = lane; e < entries; e += 64) {
        const int l = e / k, c = lo - c0 + (e - l * k);
        const float d = s_mean[l * sc + c] - m;
        v += __builtin_fmaf((float)lane_pixels(pixels, l, a.TP) * d, d, s_m2[l * sc + c]);
      }
      v = wave_sum(v);
      if (lane == 0) a.part[((q.n * a.slices + q.slice) * a.chunks + q.chunk) * a.G + g] = make_float2(m, v);
    }
    __syncthreads();
  }
}

// One workgroup per (image, group): joins the pieces' (mean, M2).
__device__ __forceinline__ float block_sum(float v, float *s) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(GN_THREADS) void k_norm_join(NormArgs a) {
  __shared__ float s[GN_WAVES];
  const int sc = a.us * (a.C / a.units);
  for (int64_t i = blockIdx.x; i < a.N * a.G; i += gridDim.x) {
    const int64_t n = i / a.G;
    const int g = (int)(i - n * a.G);
    const int c0 = g * a.cg, c1 = c0 + a.cg, s0 = c0 / sc, s1 = (c1 - 1) / sc;
    const float m = (float)a.P * (float)a.cg;
    // each piece's (mean, M2) and number of values
    auto each = [&](auto f) {
      for (int sl = s0; sl <= s1; sl++) {
        const int lo = sl * sc > c0 ? sl * sc : c0, hi = (sl + 1) * sc < c1 ? (sl + 1) * sc : c1;
        const float2 *p = a.part + (n * a.slices + sl) * (int64_t)a.chunks * a.G + g;
        for (int k = threadIdx.x; k < a.chunks; k += GN_THREADS) {
          const int64_t left = a.P - k * a.chunk;
          f(p[(int64_t)k * a.G], (float)(left < a.chunk ? left : a.chunk) * (float)(hi - lo));
        }
      }
    };
    float sum = 0.0f, m2 = 0.0f;
    each([&](float2 v, float cnt) { sum = __builtin_fmaf(cnt, v.x, sum); });
    const float mean = block_sum(sum, s) / m;
    each([&](float2 v, float cnt) {
      const float d = v.x - mean;
      m2 += __builtin_fmaf(cnt * d, d, v.y);
    });
    m2 = block_sum(m2, s);
    if (threadIdx.x == 0) {
      a.mean[i] = mean;
      a.rstd[i] = 1.0f / sqrtf(m2 / m + a.eps);
    }
  }
}

// ---- forward ------------------------------------------------------------------------
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(GN_THREADS) void k_norm_apply(NormArgs a) {
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const Piece q = piece_of(a, a.items - 1 - item);   // what the pass of sums read last comes first
    const int unit = q.slice * a.us + ul;
    if (pl >= a.TP || unit >= a.units) continue;
    float mu[VEC], s[VEC], b[VEC], r[VEC];
    int g[VEC];
    groups_at<VEC>(unit * VEC, a.cg, g);
    params_at<T, VEC>(a.w, unit * VEC, a.pf32, 1.0f, s);
    params_at<T, VEC>(a.b, unit * VEC, a.pf32, 0.0f, b);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      mu[j] = a.mean[q.n * a.G + g[j]];
      r[j] = a.rstd[q.n * a.G + g[j]];
    }
#pragma unroll
    for (int j = 0; j < VEC; j++) s[j] *= r[j];
    const T *x = (const T *)a.x + q.n * a.xi + (int64_t)unit * VEC;
    T *y = (T *)a.y + q.n * a.yi + (int64_t)unit * VEC;
    constexpr int U = 4;
    for (int64_t p = q.p0 + pl; p < q.p1; p += (int64_t)U * a.TP) {
      Raw<T, VEC> t[U];
#pragma unroll
      for (int k = 0; k < U; k++) {
        const int64_t pk = p + (int64_t)k * a.TP;
        t[k] = load_if<T, VEC>(pk < q.p1, x + pk * a.xp);
      }
#pragma unroll
      for (int k = 0; k < U; k++) {
        const int64_t pk = p + (int64_t)k * a.TP;
        if (pk < q.p1) {
          float v[VEC];
          to_f32<T, VEC>(t[k], v);
#pragma unroll
          for (int j = 0; j < VEC; j++) v[j] = act_of<ACT, sizeof(T) == 4>(__builtin_fmaf(v[j] - mu[j], s[j], b[j]));
          stream_f32<T, VEC>(y + pk * a.yp, v);
        }
      }
    }
  }
}

// ---- backward -----------------------------------------------------------------------
// Per (image, chunk, channel): sum dz and sum dz xh.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(GN_THREADS) void k_norm_bwd_sums(NormArgs a) {
  __shared__ float2 s_ab[GN_THREADS * VEC];
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const Piece q = piece_of(a, item);
    const int unit = q.slice * a.us + ul;
    const bool on = pl < a.TP && unit < a.units;
    float A[VEC], B[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) A[j] = B[j] = 0.0f;
    if (on) {
      float mu[VEC], rw[VEC], b[VEC], r[VEC];
      int g[VEC];
      groups_at<VEC>(unit * VEC, a.cg, g);
      params_at<T, VEC>(a.w, unit * VEC, a.pf32, 1.0f, rw);
      params_at<T, VEC>(a.b, unit * VEC, a.pf32, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        mu[j] = a.mean[q.n * a.G + g[j]];
        r[j] = a.rstd[q.n * a.G + g[j]];
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) rw[j] *= r[j];
      const T *x = (const T *)a.x + q.n * a.xi + (int64_t)unit * VEC;
      const T *dy = (const T *)a.dy + q.n * a.yi + (int64_t)unit * VEC;
      constexpr int U = 4;
      for (int64_t p = q.p0 + pl; p < q.p1; p += (int64_t)U * a.TP) {
        Raw<T, VEC> xv[U], dv[U];
#pragma unroll
        for (int k = 0; k < U; k++) {
          const int64_t pk = p + (int64_t)k * a.TP;
          xv[k] = load_if<T, VEC>(pk < q.p1, x + pk * a.xp);
          dv[k] = load_if<T, VEC>(pk < q.p1, dy + pk * a.yp);   // past the end dz = 0
        }
        float v[U][VEC], d[U][VEC];
#pragma unroll
        for (int k = 0; k < U; k++) {
          to_f32<T, VEC>(xv[k], v[k]);
          to_f32<T, VEC>(dv[k], d[k]);
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          float sa = 0.0f, sb = 0.0f;
#pragma unroll
          for (int k = 0; k < U; k++) {
            const float xc = v[k][j] - mu[j];
            const float dz = d[k][j] * act_slope<ACT, sizeof(T) == 4>(__builtin_fmaf(xc, rw[j], b[j]));
            sa += dz;
            sb = __builtin_fmaf(dz, xc, sb);
          }
          A[j] += sa;
          B[j] += sb;
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) B[j] *= a.rstd[q.n * a.G + g[j]];
    }
    if (pl < a.TP) {
#pragma unroll
      for (int j = 0; j < VEC; j++) s_ab[(pl * a.us + ul) * VEC + j] = make_float2(A[j], B[j]);
    }
    __syncthreads();
    const int sc = a.us * VEC, c0 = q.slice * sc;
    for (int c = threadIdx.x; c < sc && c0 + c < a.C; c += GN_THREADS) {
      float sa = 0.0f, sb = 0.0f;
      for (int l = 0; l < a.TP; l++) {
        const float2 v = s_ab[l * sc + c];
        sa += v.x;
        sb += v.y;
      }
      a.sums[(q.n * a.chunks + q.chunk) * a.C + c0 + c] = make_float2(sa, sb);
    }
    __syncthreads();
  }
}

// out[c] = sum over K rows of in[k][c], by a workgroup for 4 channels: 64 row lanes
// each, joined in LDS in a fixed order. Thread t < 4 holds channel c0 + t's result.
__device__ __forceinline__ float2 sum_rows4(const float2 *in, int64_t K, int C, int c0, float2 *s) {
  const int cl = threadIdx.x & 3, rl = threadIdx.x >> 2, c = c0 + cl;
  float2 t = make_float2(0.0f, 0.0f);
  if (c < C) {
    int64_t k = rl;
    for (; k + 192 < K; k += 256) {
      float2 v[4];
#pragma unroll
      for (int u = 0; u < 4; u++) v[u] = in[(k + 64 * u) * C + c];
      t.x += (v[0].x + v[1].x) + (v[2].x + v[3].x);
      t.y += (v[0].y + v[1].y) + (v[2].y + v[3].y);
    }
    for (; k < K; k += 64) {
      const float2 v = in[k * C + c];
      t.x += v.x;
      t.y += v.y;
    }
  }
  // lanes of a wave with the same channel, then the four waves
#pragma unroll
  for (int o = 4; o < 64; o <<= 1) {
    t.x += __shfl_xor(t.x, o);
    t.y += __shfl_xor(t.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 63) < 4) s[(threadIdx.x >> 6) * 4 + cl] = t;
  __syncthreads();
  float2 o = make_float2(0.0f, 0.0f);
  if (threadIdx.x < 4) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      o.x += s[k * 4 + threadIdx.x].x;
      o.y += s[k * 4 + threadIdx.x].y;
    }
  }
  return o;
}

// Per (image, channel): the chunks' sums joined.
__global__ __launch_bounds__(GN_THREADS) void k_norm_bwd_join(NormArgs a) {
  __shared__ float2 s[16];
  const int quads = (a.C + 3) / 4;
  for (int64_t i = blockIdx.x; i < a.N * quads; i += gridDim.x) {
    const int64_t n = i / quads;
    const int c0 = (int)(i - n * quads) * 4;
    const float2 o = sum_rows4(a.sums + n * a.chunks * (int64_t)a.C, a.chunks, a.C, c0, s);
    if (threadIdx.x < 4 && c0 + (int)threadIdx.x < a.C) a.joined[n * a.C + c0 + threadIdx.x] = o;
  }
}

// dx; the last workgroups of the grid sum the images' shares of dw and db instead.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(GN_THREADS) void k_norm_bwd_apply(NormArgs a, int main_blocks) {
  __shared__ float2 s_g[GN_THREADS * VEC + 2];   // (S1, S2) / m of each group the slice touches
  if ((int)blockIdx.x >= main_blocks) {
    const int quads = (a.C + 3) / 4;
    for (int i = blockIdx.x - main_blocks; i < quads; i += gridDim.x - main_blocks) {
      const float2 o = sum_rows4(a.joined, a.N, a.C, i * 4, s_g);
      const int c = i * 4 + threadIdx.x;
      if (threadIdx.x < 4 && c < a.C) {
        param_put<T>(a.db, c, a.pf32, o.x);
        param_put<T>(a.dw, c, a.pf32, o.y);
      }
    }
    return;
  }
  if (!a.dx) return;
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const float im = 1.0f / ((float)a.P * (float)a.cg);
  for (int64_t item = blockIdx.x; item < a.items; item += main_blocks) {
    const Piece q = piece_of(a, a.items - 1 - item);   // what the pass of sums read last comes first
    const int sc = a.us * VEC, c0 = q.slice * sc, c1 = c0 + sc < a.C ? c0 + sc : a.C;
    const int g0 = c0 / a.cg;
    for (int g = g0 + wv; (int64_t)g * a.cg < c1; g += GN_WAVES) {
      float s1 = 0.0f, s2 = 0.0f;
      for (int c = lane; c < a.cg; c += 64) {
        const float2 v = a.joined[q.n * a.C + (int64_t)g * a.cg + c];
        const float w = param_at<T>(a.w, g * a.cg + c, a.pf32, 1.0f);
        s1 = __builtin_fmaf(w, v.x, s1);
        s2 = __builtin_fmaf(w, v.y, s2);
      }
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if (lane == 0) s_g[g - g0] = make_float2(s1 * im, s2 * im);
    }
    __syncthreads();
    const int unit = q.slice * a.us + ul;
    if (pl < a.TP && unit < a.units) {
      // dx = (r w) dz - r t1 - (x - mu) (r^2 t2)
      float mu[VEC], rw[VEC], b[VEC], t1[VEC], t2[VEC], r[VEC];
      int g[VEC];
      groups_at<VEC>(unit * VEC, a.cg, g);
      params_at<T, VEC>(a.w, unit * VEC, a.pf32, 1.0f, rw);
      params_at<T, VEC>(a.b, unit * VEC, a.pf32, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        mu[j] = a.mean[q.n * a.G + g[j]];
        r[j] = a.rstd[q.n * a.G + g[j]];
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        rw[j] *= r[j];
        t1[j] = -r[j] * s_g[g[j] - g0].x;
        t2[j] = -r[j] * (r[j] * s_g[g[j] - g0].y);
      }
      const T *x = (const T *)a.x + q.n * a.xi + (int64_t)unit * VEC;
      const T *dy = (const T *)a.dy + q.n * a.yi + (int64_t)unit * VEC;
      T *dx = (T *)a.dx + q.n * a.di + (int64_t)unit * VEC;
      constexpr int U = 2;
      for (int64_t p = q.p0 + pl; p < q.p1; p += (int64_t)U * a.TP) {
        Raw<T, VEC> xv[U], dv[U];
#pragma unroll
        for (int k = 0; k < U; k++) {
          const int64_t pk = p + (int64_t)k * a.TP;
          xv[k] = load_if<T, VEC>(pk < q.p1, x + pk * a.xp);
          dv[k] = load_if<T, VEC>(pk < q.p1, dy + pk * a.yp);
        }
#pragma unroll
        for (int k = 0; k < U; k++) {
          const int64_t pk = p + (int64_t)k * a.TP;
          if (pk < q.p1) {
            float v[VEC], d[VEC];
            to_f32<T, VEC>(xv[k], v);
            to_f32<T, VEC>(dv[k], d);
#pragma unroll
            for (int j = 0; j < VEC; j++) {
              const float xc = v[j] - mu[j];
              const float dz = d[j] * act_slope<ACT, sizeof(T) == 4>(__builtin_fmaf(xc, rw[j], b[j]));
              v[j] = __builtin_fmaf(dz, rw[j], __builtin_fmaf(xc, t2[j], t1[j]));
            }
            stream_f32<T, VEC>(dx + pk * a.dp, v);
          }
        }
      }
    }
    __syncthreads();
  }
}

// ---- groups that one workgroup holds ------------------------------------------------
// One launch instead of three: a workgroup reads the values of one (image, group) into
// registers, R pixels per thread, and finishes them. Its threads keep to one pack of the
// group's channels each, as above.
constexpr int GS_THREADS = 512, GS_WAVES = GS_THREADS / WAVE;
constexpr int GS_FWD = 8, GS_BWD = 4;    // pixels per thread

__device__ __forceinline__ float block_sum8(float v, float *s) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < GS_WAVES; k++) t += s[k];
  return t;
}

// Workgroups go to the eight XCDs in turn: the groups of an image, whose values share
// cache lines, to one XCD.
__device__ __forceinline__ int64_t by_xcd(int64_t b, int64_t n) {
  const int64_t x = b & 7, each = n >> 3, more = n & 7;
  return x * each + (x < more ? x : more) + (b >> 3);
}

template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(GS_THREADS) void k_norm_small(NormArgs a) {
  __shared__ float s[GS_WAVES];
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  const bool on = pl < a.TP;
  const float im = 1.0f / ((float)a.P * (float)a.cg);
  for (int64_t b = blockIdx.x; b < a.N * a.G; b += gridDim.x) {
    const int64_t i = by_xcd(b, a.N * a.G), n = i / a.G;
    const int g = (int)(i - n * a.G), c0 = g * a.cg + ul * VEC;
    const T *x = (const T *)a.x + n * a.xi + c0;
    T *y = (T *)a.y + n * a.yi + c0;
    Raw<T, VEC> t[GS_FWD];
    float v[GS_FWD][VEC], sum = 0.0f, m2 = 0.0f, w[VEC], bias[VEC];
#pragma unroll
    for (int k = 0; k < GS_FWD; k++) {
      const int64_t p = pl + (int64_t)k * a.TP;
      t[k] = load_if<T, VEC>(on && p < a.P, x + p * a.xp);
    }
    params_at<T, VEC>(a.w, on ? c0 : 0, a.pf32, 1.0f, w);
    params_at<T, VEC>(a.b, on ? c0 : 0, a.pf32, 0.0f, bias);
#pragma unroll
    for (int k = 0; k < GS_FWD; k++) {
      to_f32<T, VEC>(t[k], v[k]);
#pragma unroll
      for (int j = 0; j < VEC; j++) sum += v[k][j];
    }
    const float mean = block_sum8(sum, s) * im;
#pragma unroll
    for (int k = 0; k < GS_FWD; k++)
      if (on && pl + (int64_t)k * a.TP < a.P) {
#pragma unroll
        for (int j = 0; j < VEC; j++) m2 = __builtin_fmaf(v[k][j] - mean, v[k][j] - mean, m2);
      }
    const float rstd = 1.0f / sqrtf(block_sum8(m2, s) * im + a.eps);
    if (threadIdx.x == 0) {
      a.mean[i] = mean;
      a.rstd[i] = rstd;
    }
#pragma unroll
    for (int k = 0; k < GS_FWD; k++) {
      const int64_t p = pl + (int64_t)k * a.TP;
      if (on && p < a.P) {
#pragma unroll
        for (int j = 0; j < VEC; j++) v[k][j] = act_of<ACT, sizeof(T) == 4>(__builtin_fmaf(v[k][j] - mean, rstd * w[j], bias[j]));
        store_f32<T, VEC>(y + p * a.yp, v[k]);
      }
    }
  }
}

// The same for the gradients: the channels' sums over the pixels, then dx. The shares of
// dw and db go to `joined`, or straight to dw and db if there is one image.
template <typename T, int VEC, int ACT>
__global__ __launch_bounds__(GS_THREADS) void k_norm_bwd_small(NormArgs a) {
  __shared__ float2 s_ab[GS_THREADS * VEC];
  __shared__ float2 s_g[GS_WAVES];
  const int pl = threadIdx.x / a.us, ul = threadIdx.x - pl * a.us;
  const bool on = pl < a.TP;
  const float im = 1.0f / ((float)a.P * (float)a.cg);
  for (int64_t blk = blockIdx.x; blk < a.N * a.G; blk += gridDim.x) {
    const int64_t i = by_xcd(blk, a.N * a.G), n = i / a.G;
    const int g = (int)(i - n * a.G), c0 = g * a.cg + ul * VEC;
    const T *x = (const T *)a.x + n * a.xi + c0, *dy = (const T *)a.dy + n * a.yi + c0;
    const float mean = a.mean[i], rstd = a.rstd[i];
    Raw<T, VEC> xv[GS_BWD], dv[GS_BWD];
    float v[GS_BWD][VEC], d[GS_BWD][VEC], rw[VEC], b[VEC], A[VEC], B[VEC];
#pragma unroll
    for (int k = 0; k < GS_BWD; k++) {
      const int64_t p = pl + (int64_t)k * a.TP;
      xv[k] = load_if<T, VEC>(on && p < a.P, x + p * a.xp);
      dv[k] = load_if<T, VEC>(on && p < a.P, dy + p * a.yp);
    }
    params_at<T, VEC>(a.w, on ? c0 : 0, a.pf32, 1.0f, rw);
    params_at<T, VEC>(a.b, on ? c0 : 0, a.pf32, 0.0f, b);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      rw[j] *= rstd;
      A[j] = B[j] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < GS_BWD; k++) {
      to_f32<T, VEC>(xv[k], v[k]);
      to_f32<T, VEC>(dv[k], d[k]);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        v[k][j] -= mean;
        d[k][j] *= act_slope<ACT, sizeof(T) == 4>(__builtin_fmaf(v[k][j], rw[j], b[j]));
        A[j] += d[k][j];
        B[j] = __builtin_fmaf(d[k][j], v[k][j], B[j]);
      }
    }
    if (on) {
#pragma unroll
      for (int j = 0; j < VEC; j++) s_ab[threadIdx.x * VEC + j] = make_float2(A[j], B[j] * rstd);
    }
    __syncthreads();
    // the group's channels, each by as many lanes of a wave as there are, up to 64
    const int lane = threadIdx.x & 63;
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x >> 6; c < a.cg; c += GS_WAVES) {
      float sa = 0.0f, sb = 0.0f;
      for (int l = lane; l < a.TP; l += 64) {
        const float2 t = s_ab[l * a.cg + c];
        sa += t.x;
        sb += t.y;
      }
      sa = wave_sum(sa);
      sb = wave_sum(sb);
      const int ch = g * a.cg + c;
      const float w = param_at<T>(a.w, ch, a.pf32, 1.0f);
      s1 = __builtin_fmaf(w, sa, s1);
      s2 = __builtin_fmaf(w, sb, s2);
      if (lane == 0) {
        if (a.joined) {
          a.joined[n * a.C + ch] = make_float2(sa, sb);
        } else {
          param_put<T>(a.db, ch, a.pf32, sa);
          param_put<T>(a.dw, ch, a.pf32, sb);
        }
      }
    }
    if (lane == 0) s_g[threadIdx.x >> 6] = make_float2(s1, s2);
    __syncthreads();
    s1 = s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < GS_WAVES; k++) {
      s1 += s_g[k].x;
      s2 += s_g[k].y;
    }
    if (a.dx) {
      const float t1 = -rstd * (s1 * im), t2 = -rstd * (rstd * (s2 * im));
      T *dx = (T *)a.dx + n * a.di + c0;
#pragma unroll
      for (int k = 0; k < GS_BWD; k++) {
        const int64_t p = pl + (int64_t)k * a.TP;
        if (on && p < a.P) {
#pragma unroll
          for (int j = 0; j < VEC; j++) v[k][j] = __builtin_fmaf(d[k][j], rw[j], __builtin_fmaf(v[k][j], t2, t1));
          store_f32<T, VEC>(dx + p * a.dp, v[k]);
        }
      }
    }
    __syncthreads();
  }
}

// dw and db from the images' shares.
template <typename T>
__global__ __launch_bounds__(GN_THREADS) void k_norm_bwd_params(NormArgs a) {
  __shared__ float2 s[16];
  const int quads = (a.C + 3) / 4;
  for (int i = blockIdx.x; i < quads; i += gridDim.x) {
    const float2 o = sum_rows4(a.joined, a.N, a.C, i * 4, s);
    const int c = i * 4 + threadIdx.x;
    if (threadIdx.x < 4 && c < a.C) {
      param_put<T>(a.db, c, a.pf32, o.x);
      param_put<T>(a.dw, c, a.pf32, o.y);
    }
  }
}

// dw and db of no pixels at all.
template <typename T>
__global__ __launch_bounds__(GN_THREADS) void k_norm_zero_params(NormArgs a) {
  for (int c = blockIdx.x * GN_THREADS + threadIdx.x; c < a.C; c += gridDim.x * GN_THREADS) {
    param_put<T>(a.dw, c, a.pf32, 0.0f);
    param_put<T>(a.db, c, a.pf32, 0.0f);
  }
}

// The statistics of no pixels: mean 0 and variance 0.
__global__ __launch_bounds__(GN_THREADS) void k_norm_empty_stats(NormArgs a) {
  for (int64_t i = (int64_t)blockIdx.x * GN_THREADS + threadIdx.x; i < a.N * a.G; i += (int64_t)gridDim.x * GN_THREADS) {
    a.mean[i] = 0.0f;
    a.rstd[i] = 1.0f / sqrtf(a.eps);
  }
}

// ---- launches -----------------------------------------------------------------------
// Pieces for a pass over a.P > 0 pixels: about `target` workgroups, each with at least
// `least` pixel steps per thread so that its constants and its share of the join are paid
// for.
void split(NormArgs &a, int vec, int64_t target, int64_t least) {
  a.units = a.C / vec;
  a.us = a.units < GN_THREADS ? a.units : GN_THREADS;
  a.slices = (a.units + a.us - 1) / a.us;
  a.TP = GN_THREADS / a.us;
  const int64_t steps = (a.P + a.TP - 1) / a.TP;
  int64_t chunks = target / (a.N * a.slices > 0 ? a.N * a.slices : 1);
  if (chunks > steps / least) chunks = steps / least;
  if (chunks < 1) chunks = 1;
  a.chunk = (steps + chunks - 1) / chunks * a.TP;
  a.chunks = (int)((a.P + a.chunk - 1) / a.chunk);
  if (a.chunks < 1) a.chunks = 1;
  a.items = a.N * a.slices * a.chunks;
}

// Measured (us for a whole call) at 768, 1024, 2048 and 4096 workgroups of the statistics:
// 1920x1080x32 fp16 forward 79, 81, 83, 83, forward and backward of 1024x1024x32 fp32 184,
// 184, 186, 186 and of six 1280x720x24 bf16 401, 401, 401, 407 (the first was 96, 98, 94, 95
// when 2048 was taken, before parameters were loaded under one branch). The last at 768,
// 1024, 2048 of the gradient's sums 401, 403, 398 (480, 526, 498 when 768 was taken: its
// registers let three workgroups share a CU, so that is one round).
constexpr int64_t STAT_BLOCKS = 2048, SUM_BLOCKS = 768, SUM_LEAST = 16;
constexpr int64_t APPLY_BLOCKS = 4096, APPLY_LEAST = 8;   // passes that write

unsigned blocks_of(int64_t items) { return (unsigned)(items < (1 << 20) ? items : (1 << 20)); }

// Whether to hold each group in one workgroup, `per` pixels to a thread, in packs of
// `vec` channels; sets the mapping. Only while the groups are few: a workgroup waits for
// its loads, two sums over itself and its stores in turn. bf16 forward (backward), us on
// the GPU, this form against three launches: 8 groups of 1551 x 8 values 5.9 (8.6) against
// 18.2 (22.9); 512 groups 14.4 (24.5) against 24.6 (30.1); 1024 groups 25.5 (42.4) against
// 28.7 (37.0); 2048 groups 44.5 (73.1) against 41.7 (52.4).
bool fits_small(NormArgs &a, int vec, int per) {
  if (a.N * a.G > (per == GS_FWD ? 1024 : 512)) return false;
  if (a.cg % vec || a.cg / vec > GS_THREADS) return false;
  const int us = a.cg / vec, TP = GS_THREADS / us;
  if (a.P > (int64_t)per * TP) return false;
  a.us = us;
  a.TP = TP;
  return true;
}

// Pack width: what rows and alignment allow; for groups that a workgroup can hold, also a
// divisor of the group.
int norm_vec(const splat_norm *d, const void *x, const void *y, const void *dx, int per) {
  const int64_t strides[6] = {d->x_image_stride, d->x_pixel_stride, d->y_image_stride,
                              d->y_pixel_stride, d->dx_image_stride, d->dx_pixel_stride};
  const void *ptrs[3] = {x, y, dx ? dx : x};
  const int cg = d->channels / d->groups;
  const int in_group = vec_width(dtype_bytes(d->dtype), cg, strides, dx ? 6 : 4, ptrs, 3);
  NormArgs a = {};
  a.N = d->images;
  a.G = d->groups;
  a.cg = cg;
  a.P = d->pixels;
  if (fits_small(a, in_group, per)) return in_group;
  return vec_width(dtype_bytes(d->dtype), d->channels, strides, dx ? 6 : 4, ptrs, 3);
}

NormArgs norm_args(const splat_norm *d, const void *x, const void *w, const void *b) {
  NormArgs a = {};
  a.x = x; a.w = w; a.b = b;
  a.xi = d->x_image_stride; a.xp = d->x_pixel_stride;
  a.yi = d->y_image_stride; a.yp = d->y_pixel_stride;
  a.di = d->dx_image_stride; a.dp = d->dx_pixel_stride;
  a.N = d->images; a.P = d->pixels;
  a.C = d->channels; a.G = d->groups; a.cg = d->channels / d->groups;
  a.pf32 = d->param_dtype == SPLAT_F32;
  a.eps = d->eps;
  return a;
}

template <typename T, int VEC, int ACT>
int run_norm(NormArgs a, hipStream_t stream) {
  if (fits_small(a, VEC, GS_FWD)) {
    hipLaunchKernelGGL((k_norm_small<T, VEC, ACT>), dim3(blocks_of(a.N * a.G)), dim3(GS_THREADS), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  split(a, VEC, STAT_BLOCKS, SUM_LEAST);
  hipLaunchKernelGGL((k_norm_stats<T, VEC>), dim3(blocks_of(a.items)), dim3(GN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  hipLaunchKernelGGL(k_norm_join, dim3(blocks_of(a.N * a.G)), dim3(GN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  split(a, VEC, APPLY_BLOCKS, APPLY_LEAST);
  hipLaunchKernelGGL((k_norm_apply<T, VEC, ACT>), dim3(blocks_of(a.items)), dim3(GN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T, int VEC, int ACT>
int run_norm_bwd(NormArgs a, hipStream_t stream) {
  const int quads = (a.C + 3) / 4;
  if (fits_small(a, VEC, GS_BWD)) {
    const bool params = a.dw || a.db;
    a.joined = a.N == 1 || !params ? nullptr : a.sums;
    hipLaunchKernelGGL((k_norm_bwd_small<T, VEC, ACT>), dim3(blocks_of(a.N * a.G)), dim3(GS_THREADS), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
    if (a.joined) {
      hipLaunchKernelGGL(k_norm_bwd_params<T>, dim3((unsigned)(quads < 4096 ? quads : 4096)), dim3(GN_THREADS), 0, stream, a);
      SPLAT_LAUNCH_CHECK();
    }
    return SPLAT_OK;
  }
  split(a, VEC, SUM_BLOCKS, SUM_LEAST);
  hipLaunchKernelGGL((k_norm_bwd_sums<T, VEC, ACT>), dim3(blocks_of(a.items)), dim3(GN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  hipLaunchKernelGGL(k_norm_bwd_join, dim3(blocks_of(a.N * quads)), dim3(GN_THREADS), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  split(a, VEC, APPLY_BLOCKS, APPLY_LEAST);
  const unsigned main_blocks = blocks_of(a.items);
  const unsigned extra = a.dw || a.db ? (unsigned)(quads < 4096 ? quads : 4096) : 0u;
  hipLaunchKernelGGL((k_norm_bwd_apply<T, VEC, ACT>), dim3(main_blocks + extra), dim3(GN_THREADS), 0, stream, a,
                     (int)main_blocks);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T, int VEC>
int by_act(const NormArgs &a, int act, bool bwd, hipStream_t s) {
  switch (act) {
    case SPLAT_ACT_RELU: return bwd ? run_norm_bwd<T, VEC, SPLAT_ACT_RELU>(a, s) : run_norm<T, VEC, SPLAT_ACT_RELU>(a, s);
    case SPLAT_ACT_SILU: return bwd ? run_norm_bwd<T, VEC, SPLAT_ACT_SILU>(a, s) : run_norm<T, VEC, SPLAT_ACT_SILU>(a, s);
    case SPLAT_ACT_GELU: return bwd ? run_norm_bwd<T, VEC, SPLAT_ACT_GELU>(a, s) : run_norm<T, VEC, SPLAT_ACT_GELU>(a, s);
    default: return bwd ? run_norm_bwd<T, VEC, SPLAT_ACT_NONE>(a, s) : run_norm<T, VEC, SPLAT_ACT_NONE>(a, s);
  }
}

int dispatch(const NormArgs &a, int dtype, int vec, int act, bool bwd, hipStream_t s) {
  if (dtype == SPLAT_F32) {
    if (vec == 4) return by_act<float, 4>(a, act, bwd, s);
    if (vec == 2) return by_act<float, 2>(a, act, bwd, s);
    return by_act<float, 1>(a, act, bwd, s);
  }
  if (dtype == SPLAT_F16) {
    if (vec == 8) return by_act<f16_t, 8>(a, act, bwd, s);
    if (vec == 4) return by_act<f16_t, 4>(a, act, bwd, s);
    if (vec == 2) return by_act<f16_t, 2>(a, act, bwd, s);
    return by_act<f16_t, 1>(a, act, bwd, s);
  }
  if (vec == 8) return by_act<bf16_t, 8>(a, act, bwd, s);
  if (vec == 4) return by_act<bf16_t, 4>(a, act, bwd, s);
  if (vec == 2) return by_act<bf16_t, 2>(a, act, bwd, s);
  return by_act<bf16_t, 1>(a, act, bwd, s);
}

}  // namespace

// For any pack width: the pieces of the narrowest width are the most. Alignment decides
// whether a group fits one workgroup, so only groups that fit at every width need nothing.
size_t group_norm_workspace_bytes(const splat_norm *d, bool bwd) {
  if (d->images == 0 || d->pixels == 0) return 0;      // no values, no passes
  NormArgs a = norm_args(d, nullptr, nullptr, nullptr);
  size_t most = 0;
  for (int vec = 16 / dtype_bytes(d->dtype); vec >= 1; vec >>= 1) {
    if (a.C % vec) continue;
    size_t need;
    split(a, vec, bwd ? SUM_BLOCKS : STAT_BLOCKS, SUM_LEAST);
    if (bwd)
      need = ws_align(sizeof(float2) * (size_t)a.N * a.chunks * a.C) + sizeof(float2) * (size_t)a.N * a.C;
    else
      need = sizeof(float2) * (size_t)a.N * a.slices * a.chunks * a.G;
    if (fits_small(a, vec, bwd ? GS_BWD : GS_FWD)) need = bwd && a.N > 1 ? sizeof(float2) * (size_t)a.N * a.C : 0;
    if (need > most) most = need;
  }
  return ws_align(most);
}

int launch_group_norm(const splat_norm *d, const void *x, const void *w, const void *b, void *y, float *mean,
                      float *rstd, void *ws, hipStream_t stream) {
  if (d->images == 0) return SPLAT_OK;
  NormArgs a = norm_args(d, x, w, b);
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.part = (float2 *)ws;
  if (d->pixels == 0) {
    hipLaunchKernelGGL(k_norm_empty_stats, dim3(blocks_of((a.N * a.G + GN_THREADS - 1) / GN_THREADS)), dim3(GN_THREADS),
                       0, stream, a);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  return dispatch(a, d->dtype, norm_vec(d, x, y, nullptr, GS_FWD), d->act, false, stream);
}

int launch_group_norm_bwd(const splat_norm *d, const void *d_y, const void *x, const float *mean, const float *rstd,
                          const void *w, const void *b, void *dx, void *dw, void *db, void *ws, hipStream_t stream) {
  if (!dx && !dw && !db) return SPLAT_OK;
  NormArgs a = norm_args(d, x, w, b);
  a.dy = d_y;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  if (d->images == 0 || d->pixels == 0) {
    if (!dw && !db) return SPLAT_OK;
    const dim3 grid((unsigned)((a.C + GN_THREADS - 1) / GN_THREADS));
    if (d->dtype == SPLAT_F16) hipLaunchKernelGGL(k_norm_zero_params<f16_t>, grid, dim3(GN_THREADS), 0, stream, a);
    else hipLaunchKernelGGL(k_norm_zero_params<bf16_t>, grid, dim3(GN_THREADS), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  const int vec = norm_vec(d, x, d_y, dx, GS_BWD);
  split(a, vec, SUM_BLOCKS, SUM_LEAST);
  a.sums = (float2 *)ws;
  a.joined = (float2 *)((char *)ws + ws_align(sizeof(float2) * (size_t)a.N * a.chunks * a.C));
  return dispatch(a, d->dtype, vec, d->act, true, stream);
}
