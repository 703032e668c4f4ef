// Rows of a shared feature table, and the table's gradient by sorted tokens.
//
// Forward: y[i] = s T[id_i] (a zero row where id_i is outside the table), a pure
// gather: bound by the bytes of y and of the distinct rows. One thread moves up to
// 16 bytes, LK_ITEMS of them with independent loads.
//
// Gradient: dT[v] = s sum over {i : id_i = v} dy[i], every row of dT written once.
// Adding rows atomically would make the sum depend on the order of arrival, so the
// tokens are sorted by id (stable, so each row's tokens keep their order) and each
// row is summed in a fixed order:
//   1. counting sort by digits of up to 9 bits, least significant first: counts per
//      tile of 4096 tokens, a scan per digit, a scatter that ranks equal digits
//      within a wave by ballots. Up to 4096 tokens: one workgroup, all in LDS;
//   2. the sorted list is cut into chunks of 64; a chunk that lies within one row's
//      segment is summed to one fp32 row, and 64 such sums to one of the next level;
//   3. each row adds its loose tokens and its whole chunks and writes its gradient.
// So a row that holds all n tokens costs no thread more than 4 x 64 + n / 4096 adds.
#include "learn_common.h"

namespace {

constexpr int LK_THREADS = 256;
constexpr int LK_ITEMS = 4;
constexpr int ST_THREADS = 256, ST_ITEMS = 16, ST_TILE = ST_THREADS * ST_ITEMS;
constexpr int ST_WAVES = ST_THREADS / WAVE;
constexpr int RADIX_BITS = 9, RADIX = 1 << RADIX_BITS;
constexpr int CHUNK = 64;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, int VEC, typename ID>
__global__ __launch_bounds__(LK_THREADS) void k_lookup(const T *__restrict__ table, int64_t ldt, int64_t rows,
                                                       const ID *__restrict__ ids, uint32_t total, FastDiv units,
                                                       float scale, T *__restrict__ out, int64_t ldo) {
  const uint32_t base = blockIdx.x * (LK_THREADS * LK_ITEMS) + threadIdx.x;
  float v[LK_ITEMS][VEC];
#pragma unroll
  for (int k = 0; k < LK_ITEMS; k++) {
    const uint32_t u = base + k * LK_THREADS;
#pragma unroll
    for (int j = 0; j < VEC; j++) v[k][j] = 0.0f;
    if (u < total) {
      const uint32_t i = div_by(u, units), c = (u - i * units.d) * VEC;
      const int64_t id = (int64_t)ids[i];
      if (id >= 0 && id < rows) load_f32<T, VEC>(table + id * ldt + c, v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < LK_ITEMS; k++) {
    const uint32_t u = base + k * LK_THREADS;
    if (u < total) {
      const uint32_t i = div_by(u, units), c = (u - i * units.d) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; j++) v[k][j] *= scale;
      store_f32<T, VEC>(out + (int64_t)i * ldo + c, v[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// sort by id
// ---------------------------------------------------------------------------
// A token's key: its id, or `rows` (after every row) where the id is outside.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(const ID *ids, uint32_t i, uint32_t rows) {
  const int64_t id = (int64_t)ids[i];
  return id >= 0 && id < (int64_t)rows ? (uint32_t)id : rows;
}

// Where pass p reads its keys: the caller's ids in the first pass, the workspace after.
template <typename ID>
struct KeySource {
  const ID *ids;
  const uint32_t *keys;   // NULL in the first pass
  const uint32_t *perm;
  uint32_t n, rows;
  __device__ uint32_t key(uint32_t i) const { return keys ? keys[i] : key_of(ids, i, rows); }
  __device__ uint32_t token(uint32_t i) const { return keys ? perm[i] : i; }
};

// counts[digit][tile]; also clears the rows' segment bounds (each thread a share).
template <typename ID>
__global__ __launch_bounds__(ST_THREADS) void k_sort_count(KeySource<ID> src, int shift, int bits, uint32_t tiles,
                                                           uint32_t *__restrict__ counts, int2 *bounds,
                                                           uint32_t nbounds) {
  __shared__ uint32_t h[RADIX];
  for (int d = threadIdx.x; d < RADIX; d += ST_THREADS) h[d] = 0;
  __syncthreads();
  const uint32_t mask = (1u << bits) - 1u, t0 = blockIdx.x * (uint32_t)ST_TILE;
#pragma unroll
  for (int j = 0; j < ST_ITEMS; j++) {
    const uint32_t i = t0 + j * ST_THREADS + threadIdx.x;
    if (i < src.n) atomicAdd(&h[(src.key(i) >> shift) & mask], 1u);
  }
  if (bounds)
    for (uint32_t r = blockIdx.x * ST_THREADS + threadIdx.x; r < nbounds; r += gridDim.x * ST_THREADS)
      bounds[r] = make_int2(0, 0);
  __syncthreads();
  for (int d = threadIdx.x; d < (1 << bits); d += ST_THREADS) counts[(size_t)d * tiles + blockIdx.x] = h[d];
}

// Inclusive scan over the workgroup's threads (WAVES waves); s: WAVES words of LDS.
template <int WAVES>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *s, uint32_t *total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) s[w] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < WAVES; k++) {
    const uint32_t t = s[k];
    if (k < w) before += t;
    all += t;
  }
  *total = all;
  return x + before;
}

// One workgroup per digit: exclusive scan of its counts over the tiles, and its total.
__global__ __launch_bounds__(ST_THREADS) void k_sort_scan(uint32_t *__restrict__ counts, uint32_t tiles,
                                                          uint32_t *__restrict__ totals) {
  __shared__ uint32_t s[ST_WAVES];
  uint32_t *row = counts + (size_t)blockIdx.x * tiles;
  uint32_t run = 0;
  for (uint32_t t0 = 0; t0 < tiles; t0 += ST_THREADS) {
    const uint32_t t = t0 + threadIdx.x;
    const uint32_t c = t < tiles ? row[t] : 0u;
    uint32_t total;
    const uint32_t inc = block_scan<ST_WAVES>(c, s, &total);
    if (t < tiles) row[t] = run + inc - c;
    run += total;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// Rank of this lane's digit among the wave's items so far, adding the wave's items to
// hist (this wave's counters). Lanes with equal digits find each other by one ballot
// per bit; the lowest of them updates the counter. Inactive lanes pass ok = false.
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, int bits, bool ok, volatile uint32_t *hist) {
  uint64_t peers = ballot64(ok);
#pragma unroll
  for (int b = 0; b < RADIX_BITS; b++) {
    if (b < bits) {
      const bool one = (digit >> b) & 1u;
      const uint64_t m = ballot64(one);
      peers &= one ? m : ~m;
    }
  }
  const uint64_t below = peers & ((1ull << lane_id()) - 1ull);
  uint32_t old = 0;
  if (ok) old = hist[digit];
  __builtin_amdgcn_wave_barrier();
  if (ok && below == 0) hist[digit] = old + (uint32_t)__popcll(peers);
  __builtin_amdgcn_wave_barrier();
  return old + (uint32_t)__popcll(below);
}

template <typename ID>
__global__ __launch_bounds__(ST_THREADS) void k_sort_scatter(KeySource<ID> src, int shift, int bits, uint32_t tiles,
                                                             const uint32_t *__restrict__ counts,
                                                             const uint32_t *__restrict__ totals,
                                                             uint32_t *__restrict__ keys_out,
                                                             uint32_t *__restrict__ perm_out) {
  __shared__ uint32_t hist[ST_WAVES][RADIX];
  __shared__ uint32_t s[ST_WAVES];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int d = threadIdx.x; d < ST_WAVES * RADIX; d += ST_THREADS) (&hist[0][0])[d] = 0;
  const uint32_t mask = (1u << bits) - 1u;
  const uint32_t i0 = blockIdx.x * (uint32_t)ST_TILE + w * (ST_TILE / ST_WAVES) + lane;
  uint32_t key[ST_ITEMS], tok[ST_ITEMS], rank[ST_ITEMS];
#pragma unroll
  for (int j = 0; j < ST_ITEMS; j++) {
    const uint32_t i = i0 + j * WAVE;
    key[j] = i < src.n ? src.key(i) : 0u;
    tok[j] = i < src.n ? src.token(i) : 0u;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ST_ITEMS; j++)
    rank[j] = wave_rank((key[j] >> shift) & mask, bits, i0 + j * WAVE < src.n, hist[w]);
  // each digit's first slot for each wave: the digits before it in all tiles, its
  // own items in earlier tiles, its items in earlier waves of this tile
  constexpr int DPT = RADIX / ST_THREADS;
  uint32_t tot[DPT], sum = 0, all;
#pragma unroll
  for (int k = 0; k < DPT; k++) {
    const uint32_t d = threadIdx.x * DPT + k;
    tot[k] = d <= mask ? totals[d] : 0u;
    sum += tot[k];
  }
  uint32_t at = block_scan<ST_WAVES>(sum, s, &all) - sum;   // its barriers also end the ranking
#pragma unroll
  for (int k = 0; k < DPT; k++) {
    const uint32_t d = threadIdx.x * DPT + k;
    if (d <= mask) {
      uint32_t run = at + counts[(size_t)d * tiles + blockIdx.x];
#pragma unroll
      for (int v = 0; v < ST_WAVES; v++) {
        const uint32_t c = hist[v][d];
        hist[v][d] = run;
        run += c;
      }
    }
    at += tot[k];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ST_ITEMS; j++) {
    if (i0 + j * WAVE < src.n) {
      const uint32_t p = hist[w][(key[j] >> shift) & mask] + rank[j];
      keys_out[p] = key[j];
      perm_out[p] = tok[j];
    }
  }
}

// Up to ST_TILE tokens: workgroup 0 sorts them in LDS, the others clear the bounds.
constexpr int SM_THREADS = 1024, SM_WAVES = SM_THREADS / WAVE, SM_ITEMS = ST_TILE / SM_THREADS;
template <typename ID>
__global__ __launch_bounds__(SM_THREADS) void k_sort_small(const ID *__restrict__ ids, uint32_t n, uint32_t rows,
                                                           int bits, int passes, uint32_t *__restrict__ keys_out,
                                                           uint32_t *__restrict__ perm_out, int2 *bounds) {
  if (blockIdx.x > 0) {
    for (uint32_t r = (blockIdx.x - 1) * SM_THREADS + threadIdx.x; r < rows; r += (gridDim.x - 1) * SM_THREADS)
      bounds[r] = make_int2(0, 0);
    return;
  }
  __shared__ uint32_t hist[SM_WAVES][RADIX];
  __shared__ uint32_t s[SM_WAVES];
  __shared__ uint32_t sk[ST_TILE], sp[ST_TILE];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t i0 = w * (ST_TILE / SM_WAVES) + lane;
  uint32_t key[SM_ITEMS], tok[SM_ITEMS], rank[SM_ITEMS];
#pragma unroll
  for (int j = 0; j < SM_ITEMS; j++) {
    const uint32_t i = i0 + j * WAVE;
    key[j] = i < n ? key_of(ids, i, rows) : 0u;
    tok[j] = i;
  }
  const int dbits = (bits + passes - 1) / passes;
  for (int p = 0; p < passes; p++) {
    const int shift = p * dbits;
    const uint32_t mask = (1u << dbits) - 1u;
    for (int d = threadIdx.x; d < SM_WAVES * RADIX; d += SM_THREADS) (&hist[0][0])[d] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SM_ITEMS; j++)
      rank[j] = wave_rank((key[j] >> shift) & mask, dbits, i0 + j * WAVE < n, hist[w]);
    __syncthreads();
    const uint32_t d = threadIdx.x;   // SM_THREADS >= RADIX
    uint32_t sum = 0, all;
    if (d < RADIX)
      for (int v = 0; v < SM_WAVES; v++) sum += hist[v][d];
    uint32_t run = block_scan<SM_WAVES>(sum, s, &all) - sum;
    if (d < RADIX)
      for (int v = 0; v < SM_WAVES; v++) {
        const uint32_t c = hist[v][d];
        hist[v][d] = run;
        run += c;
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SM_ITEMS; j++)
      if (i0 + j * WAVE < n) {
        const uint32_t at = hist[w][(key[j] >> shift) & mask] + rank[j];
        sk[at] = key[j];
        sp[at] = tok[j];
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SM_ITEMS; j++) {
      const uint32_t i = i0 + j * WAVE;
      if (i < n) {
        key[j] = sk[i];
        tok[j] = sp[i];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < SM_ITEMS; j++) {
    const uint32_t i = i0 + j * WAVE;
    if (i < n) {
      keys_out[i] = key[j];
      perm_out[i] = tok[j];
    }
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
// How a wave covers a row of `units` packs: 2^lg lanes per row (64 if the row has 64
// packs or more, then one slice of 64 packs per wave), so 64 >> lg rows at once.
struct SumArgs {
  const void *dy;
  int64_t ldy;
  const uint32_t *perm, *keys;
  int2 *bounds;
  float *part1, *part2;     // sums of whole chunks of 64 and of 64 x 64 tokens [.][dim]
  void *grad;
  int64_t ldg;
  uint32_t n, rows;
  int dim, units, lg, slices, two_levels, accumulate;
  float scale;
};

// Adds rows [p0, p1) of a list to acc, the wave's 64 >> lg row lanes in turn: row lane
// g takes p0 + g, p0 + g + G, ...; U loads in flight each. Rows are tokens of dy, found
// through perm (src = T), or chunk sums (src = float, perm NULL).
template <typename T, int VEC, int U>
__device__ __forceinline__ void add_rows(const T *src, int64_t ld, const uint32_t *perm, uint32_t p0, uint32_t p1,
                                         uint32_t g, uint32_t G, int col, bool on, float (&acc)[VEC]) {
  for (uint32_t p = p0 + g; p < p1; p += U * G) {
    float v[U][VEC];
    uint32_t at[U];
#pragma unroll
    for (int k = 0; k < U; k++) {
      const uint32_t q = p + k * G;
      at[k] = q < p1 ? (perm ? perm[q] : q) : 0u;
    }
#pragma unroll
    for (int k = 0; k < U; k++) {
#pragma unroll
      for (int j = 0; j < VEC; j++) v[k][j] = 0.0f;
      if (on && p + k * G < p1) {
        if constexpr (sizeof(T) == 4 && VEC == 8) load_sums<VEC>((const float *)src + (int64_t)at[k] * ld + col, v[k]);
        else load_f32<T, VEC>(src + (int64_t)at[k] * ld + col, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; k++)
#pragma unroll
      for (int j = 0; j < VEC; j++) acc[j] += v[k][j];
  }
}

// Sum over the wave's row lanes, the same in each of them afterwards.
template <int VEC>
__device__ __forceinline__ void join_row_lanes(float (&acc)[VEC], int lg) {
  for (int o = 1 << lg; o < 64; o <<= 1)
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] += __shfl_xor(acc[j], o);
}

// One wave per (chunk, slice): the bounds of the segments that begin or end in the
// chunk, and the chunk's sum if one row holds all of it.
template <typename T, int VEC>
__device__ __forceinline__ void chunk_sum(const SumArgs &a, uint32_t c, uint32_t slice, uint32_t lane) {
  const uint32_t p = c * CHUNK + lane;
  const uint32_t key = p < a.n ? a.keys[p] : a.rows;
  const uint32_t first = __shfl(key, 0), last = __shfl(key, 63);
  if (slice == 0 && key < a.rows) {
    if (p == 0 || a.keys[p - 1] != key) a.bounds[key].x = (int)p;
    if (p + 1 == a.n || a.keys[p + 1] != key) a.bounds[key].y = (int)p + 1;
  }
  if (first != last || first >= a.rows) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  const uint32_t G = 64u >> a.lg, g = lane >> a.lg;
  const int unit = (int)(slice << 6) + (int)(lane & ((1u << a.lg) - 1u));
  const bool on = unit < a.units;
  add_rows<T, VEC, 8>((const T *)a.dy, a.ldy, a.perm, c * CHUNK, c * CHUNK + CHUNK, g, G, unit * VEC, on, acc);
  join_row_lanes<VEC>(acc, a.lg);
  if (g == 0 && on) store_sums<VEC>(a.part1 + (size_t)c * a.dim + unit * VEC, acc);
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void k_chunk_sums(SumArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t waves = (uint64_t)((a.n + CHUNK - 1) / CHUNK) * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4)
    chunk_sum<T, VEC>(a, (uint32_t)(wv / (uint32_t)a.slices), (uint32_t)(wv % (uint32_t)a.slices), lane);
}
// The next level: one wave per (64 chunks, slice) that one row holds wholly.
template <int VEC>
__device__ __forceinline__ void chunk_sum2(const SumArgs &a, uint32_t c, uint32_t slice, uint32_t lane) {
  const uint32_t first = a.keys[c * (CHUNK * CHUNK)], last = a.keys[c * (CHUNK * CHUNK) + CHUNK * CHUNK - 1];
  if (first != last || first >= a.rows) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  const uint32_t G = 64u >> a.lg, g = lane >> a.lg;
  const int unit = (int)(slice << 6) + (int)(lane & ((1u << a.lg) - 1u));
  const bool on = unit < a.units;
  add_rows<float, VEC, 4>(a.part1, a.dim, nullptr, c * CHUNK, c * CHUNK + CHUNK, g, G, unit * VEC, on, acc);
  join_row_lanes<VEC>(acc, a.lg);
  if (g == 0 && on) store_sums<VEC>(a.part2 + (size_t)c * a.dim + unit * VEC, acc);
}

template <int VEC>
__global__ __launch_bounds__(256) void k_chunk_sums2(SumArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t waves = (uint64_t)(a.n / (CHUNK * CHUNK)) * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4)
    chunk_sum2<VEC>(a, (uint32_t)(wv / (uint32_t)a.slices), (uint32_t)(wv % (uint32_t)a.slices), lane);
}

template <typename T, int VEC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t row, int col, float (&acc)[VEC]) {
  T *o = (T *)a.grad + (int64_t)row * a.ldg + col;
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] *= a.scale;
  if (a.accumulate) {
    float old[VEC];
    load_f32<T, VEC>(o, old);
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] += old[j];
  }
  store_f32<T, VEC>(o, acc);
}

// Every row of the gradient. A wave holds 64 >> lg rows, one per row lane; a row of at
// most 64 tokens is summed by its own lanes, a longer one by the whole wave.
template <typename T, int VEC>
__device__ __forceinline__ void row_grads(const SumArgs &a, uint32_t row0, uint32_t slice, uint32_t lane) {
  const uint32_t G = 64u >> a.lg, g = lane >> a.lg, row = row0 + g;
  const int unit = (int)(slice << 6) + (int)(lane & ((1u << a.lg) - 1u));
  const bool on = unit < a.units;
  const int col = unit * VEC;
  const int2 b = row < a.rows ? a.bounds[row] : make_int2(0, 0);
  const T *dy = (const T *)a.dy;
  const bool heavy = b.y - b.x > CHUNK;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  if (!heavy) {
    add_rows<T, VEC, 4>(dy, a.ldy, a.perm, (uint32_t)b.x, (uint32_t)b.y, 0, 1, col, on, acc);
    if (row < a.rows && on && (b.y > b.x || !a.accumulate)) write_row<T, VEC>(a, row, col, acc);
  }
  uint64_t todo = ballot64(heavy);
  while (todo) {
    const uint32_t h = (uint32_t)__builtin_ctzll(todo) >> a.lg;
    todo &= a.lg == 6 ? 0ull : ~(((1ull << (1u << a.lg)) - 1ull) << (h << a.lg));
    const uint32_t s = (uint32_t)__shfl(b.x, (int)(h << a.lg)), e = (uint32_t)__shfl(b.y, (int)(h << a.lg));
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
    uint32_t c0 = (s + CHUNK - 1) / CHUNK, c1 = e / CHUNK;
    if (c0 >= c1) {
      add_rows<T, VEC, 4>(dy, a.ldy, a.perm, s, e, g, G, col, on, acc);
    } else {
      add_rows<T, VEC, 4>(dy, a.ldy, a.perm, s, c0 * CHUNK, g, G, col, on, acc);
      const uint32_t d0 = (c0 + CHUNK - 1) / CHUNK, d1 = c1 / CHUNK;
      if (!a.two_levels || d0 >= d1) {
        add_rows<float, VEC, 4>(a.part1, a.dim, nullptr, c0, c1, g, G, col, on, acc);
      } else {
        add_rows<float, VEC, 4>(a.part1, a.dim, nullptr, c0, d0 * CHUNK, g, G, col, on, acc);
        add_rows<float, VEC, 4>(a.part2, a.dim, nullptr, d0, d1, g, G, col, on, acc);
        add_rows<float, VEC, 4>(a.part1, a.dim, nullptr, d1 * CHUNK, c1, g, G, col, on, acc);
      }
      add_rows<T, VEC, 4>(dy, a.ldy, a.perm, c1 * CHUNK, e, g, G, col, on, acc);
    }
    join_row_lanes<VEC>(acc, a.lg);
    if (g == 0 && on) write_row<T, VEC>(a, row0 + h, col, acc);
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void k_row_grads(SumArgs a) {
  const uint32_t lane = threadIdx.x & 63, G = 64u >> a.lg;
  const uint64_t waves = (uint64_t)((a.rows + G - 1) / G) * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4)
    row_grads<T, VEC>(a, (uint32_t)(wv / (uint32_t)a.slices) * G, (uint32_t)(wv % (uint32_t)a.slices), lane);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename T, int VEC, typename ID>
int run_lookup(const void *table, int64_t ldt, int64_t rows, int dim, const void *ids, int64_t n, float scale,
               void *out, int64_t ldo, hipStream_t stream) {
  const uint32_t units = (uint32_t)(dim / VEC);
  const FastDiv fd = fast_div(units);
  // the kernel's unit index has 31 bits: more tokens take more launches
  const int64_t step = ((1ll << 31) - 1) / units;
  for (int64_t i = 0; i < n; i += step) {
    const int64_t m = n - i < step ? n - i : step;
    const uint32_t total = (uint32_t)(m * units);
    const unsigned per = LK_THREADS * LK_ITEMS;
    hipLaunchKernelGGL((k_lookup<T, VEC, ID>), dim3((total + per - 1) / per), dim3(LK_THREADS), 0, stream,
                       (const T *)table, ldt, rows, (const ID *)ids + i, total, fd, scale, (T *)out + i * ldo, ldo);
    SPLAT_LAUNCH_CHECK();
  }
  return SPLAT_OK;
}

struct BwdLayout {
  uint32_t *keys[2], *perm[2], *counts, *totals;
  int2 *bounds;
  float *part1, *part2;
  size_t bytes;
};

BwdLayout bwd_layout(void *base, int64_t n, int64_t rows, int dim) {
  BwdLayout L;
  char *p = (char *)base;
  auto take = [&](size_t b) {
    char *q = p;
    p += ws_align(b);
    return (void *)q;
  };
  const size_t tiles = (size_t)((n + ST_TILE - 1) / ST_TILE);
  for (int k = 0; k < 2; k++) {
    L.keys[k] = (uint32_t *)take(4 * (size_t)n);
    L.perm[k] = (uint32_t *)take(4 * (size_t)n);
  }
  L.counts = (uint32_t *)take(4 * RADIX * tiles);
  L.totals = (uint32_t *)take(4 * RADIX);
  L.bounds = (int2 *)take(8 * (size_t)rows);
  L.part1 = (float *)take(4 * (size_t)(n / CHUNK) * dim);
  L.part2 = (float *)take(4 * (size_t)(n / (CHUNK * CHUNK)) * dim);
  L.bytes = (size_t)(p - (char *)base);
  return L;
}

// Workgroups of four waves, few enough that threads count below 2^32.
unsigned wave_grid(uint64_t waves) {
  const uint64_t b = (waves + 3) / 4;
  return (unsigned)(b < (1u << 22) ? b : (1u << 22));
}

// Sorts the tokens by id: keys and tokens end in the returned half of the workspace.
template <typename ID>
int sort_tokens(const void *ids, uint32_t n, uint32_t rows, const BwdLayout &L, int *half, hipStream_t stream) {
  int bits = 1;
  while (bits < 32 && (rows >> bits)) bits++;        // keys 0 .. rows
  const int passes = (bits + RADIX_BITS - 1) / RADIX_BITS;
  if (n <= ST_TILE) {
    unsigned clear = (rows + 4 * SM_THREADS - 1) / (4 * SM_THREADS);
    clear = clear > 1024 ? 1024 : clear;
    hipLaunchKernelGGL((k_sort_small<ID>), dim3(1 + clear), dim3(SM_THREADS), 0, stream, (const ID *)ids, n, rows,
                       bits, passes, L.keys[0], L.perm[0], L.bounds);
    SPLAT_LAUNCH_CHECK();
    *half = 0;
    return SPLAT_OK;
  }
  const uint32_t tiles = (n + ST_TILE - 1) / ST_TILE;
  const int dbits = (bits + passes - 1) / passes;
  for (int p = 0; p < passes; p++) {
    KeySource<ID> src;
    src.ids = (const ID *)ids;
    src.keys = p ? L.keys[(p - 1) & 1] : nullptr;
    src.perm = p ? L.perm[(p - 1) & 1] : nullptr;
    src.n = n;
    src.rows = rows;
    const int shift = p * dbits, b = bits - shift < dbits ? bits - shift : dbits;
    hipLaunchKernelGGL((k_sort_count<ID>), dim3(tiles), dim3(ST_THREADS), 0, stream, src, shift, b, tiles, L.counts,
                       p ? (int2 *)nullptr : L.bounds, rows);
    SPLAT_LAUNCH_CHECK();
    hipLaunchKernelGGL(k_sort_scan, dim3(1u << b), dim3(ST_THREADS), 0, stream, L.counts, tiles, L.totals);
    SPLAT_LAUNCH_CHECK();
    hipLaunchKernelGGL((k_sort_scatter<ID>), dim3(tiles), dim3(ST_THREADS), 0, stream, src, shift, b, tiles, L.counts,
                       L.totals, L.keys[p & 1], L.perm[p & 1]);
    SPLAT_LAUNCH_CHECK();
  }
  *half = (passes - 1) & 1;
  return SPLAT_OK;
}

// Every row zero: no token to add.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void k_zero_rows(T *grad, int64_t ldg, uint64_t total, uint32_t units) {
  const float z[VEC] = {};
  for (uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (uint64_t)gridDim.x * 256) {
    const uint64_t r = u / units;
    store_f32<T, VEC>(grad + (int64_t)r * ldg + (int64_t)(u - r * units) * VEC, z);
  }
}

template <typename T, int VEC>
int run_lookup_bwd(SumArgs a, const void *ids, int id_type, void *ws, hipStream_t stream) {
  a.units = a.dim / VEC;
  if (a.n == 0) {
    if (a.accumulate) return SPLAT_OK;
    const uint64_t total = (uint64_t)a.rows * a.units;
    const uint64_t blocks = (total + 255) / 256;
    hipLaunchKernelGGL((k_zero_rows<T, VEC>), dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream,
                       (T *)a.grad, a.ldg, total, (uint32_t)a.units);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  const BwdLayout L = bwd_layout(ws, a.n, a.rows, a.dim);
  int half = 0;
  const int st = id_type == SPLAT_I64 ? sort_tokens<int64_t>(ids, a.n, a.rows, L, &half, stream)
                                      : sort_tokens<int32_t>(ids, a.n, a.rows, L, &half, stream);
  if (st) return st;
  a.keys = L.keys[half];
  a.perm = L.perm[half];
  a.bounds = L.bounds;
  a.part1 = L.part1;
  a.part2 = L.part2;
  a.lg = 0;
  while (a.lg < 6 && (1 << a.lg) < a.units) a.lg++;
  a.slices = (a.units + 63) / 64;
  const uint64_t w1 = (uint64_t)((a.n + CHUNK - 1) / CHUNK) * a.slices;
  hipLaunchKernelGGL((k_chunk_sums<T, VEC>), dim3(wave_grid(w1)), dim3(256), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  // below two whole second-level chunks a row has at most 128 first-level sums: not worth a launch
  a.two_levels = a.n >= 2 * CHUNK * CHUNK;
  if (a.two_levels) {
    const uint64_t w2 = (uint64_t)(a.n / (CHUNK * CHUNK)) * a.slices;
    hipLaunchKernelGGL((k_chunk_sums2<VEC>), dim3(wave_grid(w2)), dim3(256), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
  }
  const uint32_t G = 64u >> a.lg;
  const uint64_t wr = (uint64_t)((a.rows + G - 1) / G) * a.slices;
  hipLaunchKernelGGL((k_row_grads<T, VEC>), dim3(wave_grid(wr)), dim3(256), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

}  // namespace

int launch_lookup(const void *table, int dtype, int64_t rows, int dim, int64_t ldt, const void *ids, int id_type,
                  int64_t n, float scale, void *out, int64_t ldo, hipStream_t stream) {
  if (n == 0 || dim == 0) return SPLAT_OK;
  const int64_t strides[2] = {ldt, ldo};
  const void *ptrs[2] = {table, out};
  const int vec = vec_width(dtype_bytes(dtype), dim, strides, 2, ptrs, 2);
#define GO(T, V)                                                                                              \
  return id_type == SPLAT_I64 ? run_lookup<T, V, int64_t>(table, ldt, rows, dim, ids, n, scale, out, ldo, stream) \
                              : run_lookup<T, V, int32_t>(table, ldt, rows, dim, ids, n, scale, out, ldo, stream)
#define BY_VEC(T)        \
  switch (vec) {         \
    case 8: GO(T, 8);    \
    case 4: GO(T, 4);    \
    case 2: GO(T, 2);    \
    default: GO(T, 1);   \
  }
  if (dtype == SPLAT_F16) { BY_VEC(f16_t) }
  if (dtype == SPLAT_BF16) { BY_VEC(bf16_t) }
  switch (vec) {
    case 4: GO(float, 4);
    case 2: GO(float, 2);
    default: GO(float, 1);
  }
#undef GO
}

size_t lookup_bwd_workspace_bytes(int64_t n, int64_t rows, int dim) { return bwd_layout(nullptr, n, rows, dim).bytes; }

int launch_lookup_bwd(const void *d_out, int dtype, int64_t ldy, const void *ids, int id_type, int64_t n, int64_t rows,
                      int dim, float scale, void *d_table, int64_t ldg, int accumulate, void *ws, hipStream_t stream) {
  if (rows == 0 || dim == 0) return SPLAT_OK;
  SumArgs a = {};
  a.dy = d_out; a.ldy = ldy; a.grad = d_table; a.ldg = ldg;
  a.n = (uint32_t)n; a.rows = (uint32_t)rows; a.dim = dim; a.scale = scale; a.accumulate = accumulate;
  const int64_t strides[2] = {ldy, ldg};
  const void *ptrs[2] = {n ? d_out : d_table, d_table};
  const int vec = vec_width(dtype_bytes(dtype), dim, strides, 2, ptrs, 2);
#define GO(T, V) return run_lookup_bwd<T, V>(a, ids, id_type, ws, stream)
  if (dtype == SPLAT_F16) { BY_VEC(f16_t) }
  if (dtype == SPLAT_BF16) { BY_VEC(bf16_t) }
  switch (vec) {
    case 4: GO(float, 4);
    case 2: GO(float, 2);
    default: GO(float, 1);
  }
#undef GO
#undef BY_VEC
}
