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
//      tile of 1024 or 4096 tokens, a scan per digit, a scatter that ranks equal digits
//      within a wave by ballots (few tokens: one launch that counts and scatters);
//   2. the sorted list is cut into chunks of 64; a chunk that lies within one row's
//      segment is summed to one fp32 row, and 64 such sums to one of the next level;
//   3. each row is written by adding its tokens, or its loose tokens and whole chunks.
// So a row that holds all n tokens costs no lane more than 4 x 64 + n / 4096 adds. Few
// tokens in few rows skip all of this (k_few_grads).
#include "learn_common.h"

namespace {

constexpr int LK_THREADS = 256;
constexpr int LK_ITEMS = 4;
constexpr int ST_THREADS = 256;              // sort tiles: 4 or 16 tokens a thread
constexpr int ST_WAVES = ST_THREADS / WAVE;
constexpr int RADIX_BITS = 9, RADIX = 1 << RADIX_BITS;
constexpr int CHUNK = 64;
// Tokens up to which a sorting workgroup counts every tile's keys itself: a launch instead
// of three for a digit, of a longer chain. Gradient of fp32 rows of 32 in us: 8192 tokens,
// 65536 rows, even ids 31 (36 with counts of their own), skewed 35 (39), all alike 36 (34);
// 16384 tokens, 200000 rows 40 (37), 46 (42), 52 (36); 4096 x 16 fp16, 1M rows 34 (47).
constexpr uint32_t COUNT_ALONE = 8192;
// Tokens up to which tiles are small: more workgroups for the same chain of rankings.
constexpr int64_t SMALL_TILES = 256 << 10;
constexpr int tile_items(int64_t n) { return n <= SMALL_TILES ? 4 : 16; }

// A row of any length at any address is walked in packs of VEC elements, the last of which
// ends with the row: it overlaps the one before by what is missing. Both compute the
// overlap alike and write the same values (sums that are added to what a row holds take
// packs that divide it instead).
__device__ __forceinline__ uint32_t col_of(uint32_t col, uint32_t dim, uint32_t vec) {
  return col + vec <= dim ? col : dim - vec;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, int VEC, typename ID>
__global__ __launch_bounds__(LK_THREADS) void k_lookup(const T *__restrict__ table, int64_t ldt, int64_t rows,
                                                       const ID *__restrict__ ids, uint32_t total, FastDiv units,
                                                       uint32_t dim, float scale, T *__restrict__ out, int64_t ldo) {
  const uint32_t base = blockIdx.x * (LK_THREADS * LK_ITEMS) + threadIdx.x;
  uint32_t row[LK_ITEMS], col[LK_ITEMS];
  ID id[LK_ITEMS];
  Raw<T, VEC> x[LK_ITEMS];
#pragma unroll
  for (int k = 0; k < LK_ITEMS; k++) {
    const uint32_t u = base + k * LK_THREADS;
    row[k] = div_by(u, units);
    col[k] = col_of((u - row[k] * units.d) * VEC, dim, VEC);
    id[k] = -1;
    if (u < total) id[k] = ids[row[k]];
  }
#pragma unroll
  for (int k = 0; k < LK_ITEMS; k++)
    x[k] = load_loose_if<T, VEC>(id[k] >= 0 && (int64_t)id[k] < rows, table + (int64_t)id[k] * ldt + col[k]);
#pragma unroll
  for (int k = 0; k < LK_ITEMS; k++)
    if (base + k * LK_THREADS < total) {
      float v[VEC];
      to_f32<T, VEC>(x[k], v);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] *= scale;
      stream_loose<T, VEC>(out + (int64_t)row[k] * ldo + col[k], v);
    }
}

// ---------------------------------------------------------------------------
// sort by id
// ---------------------------------------------------------------------------
// A token's key: its id, or `rows` (after every row) where the id is outside.
__device__ __forceinline__ uint32_t key_of(int64_t id, uint32_t rows) {
  return id >= 0 && id < (int64_t)rows ? (uint32_t)id : rows;
}

// A pass's (key, token) pairs: from the caller's ids in the first pass, from the
// workspace after. `word` is what is loaded; `pair` forms the pair once all are under way
// (a compare next to its load, under the load's condition, would wait for that load).
template <typename ID, bool FIRST>
struct KeySource;
template <typename ID>
struct KeySource<ID, true> {
  const ID *from;
  uint32_t n, rows;
  typedef ID Word;
  __device__ Word word(uint32_t i) const {
    ID x = -1;
    if (i < n) x = from[i];
    return x;
  }
  __device__ uint2 pair(Word x, uint32_t i) const { return make_uint2(key_of((int64_t)x, rows), i); }
};
template <typename ID>
struct KeySource<ID, false> {
  const uint2 *from;
  uint32_t n, rows;
  typedef uint2 Word;
  __device__ Word word(uint32_t i) const {
    uint2 x = make_uint2(0u, 0u);
    if (i < n) x = from[i];
    return x;
  }
  __device__ uint2 pair(Word x, uint32_t) const { return x; }
};

// Rows without tokens keep empty bounds. Workgroup `block` of `blocks`.
__device__ __forceinline__ void clear_bounds(int2 *bounds, uint32_t nbounds, uint32_t block, uint32_t blocks) {
  for (uint64_t r = block * ST_THREADS + threadIdx.x; r < nbounds; r += blocks * ST_THREADS) bounds[r] = make_int2(0, 0);
}

// counts[tile][digit]; workgroups past the tiles clear the rows' segment bounds.
template <typename ID, bool FIRST, int ITEMS>
__global__ __launch_bounds__(ST_THREADS) void k_sort_count(KeySource<ID, FIRST> src, int shift, int bits,
                                                           uint32_t *__restrict__ counts, uint32_t tiles,
                                                           int2 *bounds, uint32_t nbounds) {
  if (blockIdx.x >= tiles) {
    clear_bounds(bounds, nbounds, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  __shared__ uint32_t h[RADIX];
  for (int d = threadIdx.x; d < RADIX; d += ST_THREADS) h[d] = 0;
  const uint32_t mask = (1u << bits) - 1u, i0 = blockIdx.x * (uint32_t)(ST_THREADS * ITEMS) + threadIdx.x;
  typename KeySource<ID, FIRST>::Word word[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; j++) word[j] = src.word(i0 + j * ST_THREADS);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
    if (i0 + j * ST_THREADS < src.n) atomicAdd(&h[(src.pair(word[j], 0).x >> shift) & mask], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < (1 << bits); d += ST_THREADS) counts[((size_t)blockIdx.x << bits) + d] = h[d];
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

// Exclusive scan of each digit's counts over the tiles, and its total. A workgroup takes 16
// digits, a thread one of them and 8 tiles at a time, so that it reads whole 64-byte runs
// (a digit's counts side by side, as the scan alone would like, made every tile write and
// read 512 scattered words).
constexpr int SC_THREADS = 1024, SC_DIGITS = 16, SC_LANES = SC_THREADS / SC_DIGITS, SC_TILES = 8;
__global__ __launch_bounds__(SC_THREADS) void k_sort_scan(uint32_t *__restrict__ counts, uint32_t tiles, uint32_t digits,
                                                          uint32_t *__restrict__ totals) {
  __shared__ uint32_t s[SC_LANES][SC_DIGITS];
  const uint32_t dl = threadIdx.x % SC_DIGITS, tl = threadIdx.x / SC_DIGITS, d = blockIdx.x * SC_DIGITS + dl;
  uint32_t carry = 0;
  for (uint32_t t0 = 0; t0 < tiles; t0 += SC_LANES * SC_TILES) {
    uint32_t c[SC_TILES], sum = 0;
#pragma unroll
    for (int k = 0; k < SC_TILES; k++) {
      const uint32_t t = t0 + tl * SC_TILES + k;
      c[k] = 0;
      if (t < tiles && d < digits) c[k] = counts[(size_t)t * digits + d];
    }
#pragma unroll
    for (int k = 0; k < SC_TILES; k++) sum += c[k];
    __syncthreads();
    s[tl][dl] = sum;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll 8
    for (uint32_t k = 0; k < SC_LANES; k++) {
      const uint32_t v = s[k][dl];
      if (k < tl) before += v;
      all += v;
    }
    uint32_t run = carry + before;
#pragma unroll
    for (int k = 0; k < SC_TILES; k++) {
      const uint32_t t = t0 + tl * SC_TILES + k;
      if (t < tiles && d < digits) counts[(size_t)t * digits + d] = run;
      run += c[k];
    }
    carry += all;
  }
  if (tl == 0 && d < digits) totals[d] = carry;
}

// Rank of this lane's digit among the wave's items so far, adding the wave's items to
// hist (this wave's counters). Lanes with equal digits find each other by one ballot
// per bit; the lowest of them updates the counter. Inactive lanes pass ok = false.
typedef volatile __attribute__((address_space(3))) uint32_t *LdsCounters;
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, int bits, bool ok, LdsCounters hist) {
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

// The tile's pairs are put in digit order in LDS first, so that a wave's store covers a
// few runs of consecutive pairs instead of 64 places.
// COUNTS: a workgroup counts all keys for itself, and the pass is one launch; workgroups
// past the tiles clear the rows' bounds.
template <typename ID, bool FIRST, int ITEMS, bool COUNTS>
__global__ __launch_bounds__(ST_THREADS) void k_sort_scatter(KeySource<ID, FIRST> src, int shift, int bits,
                                                             const uint32_t *__restrict__ counts,
                                                             const uint32_t *__restrict__ totals,
                                                             uint2 *__restrict__ out, uint32_t tiles, int2 *bounds,
                                                             uint32_t nbounds) {
  constexpr int ST_TILE = ST_THREADS * ITEMS;
  if (COUNTS && blockIdx.x >= tiles) {
    clear_bounds(bounds, nbounds, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  __shared__ uint32_t hist[ST_WAVES][RADIX];   // a wave's counts, then its first place in the tile, per digit
  __shared__ uint32_t away[RADIX];             // a digit's first place in the output less that in the tile
  __shared__ uint2 tile[ST_TILE];
  __shared__ uint32_t s[ST_WAVES];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int d = threadIdx.x; d < ST_WAVES * RADIX; d += ST_THREADS) (&hist[0][0])[d] = 0;
  const uint32_t mask = (1u << bits) - 1u, t0 = blockIdx.x * (uint32_t)ST_TILE;
  const uint32_t i0 = t0 + w * (ST_TILE / ST_WAVES) + lane;
  typename KeySource<ID, FIRST>::Word word[ITEMS];
  uint2 pair[ITEMS];
  uint32_t rank[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; j++) word[j] = src.word(i0 + j * WAVE);
  constexpr int DPT = RADIX / ST_THREADS;
  uint32_t tot[DPT], cnt[DPT], sum = 0, all;
  if (COUNTS) {
    // keys of the tiles before this one, and of the others
    __shared__ uint32_t h[2][RADIX];
    for (int d = threadIdx.x; d < 2 * RADIX; d += ST_THREADS) (&h[0][0])[d] = 0;
    __syncthreads();
    constexpr int FLIGHT = 8;
    for (uint32_t i = threadIdx.x; i < src.n; i += ST_THREADS * FLIGHT) {
      typename KeySource<ID, FIRST>::Word x[FLIGHT];
#pragma unroll
      for (int j = 0; j < FLIGHT; j++) x[j] = src.word(i + j * ST_THREADS);
#pragma unroll
      for (int j = 0; j < FLIGHT; j++)
        if (i + j * ST_THREADS < src.n)
          atomicAdd(&h[i + j * ST_THREADS >= t0][(src.pair(x[j], 0).x >> shift) & mask], 1u);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < DPT; k++) {
      cnt[k] = h[0][threadIdx.x * DPT + k];
      tot[k] = cnt[k] + h[1][threadIdx.x * DPT + k];
      sum += tot[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < DPT; k++) {
      const uint32_t d = threadIdx.x * DPT + k;
      tot[k] = d <= mask ? totals[d] : 0u;
      cnt[k] = d <= mask ? counts[((size_t)blockIdx.x << bits) + d] : 0u;
      sum += tot[k];
    }
  }
#pragma unroll
  for (int j = 0; j < ITEMS; j++) pair[j] = src.pair(word[j], i0 + j * WAVE);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
    rank[j] = wave_rank((pair[j].x >> shift) & mask, bits, i0 + j * WAVE < src.n, (LdsCounters)hist[w]);
  // first places: in the output, after the smaller digits of all tiles and the digit's
  // earlier tiles; in the tile, after its smaller digits and the digit's earlier waves
  uint32_t at = block_scan<ST_WAVES>(sum, s, &all) - sum;   // its barriers also end the ranking
  uint32_t mine = 0;
#pragma unroll
  for (int k = 0; k < DPT; k++)
#pragma unroll
    for (int v = 0; v < ST_WAVES; v++) mine += hist[v][threadIdx.x * DPT + k];
  uint32_t in_tile = block_scan<ST_WAVES>(mine, s, &all) - mine;
#pragma unroll
  for (int k = 0; k < DPT; k++) {
    const uint32_t d = threadIdx.x * DPT + k;
    away[d] = at + cnt[k] - in_tile;
    at += tot[k];
#pragma unroll
    for (int v = 0; v < ST_WAVES; v++) {
      const uint32_t c = hist[v][d];
      hist[v][d] = in_tile;
      in_tile += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
    if (i0 + j * WAVE < src.n) tile[hist[w][(pair[j].x >> shift) & mask] + rank[j]] = pair[j];
  __syncthreads();
  const uint32_t m = src.n - t0 < ST_TILE ? src.n - t0 : ST_TILE;
#pragma unroll
  for (int j = 0; j < ITEMS; j++) {
    const uint32_t i = j * ST_THREADS + threadIdx.x;
    if (i < m) {
      const uint2 v = tile[i];
      out[away[(v.x >> shift) & mask] + i] = v;
    }
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
// How a wave covers a row of `units` packs: 2^lg lanes per row (64 if the row has 64
// packs or more, then one slice of 64 packs per wave), so G = 64 >> lg rows at once.
struct SumArgs {
  const void *dy;
  int64_t ldy;
  const uint2 *sorted;      // (row, token) by row, then token
  int2 *bounds;             // [rows] segment of each row in `sorted`, (0, 0) without tokens
  float *part1, *part2;     // sums of whole chunks of 64 and of 64 x 64 tokens [.][width]
  void *grad;
  int64_t ldg;
  uint32_t n, rows, chunks;
  int dim, width, units, lg, slices, two_levels, accumulate;   // width: units x VEC, a chunk sum's length
  float scale;
};

// This lane's place in a wave's share of the work.
struct Place {
  uint32_t lane, g, G;      // row lane and row lanes per wave
  int col, sum;             // first column of its pack, and the pack's place in a chunk sum
  bool on;
};
template <int VEC>
__device__ __forceinline__ Place place_of(const SumArgs &a, uint32_t slice) {
  Place q;
  q.lane = threadIdx.x & 63;
  q.G = 64u >> a.lg;
  q.g = q.lane >> a.lg;
  const int unit = (int)(slice << a.lg) + (int)(q.lane & ((1u << a.lg) - 1u));
  q.on = unit < a.units;
  q.sum = unit * VEC;
  q.col = (int)col_of((uint32_t)q.sum, (uint32_t)a.dim, VEC);
  return q;
}

// Adds rows p0 .. p1 of `src` to acc, the wave's G row lanes in turn, U loads in flight
// each; the rows are those of chunk sums, in order.
template <int VEC, int U>
__device__ __forceinline__ void add_sums(const float *src, int64_t ld, uint32_t p0, uint32_t p1, const Place &q,
                                         float (&acc)[VEC]) {
  for (uint32_t p = p0 + q.g; p < p1; p += U * q.G) {
    float v[U][VEC];
#pragma unroll
    for (int k = 0; k < U; k++) {
#pragma unroll
      for (int j = 0; j < VEC; j++) v[k][j] = 0.0f;
      if (q.on && p + k * q.G < p1) load_sums<VEC>(src + (int64_t)(p + k * q.G) * ld + q.sum, v[k]);
    }
#pragma unroll
    for (int k = 0; k < U; k++)
#pragma unroll
      for (int j = 0; j < VEC; j++) acc[j] += v[k][j];
  }
}

// Adds the rows of dy of sorted tokens [p0, p1) to acc, the wave's G row lanes in turn.
// The lanes fetch 64 token numbers at once and pass them round, so that only the rows
// themselves are waited for. Every lane of the wave calls it.
template <typename T, int VEC, int U>
__device__ __forceinline__ void add_tokens(const SumArgs &a, uint32_t p0, uint32_t p1, const Place &q, float (&acc)[VEC]) {
  const T *dy = (const T *)a.dy + q.col;
  for (uint32_t b = p0; b < p1; b += 64) {
    const uint32_t m = p1 - b < 64u ? p1 - b : 64u;
    const uint32_t tok = q.lane < m ? a.sorted[b + q.lane].y : 0u;
    for (uint32_t k0 = 0; k0 < m; k0 += U * q.G) {
      Raw<T, VEC> x[U];
#pragma unroll
      for (int k = 0; k < U; k++) {
        const uint32_t t = k0 + k * q.G + q.g;
        const uint32_t at = __shfl(tok, (int)(t & 63u));
        x[k] = load_loose_if<T, VEC>(q.on && t < m, dy + (int64_t)at * a.ldy);
      }
#pragma unroll
      for (int k = 0; k < U; k++) {
        float v[VEC];
        to_f32<T, VEC>(x[k], v);
#pragma unroll
        for (int j = 0; j < VEC; j++) acc[j] += v[j];
      }
    }
  }
}

// Sum over the wave's row lanes, the same in each of them afterwards.
template <int VEC>
__device__ __forceinline__ void join_row_lanes(float (&acc)[VEC], int lg) {
  for (int o = 1 << lg; o < 64; o <<= 1)
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] += __shfl_xor(acc[j], o);
}

// Row loads in flight per lane (16: 30 -> 35 us for the chunk sums of 2M x 32 fp32).
constexpr int DEEP = 8;

// One wave per (chunk, slice): the bounds of the segments that begin or end in the
// chunk, and the chunk's sum if one row holds all of it.
template <typename T, int VEC>
__device__ __forceinline__ void chunk_sum(const SumArgs &a, uint32_t c, uint32_t slice) {
  const Place q = place_of<VEC>(a, slice);
  const uint32_t p = c * CHUNK + q.lane;
  const uint32_t key = p < a.n ? a.sorted[p].x : a.rows;
  const uint32_t first = __shfl(key, 0), last = __shfl(key, 63);
  if (slice == 0 && key < a.rows) {
    if (p == 0 || a.sorted[p - 1].x != key) a.bounds[key].x = (int)p;
    if (p + 1 == a.n || a.sorted[p + 1].x != key) a.bounds[key].y = (int)p + 1;
  }
  if (first != last || first >= a.rows) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  add_tokens<T, VEC, DEEP>(a, c * CHUNK, c * CHUNK + CHUNK, q, acc);
  join_row_lanes<VEC>(acc, a.lg);
  if (q.g == 0 && q.on) store_sums<VEC>(a.part1 + (size_t)c * a.width + q.sum, acc);
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void k_chunk_sums(SumArgs a) {
  const uint64_t waves = (uint64_t)a.chunks * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4)
    chunk_sum<T, VEC>(a, (uint32_t)(wv / (uint32_t)a.slices), (uint32_t)(wv % (uint32_t)a.slices));
}

// The next level: one wave per (64 chunks, slice) that one row holds wholly.
template <int VEC>
__device__ __forceinline__ void chunk_sum2(const SumArgs &a, uint32_t c, uint32_t slice) {
  const Place q = place_of<VEC>(a, slice);
  const uint32_t first = a.sorted[c * (CHUNK * CHUNK)].x, last = a.sorted[c * (CHUNK * CHUNK) + CHUNK * CHUNK - 1].x;
  if (first != last || first >= a.rows) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  add_sums<VEC, DEEP>(a.part1, a.width, c * CHUNK, c * CHUNK + CHUNK, q, acc);
  join_row_lanes<VEC>(acc, a.lg);
  if (q.g == 0 && q.on) store_sums<VEC>(a.part2 + (size_t)c * a.width + q.sum, acc);
}

template <int VEC>
__global__ __launch_bounds__(256) void k_chunk_sums2(SumArgs a) {
  const uint64_t waves = (uint64_t)(a.n / (CHUNK * CHUNK)) * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4)
    chunk_sum2<VEC>(a, (uint32_t)(wv / (uint32_t)a.slices), (uint32_t)(wv % (uint32_t)a.slices));
}

template <typename T, int VEC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t row, int col, float (&acc)[VEC]) {
  T *o = (T *)a.grad + (int64_t)row * a.ldg + col;
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] *= a.scale;
  if (a.accumulate) {
    float old[VEC];
    to_f32<T, VEC>(load_loose_if<T, VEC>(true, o), old);
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] += old[j];
  }
  stream_loose<T, VEC>(o, acc);
}

// A row of more than 64 tokens, by a wave: its segment holds a multiple of 64, and the
// first one's chunk stands for the row. Loose tokens at both ends, whole chunks between.
template <typename T, int VEC>
__device__ __forceinline__ void heavy_row(const SumArgs &a, uint32_t c, uint32_t slice) {
  const uint32_t row = a.sorted[c * CHUNK].x;
  if (row >= a.rows) return;
  const int2 b = a.bounds[row];
  const uint32_t s = (uint32_t)b.x, e = (uint32_t)b.y;
  if (e - s <= CHUNK || (s + CHUNK - 1) / CHUNK != c) return;
  const Place q = place_of<VEC>(a, slice);
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
  const uint32_t c1 = e / CHUNK;
  add_tokens<T, VEC, DEEP>(a, s, c * CHUNK, q, acc);
  const uint32_t d0 = (c + CHUNK - 1) / CHUNK, d1 = c1 / CHUNK;
  if (!a.two_levels || d0 >= d1) {
    add_sums<VEC, DEEP>(a.part1, a.width, c, c1, q, acc);
  } else {
    add_sums<VEC, DEEP>(a.part1, a.width, c, d0 * CHUNK, q, acc);
    add_sums<VEC, DEEP>(a.part2, a.width, d0, d1, q, acc);
    add_sums<VEC, DEEP>(a.part1, a.width, d1 * CHUNK, c1, q, acc);
  }
  add_tokens<T, VEC, DEEP>(a, c1 * CHUNK, e, q, acc);
  join_row_lanes<VEC>(acc, a.lg);
  if (q.g == 0 && q.on) write_row<T, VEC>(a, row, q.col, acc);
}

// Rows of at most 64 tokens, SETS sets of G in a wave: a set at a time, each row by its
// own lanes. The bounds of all sets are fetched at once, so that rows without tokens wait
// for nothing else. A wave's sets lie far apart, because neighbouring ids are often
// alike: frequent ones come first in many tables.
template <typename T, int VEC, int SETS>
__device__ __forceinline__ void light_rows(const SumArgs &a, uint32_t set, uint32_t stride, uint32_t slice) {
  const Place q = place_of<VEC>(a, slice);
  int2 b[SETS];
#pragma unroll
  for (int u = 0; u < SETS; u++) {
    const uint64_t row = ((uint64_t)set + (uint64_t)u * stride) * q.G + q.g;
    b[u] = row < a.rows ? a.bounds[row] : make_int2(0, CHUNK + 1);
  }
#pragma unroll
  for (int u = 0; u < SETS; u++) {
    const uint32_t s = (uint32_t)b[u].x, e = (uint32_t)b[u].y;
    if (e - s > CHUNK) continue;                   // another wave's, or past the end
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
    constexpr int U = 8;
    for (uint32_t p = s; p < e; p += U) {
      Raw<T, VEC> x[U];
      uint32_t at[U];
#pragma unroll
      for (int k = 0; k < U; k++) at[k] = p + k < e ? a.sorted[p + k].y : 0u;
#pragma unroll
      for (int k = 0; k < U; k++)
        x[k] = load_loose_if<T, VEC>(q.on && p + k < e, (const T *)a.dy + (int64_t)at[k] * a.ldy + q.col);
#pragma unroll
      for (int k = 0; k < U; k++) {
        float v[VEC];
        to_f32<T, VEC>(x[k], v);
#pragma unroll
        for (int j = 0; j < VEC; j++) acc[j] += v[j];
      }
    }
    if (q.on && (e > s || !a.accumulate)) write_row<T, VEC>(a, (set + u * stride) * q.G + q.g, q.col, acc);
  }
}

// Every row of the gradient: first the waves that look for heavy rows, one per chunk and
// slice, then those of the light rows.
template <typename T, int VEC, int SETS>
__global__ __launch_bounds__(256) void k_row_grads(SumArgs a) {
  const uint32_t G = 64u >> a.lg, sets = (a.rows + G - 1) / G, stride = (sets + SETS - 1) / SETS;
  const uint64_t heavy = a.n > CHUNK ? (uint64_t)a.chunks * a.slices : 0;
  const uint64_t waves = heavy + (uint64_t)stride * a.slices;
  for (uint64_t wv = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); wv < waves; wv += (uint64_t)gridDim.x * 4) {
    if (wv < heavy) {
      heavy_row<T, VEC>(a, (uint32_t)(wv / (uint32_t)a.slices), (uint32_t)(wv % (uint32_t)a.slices));
    } else {
      const uint64_t v = wv - heavy;
      light_rows<T, VEC, SETS>(a, (uint32_t)(v / (uint32_t)a.slices), stride, (uint32_t)(v % (uint32_t)a.slices));
    }
  }
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
// The whole gradient in one launch for up to FEW tokens: a workgroup owns a run of rows
// (and a slice of 64 packs), keeps the tokens whose ids fall in it, in order, in LDS, and
// sums row by row. Short lists go a row to a wave; long ones (many tokens in few rows) a
// row to the whole workgroup, each wave taking every eighth part of 64 entries. Nothing is
// sorted, and no workspace is needed. What bounds it is its chain of waits: ids, rows,
// stores.
// Every row of a run walks the run's whole list, so the rule bounds a run's rows times its
// tokens. In us, even and skewed ids, here and sorted: 4096 tokens in 8000 rows x 64 fp32 10
// and 16 (25 and 29), 1000 in 4000 x 16 fp16 10 and 10 (23 and 30); past the rule 4096 in
// 60000 x 32 fp32 14 and 94 (25 and 27), 1000 in 1M x 16 fp16 103 and 975 (28 and 33).
constexpr int FW_THREADS = 512, FW_WAVES = FW_THREADS / WAVE, FW_ITEMS = 8;
constexpr int64_t FEW = FW_THREADS * FW_ITEMS;
constexpr int FW_LONG = 256;               // entries from which the workgroup works together
constexpr int64_t FW_RUNS = 1024;          // runs of rows, at most
constexpr int64_t few_run(int64_t rows) { return (rows + FW_RUNS - 1) / FW_RUNS; }
constexpr bool few_tokens(int64_t n, int64_t rows) { return n <= FEW && few_run(rows) * (n + 1024) <= 65536; }

// Adds the rows of the tokens buf[0 .. m), m <= 64, to acc, the wave's row lanes in turn.
template <typename T, int VEC>
__device__ __forceinline__ void add_few(const SumArgs &a, const uint16_t *buf, uint32_t m, const Place &q, float (&acc)[VEC]) {
  const T *dy = (const T *)a.dy + q.col;
  float sum[VEC] = {};                         // of their own: chains stay short
  for (uint32_t k0 = 0; k0 < m; k0 += DEEP * q.G) {
    Raw<T, VEC> x[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; k++) {
      const uint32_t t = k0 + k * q.G + q.g;
      x[k] = load_loose_if<T, VEC>(q.on && t < m, dy + (int64_t)(t < m ? buf[t] : 0) * a.ldy);
    }
#pragma unroll
    for (int k = 0; k < DEEP; k++) {
      float v[VEC];
      to_f32<T, VEC>(x[k], v);
#pragma unroll
      for (int j = 0; j < VEC; j++) sum[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] += sum[j];
}

template <typename T, int VEC, typename ID>
__global__ __launch_bounds__(FW_THREADS) void k_few_grads(SumArgs a, const ID *__restrict__ ids, uint32_t run) {
  __shared__ uint16_t s_row[FEW];            // row within the run, and token, of each entry
  __shared__ uint16_t s_tok[FEW];
  __shared__ uint16_t s_buf[FW_WAVES][128];
  __shared__ uint32_t s_cnt[FW_WAVES];
  __shared__ float s_sum[FW_WAVES][WAVE * VEC];
  const uint32_t r0 = blockIdx.x * run, rows = a.rows - r0 < run ? a.rows - r0 : run;
  const Place q = place_of<VEC>(a, blockIdx.y);
  const uint32_t w = threadIdx.x >> 6, i0 = w * (WAVE * FW_ITEMS) + q.lane;
  ID id[FW_ITEMS];
  uint32_t row[FW_ITEMS], rank[FW_ITEMS], mine = 0;
#pragma unroll
  for (int j = 0; j < FW_ITEMS; j++) {
    id[j] = -1;
    if (i0 + j * WAVE < a.n) id[j] = ids[i0 + j * WAVE];
  }
#pragma unroll
  for (int j = 0; j < FW_ITEMS; j++) row[j] = key_of((int64_t)id[j], a.rows) - r0;   // ids outside lie past every run
#pragma unroll
  for (int j = 0; j < FW_ITEMS; j++) {
    const uint64_t m = ballot64(row[j] < rows);
    rank[j] = mine + (uint32_t)__popcll(m & ((1ull << q.lane) - 1ull));
    mine += (uint32_t)__popcll(m);
  }
  if (q.lane == 0) s_cnt[w] = mine;
  __syncthreads();
  uint32_t base = 0, len = 0;
#pragma unroll
  for (uint32_t k = 0; k < FW_WAVES; k++) {
    if (k < w) base += s_cnt[k];
    len += s_cnt[k];
  }
#pragma unroll
  for (int j = 0; j < FW_ITEMS; j++)
    if (row[j] < rows) {
      s_row[base + rank[j]] = (uint16_t)row[j];
      s_tok[base + rank[j]] = (uint16_t)(i0 + j * WAVE);
    }
  __syncthreads();
  if (len == 0) {                              // no token here: G rows to a store
    if (a.accumulate || !q.on) return;
    for (uint32_t r = w * q.G + q.g; r < rows; r += FW_WAVES * q.G) {
      float zero[VEC] = {};
      stream_loose<T, VEC>((T *)a.grad + (int64_t)(r0 + r) * a.ldg + q.col, zero);
    }
    return;
  }
  const bool together = len > FW_LONG;
  uint16_t *buf = s_buf[w];
  for (uint32_t r = together ? 0 : w; r < rows; r += together ? 1 : FW_WAVES) {
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
    uint32_t held = 0, seen = 0;               // tokens waiting in buf, and found in all
    for (uint32_t p = together ? w * 64 : 0; p < len; p += together ? FW_WAVES * 64 : 64) {
      const bool hit = p + q.lane < len && s_row[p + q.lane] == r;
      const uint64_t m = ballot64(hit);
      if (hit) buf[held + (uint32_t)__popcll(m & ((1ull << q.lane) - 1ull))] = s_tok[p + q.lane];
      held += (uint32_t)__popcll(m);
      seen += (uint32_t)__popcll(m);
      __builtin_amdgcn_wave_barrier();
      if (held >= 64) {
        add_few<T, VEC>(a, buf, 64, q, acc);
        const uint16_t rest = buf[64 + q.lane];
        __builtin_amdgcn_wave_barrier();
        held -= 64;
        if (q.lane < held) buf[q.lane] = rest;
        __builtin_amdgcn_wave_barrier();
      }
    }
    if (held) add_few<T, VEC>(a, buf, held, q, acc);
    __builtin_amdgcn_wave_barrier();
    if (seen) join_row_lanes<VEC>(acc, a.lg);
    if (together) {
      __syncthreads();                         // the last row's sums have been read
#pragma unroll
      for (int j = 0; j < VEC; j++) s_sum[w][q.lane * VEC + j] = acc[j];
      if (q.lane == 0) s_cnt[w] = seen;
      __syncthreads();
      if (w > 0) continue;
      seen = 0;
#pragma unroll
      for (uint32_t k = 0; k < FW_WAVES; k++) seen += s_cnt[k];
#pragma unroll
      for (uint32_t k = 1; k < FW_WAVES; k++)
#pragma unroll
        for (int j = 0; j < VEC; j++) acc[j] += s_sum[k][q.lane * VEC + j];
    }
    if (q.g == 0 && q.on && (seen || !a.accumulate)) write_row<T, VEC>(a, r0 + r, q.col, acc);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Elements per pack: 16 bytes, or less for shorter rows and where packs have to divide them.
// Overlapping packs against the widest that divides the row and its alignment, lookup and
// gradient in us: 1M rows of 33 fp32 29 and 99 (43 and 133), of 31 fp16 19 and 92 (40 and
// 109), 47337 of 383 fp16 11 and 57 (24 and 92), 20000 of 2723 bf16 25 and 57 (62 and 90),
// 1M of 36 bf16 18 and 91 (19 and 88). They lose in the gradient of short rows that half a
// pack divides: 1M of 20 fp16 12 and 88 (12 and 82), of 12 fp16 10 and 88 (10 and 81).
int pack_width(int bytes, int dim, bool divide) {
  int v = 16 / bytes;
  while (v > dim || (divide && dim % v)) v >>= 1;
  return v;
}

template <typename T, int VEC, typename ID>
int run_lookup(const void *table, int64_t ldt, int64_t rows, int dim, const void *ids, int64_t n, float scale,
               void *out, int64_t ldo, hipStream_t stream) {
  const uint32_t units = (uint32_t)((dim + VEC - 1) / VEC);
  const FastDiv fd = fast_div(units);
  // the kernel's unit index has 31 bits: more tokens take more launches
  const int64_t step = ((1ll << 31) - 1) / units;
  for (int64_t i = 0; i < n; i += step) {
    const int64_t m = n - i < step ? n - i : step;
    const uint32_t total = (uint32_t)(m * units);
    const unsigned per = LK_THREADS * LK_ITEMS;
    hipLaunchKernelGGL((k_lookup<T, VEC, ID>), dim3((total + per - 1) / per), dim3(LK_THREADS), 0, stream,
                       (const T *)table, ldt, rows, (const ID *)ids + i, total, fd, (uint32_t)dim, scale, (T *)out + i * ldo, ldo);
    SPLAT_LAUNCH_CHECK();
  }
  return SPLAT_OK;
}

struct BwdLayout {
  uint2 *pairs[2];
  uint32_t *counts, *totals;
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
  const int tile = ST_THREADS * tile_items(n);
  const size_t tiles = (size_t)((n + tile - 1) / tile);
  for (int k = 0; k < 2; k++) L.pairs[k] = (uint2 *)take(8 * (size_t)n);
  L.counts = (uint32_t *)take(4 * RADIX * tiles);
  L.totals = (uint32_t *)take(4 * RADIX);
  L.bounds = (int2 *)take(8 * (size_t)rows);
  L.part1 = (float *)take(4 * (size_t)(n / CHUNK) * (dim + 7));
  L.part2 = (float *)take(4 * (size_t)(n / (CHUNK * CHUNK)) * (dim + 7));
  L.bytes = (size_t)(p - (char *)base);
  return L;
}

// Workgroups of four waves, few enough that threads count below 2^32.
unsigned wave_grid(uint64_t waves) {
  const uint64_t b = (waves + 3) / 4;
  return (unsigned)(b < (1u << 22) ? b : (1u << 22));
}

template <typename ID, int ITEMS>
int sort_passes(const ID *ids, uint32_t n, uint32_t rows, int bits, int passes, const BwdLayout &L, int *half,
                hipStream_t stream) {
  constexpr uint32_t TOKENS = ST_THREADS * ITEMS;
  const uint32_t tiles = (n + TOKENS - 1) / TOKENS;
  const int dbits = (bits + passes - 1) / passes;
  const bool alone = n <= COUNT_ALONE;
  auto pass = [&](auto src, auto count, auto scatter, auto whole, int p) -> int {
    const int shift = p * dbits, b = bits - shift < dbits ? bits - shift : dbits;
    src.n = n;
    src.rows = rows;
    const unsigned clear = p ? 0u : rows < 1024u * ST_THREADS ? (rows + ST_THREADS - 1) / ST_THREADS : 1024u;
    if (alone) {
      hipLaunchKernelGGL(whole, dim3(tiles + clear), dim3(ST_THREADS), 0, stream, src, shift, b, nullptr, nullptr,
                         L.pairs[p & 1], tiles, L.bounds, rows);
      SPLAT_LAUNCH_CHECK();
      return SPLAT_OK;
    }
    hipLaunchKernelGGL(count, dim3(tiles + clear), dim3(ST_THREADS), 0, stream, src, shift, b, L.counts, tiles, L.bounds,
                       rows);
    SPLAT_LAUNCH_CHECK();
    hipLaunchKernelGGL(k_sort_scan, dim3(((1u << b) + SC_DIGITS - 1) / SC_DIGITS), dim3(SC_THREADS), 0, stream, L.counts,
                       tiles, 1u << b, L.totals);
    SPLAT_LAUNCH_CHECK();
    hipLaunchKernelGGL(scatter, dim3(tiles), dim3(ST_THREADS), 0, stream, src, shift, b, L.counts, L.totals,
                       L.pairs[p & 1], tiles, nullptr, 0u);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  };
  for (int p = 0; p < passes; p++) {
    int st;
    if (p == 0) {
      KeySource<ID, true> src;
      src.from = ids;
      st = pass(src, k_sort_count<ID, true, ITEMS>, k_sort_scatter<ID, true, ITEMS, false>,
                k_sort_scatter<ID, true, 4, true>, p);
    } else {
      KeySource<ID, false> src;
      src.from = L.pairs[(p - 1) & 1];
      st = pass(src, k_sort_count<ID, false, ITEMS>, k_sort_scatter<ID, false, ITEMS, false>,
                k_sort_scatter<ID, false, 4, true>, p);
    }
    if (st) return st;
  }
  *half = (passes - 1) & 1;
  return SPLAT_OK;
}

// Sorts the tokens by id into pairs[*half].
template <typename ID>
int sort_tokens(const void *ids, uint32_t n, uint32_t rows, const BwdLayout &L, int *half, hipStream_t stream) {
  int bits = 1;
  while (bits < 32 && (rows >> bits)) bits++;        // keys 0 .. rows
  const int passes = (bits + RADIX_BITS - 1) / RADIX_BITS;
  return tile_items(n) == 4 ? sort_passes<ID, 4>((const ID *)ids, n, rows, bits, passes, L, half, stream)
                            : sort_passes<ID, 16>((const ID *)ids, n, rows, bits, passes, L, half, stream);
}

// Every row zero: no token to add.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void k_zero_rows(T *grad, int64_t ldg, uint64_t total, uint32_t units, uint32_t dim) {
  const float z[VEC] = {};
  for (uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (uint64_t)gridDim.x * 256) {
    const uint64_t r = u / units;
    stream_loose<T, VEC>(grad + (int64_t)r * ldg + col_of((uint32_t)(u - r * units) * VEC, dim, VEC), z);
  }
}

template <typename T, int VEC, typename ID>
int run_few(SumArgs a, const void *ids, hipStream_t stream) {
  const uint32_t run = (uint32_t)few_run(a.rows);
  const dim3 grid((a.rows + run - 1) / run, (unsigned)a.slices);
  hipLaunchKernelGGL((k_few_grads<T, VEC, ID>), grid, dim3(FW_THREADS), 0, stream, a, (const ID *)ids, run);
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

template <typename T, int VEC>
int run_lookup_bwd(SumArgs a, const void *ids, int id_type, void *ws, hipStream_t stream) {
  a.units = (a.dim + VEC - 1) / VEC;
  a.width = a.units * VEC;
  if (a.n == 0) {
    if (a.accumulate) return SPLAT_OK;
    const uint64_t total = (uint64_t)a.rows * a.units;
    const uint64_t blocks = (total + 255) / 256;
    hipLaunchKernelGGL((k_zero_rows<T, VEC>), dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream,
                       (T *)a.grad, a.ldg, total, (uint32_t)a.units, (uint32_t)a.dim);
    SPLAT_LAUNCH_CHECK();
    return SPLAT_OK;
  }
  a.lg = 0;
  while (a.lg < 6 && (1 << a.lg) < a.units) a.lg++;
  a.slices = (a.units + 63) / 64;
  if (few_tokens(a.n, a.rows))
    return id_type == SPLAT_I64 ? run_few<T, VEC, int64_t>(a, ids, stream) : run_few<T, VEC, int32_t>(a, ids, stream);
  const BwdLayout L = bwd_layout(ws, a.n, a.rows, a.dim);
  int half = 0;
  const int st = id_type == SPLAT_I64 ? sort_tokens<int64_t>(ids, a.n, a.rows, L, &half, stream)
                                      : sort_tokens<int32_t>(ids, a.n, a.rows, L, &half, stream);
  if (st) return st;
  a.sorted = L.pairs[half];
  a.chunks = (a.n + CHUNK - 1) / CHUNK;
  a.bounds = L.bounds;
  a.part1 = L.part1;
  a.part2 = L.part2;
  const uint64_t w1 = (uint64_t)a.chunks * a.slices;
  hipLaunchKernelGGL((k_chunk_sums<T, VEC>), dim3(wave_grid(w1)), dim3(256), 0, stream, a);
  SPLAT_LAUNCH_CHECK();
  // below two whole second-level chunks a row has at most 128 first-level sums: not worth a launch
  a.two_levels = a.n >= 2 * CHUNK * CHUNK;
  if (a.two_levels) {
    const uint64_t w2 = (uint64_t)(a.n / (CHUNK * CHUNK)) * a.slices;
    hipLaunchKernelGGL((k_chunk_sums2<VEC>), dim3(wave_grid(w2)), dim3(256), 0, stream, a);
    SPLAT_LAUNCH_CHECK();
  }
  const uint32_t G = 64u >> a.lg, sets = (a.rows + G - 1) / G;
  const uint64_t heavy = a.n > CHUNK ? a.chunks : 0;
  if (a.n < a.rows) {      // most rows empty
    hipLaunchKernelGGL((k_row_grads<T, VEC, 8>), dim3(wave_grid((heavy + (sets + 7) / 8) * a.slices)), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((k_row_grads<T, VEC, 1>), dim3(wave_grid((heavy + sets) * a.slices)), dim3(256), 0, stream, a);
  }
  SPLAT_LAUNCH_CHECK();
  return SPLAT_OK;
}

}  // namespace

int launch_lookup(const void *table, int dtype, int64_t rows, int dim, int64_t ldt, const void *ids, int id_type,
                  int64_t n, float scale, void *out, int64_t ldo, hipStream_t stream) {
  if (n == 0 || dim == 0) return SPLAT_OK;
  const int vec = pack_width(dtype_bytes(dtype), dim, false);
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

size_t lookup_bwd_workspace_bytes(int64_t n, int64_t rows, int dim) {
  return few_tokens(n, rows) ? 0 : bwd_layout(nullptr, n, rows, dim).bytes;
}

int launch_lookup_bwd(const void *d_out, int dtype, int64_t ldy, const void *ids, int id_type, int64_t n, int64_t rows,
                      int dim, float scale, void *d_table, int64_t ldg, int accumulate, void *ws, hipStream_t stream) {
  if (rows == 0 || dim == 0) return SPLAT_OK;
  SumArgs a = {};
  a.dy = d_out; a.ldy = ldy; a.grad = d_table; a.ldg = ldg;
  a.n = (uint32_t)n; a.rows = (uint32_t)rows; a.dim = dim; a.scale = scale; a.accumulate = accumulate;
  const int vec = pack_width(dtype_bytes(dtype), dim, accumulate != 0);
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
