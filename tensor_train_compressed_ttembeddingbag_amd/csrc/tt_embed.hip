// tt_embed.hip -- rows of a dense (or int8) table times a scale, and the table's gradient by
// sorted tokens.
//
//   out[n] = s W[i_n]        dW[v] = s sum over n with i_n = v, in the order of n, of dout[n]
//
// Both are bytes alone.  The forward is a gather: a thread moves groups of eight elements (65536 x 4096
// bf16 of 131072 rows, a third of them distinct: 0.54 GB written in 170-190 us).
// The gradient writes all V rows in one pass (rows that no token names are zeros) and reads
// every gradient row once: the tokens are sorted by row, stably, a block takes some rows of the
// table by some columns, finds their tokens and adds each row's in their order.  Long runs of one
// row go to blocks of their own, beside each other along the row and over groups of lanes; of many
// tokens their whole pieces of 64 in the sorted order are summed beforehand by further ones.
// So a token that fills half a batch does not leave its row to one wave (8192 times one token, 2048
// columns, 32000 rows: 98 us).  Sums are fp32, their order depends on the tokens alone, and each is rounded once.
//
// Measured, cold: 65536 x 4096 bf16 into 131072 rows, 1.6 GB: the sort 25 us, pieces 18, rows 310-320 (5.0 TB/s);
// 4096 x 2048 into 32000, 148 MB: the sort 8 us, rows 39-42 (3.7 TB/s: some seven dependent waits a block);
// 333 x 515 fp32 into 10007, 21 MB: one launch of 11 (warm) to 15 us, 5 us of it with nothing to do.
#include <algorithm>

#include "tt_internal.h"
#include "tt_mfma.h"
#include "tt_rows.h"

namespace ttb {

typedef unsigned long long u64;

constexpr int PIECE_T = 64;      // sorted tokens per piece of a long run
constexpr int LONG_RUN = 2 * PIECE_T;  // from here on a run has a whole piece
constexpr int ROWS_MAX = 64;     // rows of the table per block, at most
constexpr int SHORT = 16;        // tokens of a run that one group of lanes adds up by itself
constexpr int LIST = 1024;       // tokens that are looked for without a sort
static_assert(ROWS_MAX * SHORT <= LIST, "all short runs of a block in LDS");
// What a block writes, from measurements (us of the rows' kernel, cold, blocks of 16, 32 and 64 KiB): 4096 tokens x
// 2048 of 32000 rows bf16 42, 50, 65; 20000 x 512 of 131072 53, 60, 74; 65536 x 4096 of 131072 396, 312, 313.
constexpr int BLOCK_BYTES = 16384;
constexpr int64_t MOST_BLOCKS = 32768;
constexpr int MAX_BITS = 10;     // of a digit
constexpr int BINS = 1 << MAX_BITS;
constexpr int SEARCH_T_MAX = 32768;  // tokens that go without the launch for pieces
constexpr int SMALL_T = 8192;    // tokens that are sorted by counting

struct EmbedArgs {
  int64_t n, v, d, wld, gld;   // strides in elements
  int64_t pad;
  float scale;
  const int64_t *idx;
  const void *w;               // table, or dout
  const float *rs;             // int8: a scale per row
  void *out;
  int32_t *status;
  // backward
  int lpr, chunks;             // groups of eight columns per block, blocks along a row
  int long_lpr, long_chunks;   // the same of the blocks for long runs
  int rows, shift;             // rows per block: 2^shift
  int *first;                  // [blocks of rows + 1] sorted place of a block's first token
  const u64 *sorted;           // row << 32 | token; tokens without a row last, as row v
  float *part;                 // [n / PIECE_T][d] sums of the whole pieces
};

// ---------------------------------------------------------------- forward
// U groups of a thread travel together.
template <class W, class O, bool NARROW, int U>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a) {
  const int64_t cpr = (a.d + 7) / 8, total = a.n * cpr, st = (int64_t)gridDim.x * 256;
  int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t r = q / cpr, c = q % cpr;
  const int64_t dr = st / cpr, dc = st % cpr;
  for (; q < total; q += U * st) {
    int64_t rr[U], cc[U], v[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rr[u] = r;
      cc[u] = column<NARROW>(c, a.d);
      v[u] = a.idx[min(r, a.n - 1)];
      r += dr;
      c += dc;
      if (c >= cpr) c -= cpr, ++r;
    }
    Eight<W> w[U];
    float t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = v[u] >= 0 && v[u] < a.v;
      const int64_t row = in[u] ? v[u] : 0;
      w[u] = get8<NARROW>((const W *)a.w + row * a.wld + cc[u], a.d);
      t[u] = sizeof(W) == 1 ? a.rs[row] : 1.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (rr[u] >= a.n) continue;
      if (!in[u] && cc[u] == 0) set_status(a.status, TT_DEV_BAD_INDEX);
      Eight<O> o;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = sizeof(W) == 1 ? (float)w[u].x[e] * t[u] : (float)w[u].x[e];
        o.x[e] = (O)(in[u] ? x * a.scale : 0.f);
      }
      put8<NARROW>((O *)a.out + rr[u] * a.d + cc[u], o, a.d);
    }
  }
}

// ---------------------------------------------------------------- sort
// the row of a token, or v for none; bad: whether its index is outside the table (to be told later: an
// atomic between loads would make each wait for the one before)
__device__ __forceinline__ unsigned row_of(const EmbedArgs &a, int64_t v, bool &bad) {
  const bool in = v >= 0 && v < a.v;
  bad |= !in;
  return (unsigned)(in && v != a.pad ? v : a.v);
}
__device__ __forceinline__ void tell(const EmbedArgs &a, bool bad) {
  if (bad) set_status(a.status, TT_DEV_BAD_INDEX);
}
__device__ __forceinline__ int digit_of(u64 key, int shift, int bits) {
  return (int)(key >> (32 + shift)) & ((1 << bits) - 1);
}

// Stable places of a wave's elements: the lanes with the same digit are found by a ballot per
// bit, count[] (the wave's own) runs over the rounds.
template <int ROUNDS>
__device__ __forceinline__ void rank_rounds(const u64 (&key)[ROUNDS], int64_t first, int64_t n,
                                            int shift, int bits, int *count, int (&rank)[ROUNDS]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int u = 0; u < ROUNDS; ++u) {
    if (first + u * 64 >= n) break;
    const bool on = first + u * 64 + lane < n;
    const int d = digit_of(key[u], shift, bits);
    u64 same = __ballot(on);
    for (int b = 0; b < bits; ++b) {
      const u64 one = __ballot(d >> b & 1);
      same &= d >> b & 1 ? one : ~one;
    }
    const u64 below = same & ((1ull << lane) - 1);
    int before = 0;
    if (on) before = count[d];
    wave_lds_sync();
    if (on && below == 0) count[d] = before + __popcll(same);
    wave_lds_sync();
    rank[u] = before + __popcll(below);
  }
}

// the sum of x over the threads before (all threads call it)
template <int NT>
__device__ __forceinline__ int scan_bins(int x, int *s_w) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int m = __shfl_up(s, o);
    if (lane >= o) s += m;
  }
  if (lane == 63) s_w[wv] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wv; ++w) before += s_w[w];
  __syncthreads();
  return before + s - x;
}

// Up to SMALL_T tokens: a token's place is the number of those with a smaller row, or the same row before
// it.  Every workgroup compares its T tokens with all of them, staged in LDS, 256 / T lanes a token: n^2
// comparisons over the whole chip take less than the passes of a radix sort, each of them a launch or a
// workgroup by itself (4096 tokens: 14 us in one workgroup).
template <int T>
__global__ __launch_bounds__(256) void k_embed_rank(EmbedArgs a, u64 *out) {
  extern __shared__ __attribute__((aligned(16))) unsigned s_key[];  // [n rounded up to 4]
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  constexpr int L = 256 / T;
  const int tid = threadIdx.x, n = (int)a.n, quads = (n + 3) / 4;
  bool bad = false;
  for (int i0 = tid; i0 < quads * 4; i0 += 256 * 16) {
    int64_t v[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = a.idx[min(i0 + 256 * u, n - 1)];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int i = i0 + 256 * u;
      if (i < quads * 4) s_key[i] = i < n ? row_of(a, v[u], bad) : ~0u;
    }
  }
  if (blockIdx.x == 0) tell(a, bad);
  __syncthreads();
  const int first = blockIdx.x * T, i = first + tid / L, sub = tid % L;
  const unsigned own = s_key[min(i, n - 1)];
  const u4 *q = (const u4 *)s_key;
  int place = 0;
  const int q0 = first / 4, q1 = min(quads, (first + T + 3) / 4);
  // before this workgroup's tokens equal rows count, behind them they do not
#pragma unroll 4
  for (int k = sub; k < q0; k += L) {
    const u4 v = q[k];
    place += (v.x <= own) + (v.y <= own) + (v.z <= own) + (v.w <= own);
  }
  for (int k = q0 + sub; k < q1; k += L) {
    const u4 v = q[k];
    place += v.x < own || (v.x == own && 4 * k < i);
    place += v.y < own || (v.y == own && 4 * k + 1 < i);
    place += v.z < own || (v.z == own && 4 * k + 2 < i);
    place += v.w < own || (v.w == own && 4 * k + 3 < i);
  }
#pragma unroll 4
  for (int k = q1 + sub; k < quads; k += L) {
    const u4 v = q[k];
    place += (v.x < own) + (v.y < own) + (v.z < own) + (v.w < own);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) place += __shfl_xor(place, o);
  if (sub == 0 && i < n) out[place] = (u64)own << 32 | (unsigned)i;
}

// ROUNDS keys of a thread, STEP places apart: of the first pass from the indices
template <int STEP, int ROUNDS>
__device__ __forceinline__ void load_keys(const EmbedArgs &a, const u64 *in, int64_t i0, bool first,
                                          u64 (&key)[ROUNDS]) {
  int64_t v[ROUNDS];
#pragma unroll
  for (int u = 0; u < ROUNDS; ++u) {
    const int64_t i = min(i0 + u * STEP, a.n - 1);
    v[u] = in ? (int64_t)in[i] : a.idx[i];
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < ROUNDS; ++u) {
    const int64_t i = i0 + u * STEP;
    key[u] = in ? (u64)v[u] : i < a.n ? (u64)row_of(a, v[u], bad) << 32 | (unsigned)i : 0;
  }
  if (first && !in) tell(a, bad);
}

// One pass of more tokens: a tile's digits counted ..
template <int ROUNDS>
__global__ __launch_bounds__(512) void k_embed_hist(EmbedArgs a, const u64 *in, int *hist, int shift,
                                                    int bits) {
  __shared__ int count[BINS];
  const int tid = threadIdx.x, bins = 1 << bits;
  for (int i = tid; i < bins; i += 512) count[i] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * (512 * ROUNDS) + tid;
  u64 v[ROUNDS];
  load_keys<512>(a, in, i0, true, v);
#pragma unroll
  for (int u = 0; u < ROUNDS; ++u)
    if (i0 + u * 512 < a.n) atomicAdd(&count[digit_of(v[u], shift, bits)], 1);
  __syncthreads();
  for (int i = tid; i < bins; i += 512) hist[(int64_t)blockIdx.x * bins + i] = count[i];
}
// Of many tiles: each count becomes the number of its digit in the tiles before, the row behind the last tile has all
// of them.  64 digits a workgroup, its waves a share of the tiles each.  (Up to SCAN_TILES every workgroup of the
// next launch reads all counts itself, which grows with their square.)
constexpr int SCAN_TILES = 128;
__global__ __launch_bounds__(1024) void k_embed_scan(int *hist, int tiles, int bins) {
  __shared__ int s_n[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, d = blockIdx.x * 64 + lane;
  const int per = (tiles + 15) / 16, t0 = min(tiles, wv * per), t1 = min(tiles, t0 + per);
  int n = 0;
  if (d < bins)
#pragma unroll 16
    for (int t = t0; t < t1; ++t) n += hist[(int64_t)t * bins + d];
  s_n[wv][lane] = n;
  __syncthreads();
  if (d >= bins) return;
  int before = 0;
  for (int w = 0; w < wv; ++w) before += s_n[w][lane];
  if (wv == 15) hist[(int64_t)tiles * bins + d] = before + n;
  constexpr int U = 16;
  for (int t = t0; t < t1; t += U) {
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = hist[(int64_t)min(t + u, t1 - 1) * bins + d];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u < t1) hist[(int64_t)(t + u) * bins + d] = before;
      before += c[u];
    }
  }
}

// .. and put behind those of smaller digits and of the same digit in the tiles before
template <int ROUNDS>
__global__ __launch_bounds__(512) void k_embed_scatter(EmbedArgs a, const u64 *in, u64 *out,
                                                       const int *hist, int tiles, int shift,
                                                       int bits) {
  __shared__ int count[8 * BINS];
  __shared__ int s_w[8];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, bins = 1 << bits;
  for (int i = tid; i < 8 * bins; i += 512) count[i] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * (512 * ROUNDS) + wv * ROUNDS * 64;
  u64 key[ROUNDS];
  int rank[ROUNDS];
  load_keys<64>(a, in, first + lane, false, key);
  rank_rounds(key, first, a.n, shift, bits, count + wv * bins, rank);
  __syncthreads();
  int carry = 0;  // of the digits before this block of 512
  for (int d0 = 0; d0 < bins; d0 += 512) {
    const int d = d0 + tid;
    int mine = 0, all = 0;
    if (d < bins && tiles > SCAN_TILES) {
      mine = hist[(int64_t)blockIdx.x * bins + d];
      all = hist[(int64_t)tiles * bins + d];
    } else if (d < bins) {
#pragma unroll 8
      for (int t = 0; t < tiles; ++t) {
        const int c = hist[(int64_t)t * bins + d];
        mine += t < (int)blockIdx.x ? c : 0;
        all += c;
      }
    }
    const int base = carry + scan_bins<512>(all, s_w) + mine;
    // the carry over all digits of this block: the last thread's base and own count
    __shared__ int s_all;
    if (tid == 511) s_all = base - mine + all;
    __syncthreads();
    carry = s_all;
    if (d < bins) {
      int s = base;
      for (int w = 0; w < 8; ++w) {
        const int c = count[w * bins + d];
        count[w * bins + d] = s;
        s += c;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < ROUNDS; ++u)
    if (first + u * 64 + lane < a.n)
      out[count[wv * bins + digit_of(key[u], shift, bits)] + rank[u]] = key[u];
}

// ---------------------------------------------------------------- gradient
template <class G>
__device__ __forceinline__ void add8(float (&acc)[8], const Eight<G> &g) {
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] += (float)g.x[e];
}

// Where each block of rows starts in the sorted order, and the sums of the pieces whose tokens
// are all of one row.
template <class G, bool NARROW>
__global__ __launch_bounds__(256) void k_embed_pieces(EmbedArgs a) {
  const int64_t p = blockIdx.x, s = p * PIECE_T;
  if (blockIdx.y == 0) {
    const int64_t i = s + threadIdx.x;
    const int nb = (int)((a.v + a.rows - 1) >> a.shift);
    auto block_of = [&](int64_t k) {  // tokens without a row lie behind all blocks
      const u64 r = a.sorted[k] >> 32;
      return r < (u64)a.v ? (int)(r >> a.shift) : nb;
    };
    if (threadIdx.x < PIECE_T && i < a.n) {
      const int b = block_of(i);
      for (int u = i == 0 ? 0 : block_of(i - 1) + 1; u <= b; ++u) a.first[u] = (int)i;
      if (i == a.n - 1)
        for (int u = b + 1; u <= nb; ++u) a.first[u] = (int)a.n;
    }
  }
  if (s + PIECE_T > a.n) return;
  const unsigned row = (unsigned)(a.sorted[s] >> 32);
  if (row != (unsigned)(a.sorted[s + PIECE_T - 1] >> 32) || row >= (u64)a.v) return;
  __shared__ unsigned s_pos[PIECE_T];
  if (threadIdx.x < PIECE_T) s_pos[threadIdx.x] = (unsigned)a.sorted[s + threadIdx.x];
  __syncthreads();
  const int64_t cpr = (a.d + 7) / 8;
  for (int64_t q = (int64_t)blockIdx.y * 256 + threadIdx.x; q < cpr; q += (int64_t)gridDim.y * 256) {
    const int64_t c = column<NARROW>(q, a.d);
    float acc[8] = {};
    constexpr int U = 16;
    for (int k = 0; k < PIECE_T; k += U) {
      Eight<G> g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = get8<NARROW>((const G *)a.w + (int64_t)s_pos[k + u] * a.gld + c, a.d);
#pragma unroll
      for (int u = 0; u < U; ++u) add8(acc, g[u]);
    }
    Eight<float> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.x[e] = acc[e];
    put8<NARROW>(a.part + p * a.d + c, o, a.d);
  }
}

// first sorted place whose row is at least r: 64 probes at a time, all lanes of a wave
__device__ __forceinline__ int64_t lower_bound(const u64 *sorted, int64_t n, u64 r) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = n;
  while (len > 0) {
    const int64_t step = (len + 63) / 64, at = lo + lane * step;
    // probes below r: the place is past the last of them
    const int k = __popcll(__ballot(at < lo + len && sorted[min(at, n - 1)] >> 32 < r));
    if (k == 0) return lo;
    const int64_t from = lo + (k - 1) * step + 1, to = min(lo + k * step, lo + len);
    lo = from;
    len = to - from;
  }
  return lo;
}

// The lanes of a block on some columns of the table: groups of lpr lanes beside each other.
template <class G, class W, bool NARROW>
struct Lanes {
  int lpr, groups, grp;
  bool live;
  int64_t c;
  const G *src;
  __device__ __forceinline__ Lanes(const EmbedArgs &a, int chunk, int n) {
    const int tid = threadIdx.x;
    lpr = n;
    groups = 256 / lpr;
    grp = tid / lpr;
    const int64_t group = (int64_t)chunk * lpr + tid % lpr;
    c = column<NARROW>(group, a.d);
    live = grp < groups && group * 8 < a.d;
    src = (const G *)a.w + c;
  }
  __device__ __forceinline__ Eight<G> token(const EmbedArgs &a, unsigned pos) const {
    return get8<NARROW>(src + (int64_t)pos * a.gld, a.d);
  }
  __device__ __forceinline__ void store(const EmbedArgs &a, int64_t row, const float (&acc)[8]) const {
    Eight<W> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.x[e] = (W)(acc[e] * a.scale);
    put8<NARROW>((W *)a.out + row * a.d + c, o, a.d);
  }
};

// A long run of a row, at places [g0, g1) of the order: every group a share of it, in order, the
// shares added in order.  Its items are the tokens up to the first whole piece, the whole pieces
// (PIECES: where there are some), and the rest.  All threads of the block; pos_of(place): token.
template <bool PIECES, bool NARROW, class L, class Pos>
__device__ __forceinline__ void long_run(const EmbedArgs &a, const L &l, int64_t row, int64_t g0,
                                         int64_t g1, Pos pos_of, float *s_sum) {
  int64_t p0 = 0, p1 = 0;
  if (PIECES && g1 - g0 >= LONG_RUN) {
    p0 = (g0 + PIECE_T - 1) / PIECE_T;
    p1 = g1 / PIECE_T;
  }
  const int64_t np = p1 - p0, head = np ? p0 * PIECE_T - g0 : g1 - g0;
  const int64_t items = np ? head + np + (g1 - p1 * PIECE_T) : head;
  const int64_t per = (items + l.groups - 1) / l.groups;
  float acc[8] = {};
  if (l.live) {
    const int64_t to = min(items, (l.grp + 1) * per);
    int64_t m = min(items, l.grp * per);
    auto tokens = [&](int64_t g, int64_t count) {
      constexpr int U = 128 / (int)sizeof(decltype(l.token(a, 0)));
      int64_t t = 0;
      for (; t + U <= count; t += U) {
        decltype(l.token(a, 0)) x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = l.token(a, pos_of(g + t + u));
#pragma unroll
        for (int u = 0; u < U; ++u) add8(acc, x[u]);
      }
      for (; t < count; ++t) add8(acc, l.token(a, pos_of(g + t)));
    };
    if (m < head) {
      const int64_t e = min(to, head);
      tokens(g0 + m, e - m);
      m = max(m, e);
    }
    if (m < head + np && m < to) {
      const int64_t e = min(to, head + np);
      const float *p = a.part + (p0 + m - head) * a.d + l.c;
#pragma unroll 4
      for (; m < e; ++m, p += a.d) add8(acc, get8<NARROW>(p, a.d));
    }
    if (m < to) tokens(p1 * PIECE_T + (m - head - np), to - m);
  }
  if (l.groups > 1) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[e * 256 + threadIdx.x] = acc[e];
    __syncthreads();
    if (l.live && l.grp == 0)
      for (int w = 1; w < l.groups; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += s_sum[e * 256 + w * l.lpr + threadIdx.x];
  }
  if (l.live && l.grp == 0) l.store(a, row, acc);
}

// The long runs that start in one piece of the sorted order (a run of a row that half the tokens
// name would keep a block of 64 rows busy long after the others)
template <class G, class W, bool NARROW, bool PIECES>
__device__ __forceinline__ void long_runs_of_piece(const EmbedArgs &a, int64_t piece, int chunk, int lpr,
                                                   float *s_sum) {
  const int lane = threadIdx.x & 63;  // every wave for itself
  const int64_t i = piece * PIECE_T + lane;
  static_assert(PIECE_T == 64, "a token per lane");
  u64 row = a.v;
  bool starts = false;
  if (i + SHORT < a.n) {
    row = a.sorted[i] >> 32;
    starts = row < (u64)a.v && a.sorted[i + SHORT] >> 32 == row &&
             (i == 0 || a.sorted[i - 1] >> 32 != row);
  }
  u64 todo = __ballot(starts);
  if (todo == 0) return;
  const Lanes<G, W, NARROW> l(a, chunk, lpr);
  for (; todo; todo &= todo - 1) {
    const int at = __ffsll(todo) - 1;
    const u64 r = __shfl((unsigned)row, at);
    // its end: 64 places at a time, then where it lies among 64 of them
    int64_t g0 = piece * PIECE_T + at, lo = g0 + SHORT, step = 1;
    // lo is in the run; the first place past it that is not
    while (true) {  // steps of 1, 64, 4096, ..
      const int64_t p = lo + (lane + 1) * step;
      const u64 in = __ballot(p < a.n && a.sorted[min(p, a.n - 1)] >> 32 == r);
      const int k = __popcll(in);
      lo += k * step;
      if (k < 64) break;
      step *= 64;
    }
    while (step > 1) {
      step /= 64;
      const int64_t p = lo + (lane + 1) * step;
      const u64 in = __ballot(p < a.n && a.sorted[min(p, a.n - 1)] >> 32 == r);
      lo += __popcll(in) * step;
    }
    long_run<PIECES, NARROW>(a, l, (int64_t)r, g0, lo + 1,
                           [&](int64_t g) { return (unsigned)a.sorted[g]; }, s_sum);
  }
}

// A block's rows by its columns.  The tokens of its short runs go through LDS as one list in
// the sorted order; a group of lanes takes those of some consecutive rows and adds them up as a
// stream, U rows of grad_out ahead of the sums, whatever rows they belong to (most rows of a large
// vocabulary have none, so a row at a time would wait for every load).  The
// long runs have blocks of their own, the first ones of the launch.
// DIRECT: the block looks its tokens up in the unsorted list (at most LIST of them), and adds its
// long runs up itself.  SEARCH: there is no launch before that says where a block's tokens start and adds
// whole pieces up: it looks for them in the sorted order, and long runs are cut over more, narrower groups.
enum { DIRECT_T, SEARCH_T, SORTED_T };
template <class G, class W, bool NARROW, int HOW>
__global__ __launch_bounds__(256, NARROW ? 1 : 6) void k_embed_rows(EmbedArgs a) {
  constexpr bool DIRECT = HOW == DIRECT_T, SEARCH = HOW == SEARCH_T;
  __shared__ int s_start[ROWS_MAX + 1];   // a row's first token, from the block's first on
  __shared__ int s_short[ROWS_MAX + 1];   // a row's first token in the list of short runs
  __shared__ unsigned s_pos[LIST];        // that list: tokens, and their rows
  __shared__ unsigned char s_row[LIST];
  __shared__ unsigned s_all[DIRECT ? LIST : 1];  // all tokens by row
  __shared__ int s_n[DIRECT ? 256 : 2];
  __shared__ float s_sum[256 * 8];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int id = blockIdx.x;
  if constexpr (!DIRECT) {
    const int pieces = (int)((a.n + PIECE_T - 1) / PIECE_T) * a.long_chunks;
    if (id < pieces)
      return long_runs_of_piece<G, W, NARROW, !SEARCH>(a, id / a.long_chunks, id % a.long_chunks, a.long_lpr,
                                                       s_sum);
    id -= pieces;
  }
  const int chunk = id % a.chunks;
  const int64_t block = id / a.chunks;
  const int64_t r0 = block << a.shift;
  const int R = (int)min<int64_t>(a.rows, a.v - r0);
  int64_t seg = 0;  // the block's first sorted place
  int len = 0;
  if constexpr (DIRECT) {
    // the tokens of these rows by row, stably: token 256 wv + 64 u + lane, waves without any pass
    static_assert(LIST == 4 * 256 && ROWS_MAX == 64, "tokens of a thread, rows of six bits");
    int *count = s_n + wv * 64;  // the wave's tokens of each row so far
    int64_t v[4];
    int row[4], rank[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = a.n > 0 ? a.idx[min<int64_t>(wv * 256 + u * 64 + lane, a.n - 1)] : 0;
    bool bad = false;
    count[lane] = 0;
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool there = wv * 256 + u * 64 + lane < a.n;
      const int64_t r = there ? (int64_t)row_of(a, v[u], bad) - r0 : -1;
      const bool on = r >= 0 && r < R;
      row[u] = on ? (int)r : -1;
      u64 same = __ballot(on);
      if (same == 0) continue;
#pragma unroll
      for (int b = 0; b < 6; ++b) {
        const u64 one = __ballot(row[u] >> b & 1);
        same &= row[u] >> b & 1 ? one : ~one;
      }
      const u64 below = same & ((1ull << lane) - 1);
      const int before = on ? count[row[u]] : 0;
      wave_lds_sync();
      if (on && below == 0) count[row[u]] = before + __popcll(same);
      wave_lds_sync();
      rank[u] = before + __popcll(below);
    }
    __syncthreads();
    // (each wave for itself, so that one barrier less is needed)
    int before = 0, c = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int x = s_n[w * 64 + lane];
      before += w < wv ? x : 0;
      c += x;
    }
    int end = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(end, o);
      if (lane >= o) end += x;
    }
    len = __shfl(end, 63);
    if (wv == 0) {
      s_start[lane + 1] = end;
      if (lane == 0) s_start[0] = 0;
    }
    const int at = end - c + before;  // of this wave's first token of row `lane`
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int from = __shfl(at, max(row[u], 0));
      if (row[u] >= 0) s_all[from + rank[u]] = (unsigned)(wv * 256 + u * 64 + lane);
    }
    if (blockIdx.x == 0) tell(a, bad);
  } else {
    if constexpr (SEARCH) {
      if (wv < 2) {
        const int64_t at = lower_bound(a.sorted, a.n, (u64)(r0 + (wv ? R : 0)));
        if (lane == 0) s_n[wv] = (int)at;
      }
      __syncthreads();
      seg = s_n[0];
      len = s_n[1] - (int)seg;
    } else {
      seg = a.first[block];
      len = a.first[block + 1] - (int)seg;
    }
    if (tid <= R) s_start[tid] = tid == 0 ? 0 : len;
    __syncthreads();
    if (len <= 8192) {
      // a row starts where the sorted row changes; rows without tokens start where the next does
#pragma unroll 4
      for (int k = tid; k < len; k += 256) {
        const int r = (int)((a.sorted[seg + k] >> 32) - r0);
        const int before = k == 0 ? -1 : (int)((a.sorted[seg + k - 1] >> 32) - r0);
        for (int u = before + 1; u <= r; ++u) s_start[u] = k;
      }
    } else if (tid < R) {
      int lo = 0, hi = len;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((int64_t)(a.sorted[seg + mid] >> 32) - r0 < tid) lo = mid + 1;
        else hi = mid;
      }
      s_start[tid] = lo;
    }
  }
  __syncthreads();
  bool any_long = false;
  if (len > 0) {
    const int c = lane < R ? s_start[lane + 1] - s_start[lane] : 0;
    any_long = __any(c > SHORT);
    if (wv == 0) {
      int s = c <= SHORT ? c : 0;
      const int own = s;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(s, o);
        if (lane >= o) s += x;
      }
      s_short[lane + 1] = s;
      if (lane == 0) s_short[0] = 0;
      s -= own;
      for (int k = 0; DIRECT && k < own; ++k) {
        s_row[s + k] = (unsigned char)lane;
        s_pos[s + k] = s_all[s_start[lane] + k];
      }
    }
    __syncthreads();
    if constexpr (!DIRECT) {
      const int r = tid >> 2, at = s_short[r], count = s_short[r + 1] - at;  // four threads a row
      for (int k = tid & 3; k < count; k += 4) {
        s_row[at + k] = (unsigned char)r;
        s_pos[at + k] = (unsigned)a.sorted[seg + s_start[r] + k];
      }
      __syncthreads();
    }
  }
  const Lanes<G, W, NARROW> l(a, chunk, a.lpr);
  const int share = (R + l.groups - 1) / l.groups, ra = min(R, l.grp * share), rb = min(R, ra + share);
  if (l.live) {
    constexpr int U = 8 / sizeof(G);  // (more of them cost workgroups on a CU)
    int k = len > 0 ? s_short[ra] : 0, cur = -1;
    const int end = len > 0 ? s_short[rb] : 0;
    Eight<G> g[2][U];
    auto load = [&](int k, Eight<G> (&to)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < end) to[u] = l.token(a, s_pos[k + u]);
    };
    float acc[8] = {};
    auto add = [&](int k, const Eight<G> (&from)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < end) {
          const int r = s_row[k + u];
          if (r != cur) {
            if (cur >= 0) l.store(a, r0 + cur, acc);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            cur = r;
          }
          add8(acc, from[u]);
        }
    };
    load(k, g[0]);
    // the empty rows under the first loads
    const float none[8] = {};
    for (int r = ra; r < rb; ++r)
      if (s_start[r + 1] == s_start[r]) l.store(a, r0 + r, none);
    for (; k < end; k += 2 * U) {
      load(k + U, g[1]);
      add(k, g[0]);
      load(k + 2 * U, g[0]);
      add(k + U, g[1]);
    }
    if (cur >= 0) l.store(a, r0 + cur, acc);
  }
  for (int r = 0; DIRECT && any_long && r < R; ++r)
    if (s_start[r + 1] - s_start[r] > SHORT)
      long_run<false, NARROW>(a, l, r0 + r, s_start[r], s_start[r + 1],
                              [&](int64_t g) { return s_all[g]; }, s_sum);
}

// ---------------------------------------------------------------- host
static int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
static int64_t elem_size(int dtype) {
  return dtype == TT_DTYPE_F32 ? 4 : dtype == TT_DTYPE_I8 ? 1 : 2;
}

static bool direct(const EmbedArgs &a) { return a.n <= LIST; }
static bool searches(const EmbedArgs &a) { return !direct(a) && a.n <= SEARCH_T_MAX; }

// A launch has less than 2^32 threads.
static bool launches(const EmbedArgs &a) {
  const int64_t blocks = (a.v + a.rows - 1) / a.rows * a.chunks;
  const int64_t longs = direct(a) ? 0 : (a.n + PIECE_T - 1) / PIECE_T * a.long_chunks;
  return blocks + longs < 1 << 24;
}

static int embed_args(const tt_embed_desc *d, EmbedArgs &a) {
  if (!d) return TT_EINVAL;
  if (d->n < 0 || d->v < 1 || d->d < 1) return TT_EINVAL;
  if (d->dtype < TT_DTYPE_F32 || d->dtype > TT_DTYPE_I8) return TT_EINVAL;
  if (d->out_dtype < TT_DTYPE_F32 || d->out_dtype > TT_DTYPE_F16) return TT_EINVAL;
  if (!(d->scale > -INFINITY && d->scale < INFINITY)) return TT_EINVAL;
  if (d->weight_stride < d->d || d->grad_stride < d->d) return TT_EINVAL;
  // 32-bit places of tokens and rows; elements of the table are counted in 64 bits
  if (d->n > (1 << 28) || d->v > (1 << 30) || d->d > (1 << 20)) return TT_ESHAPE;
  if (d->weight_stride > (1ll << 32) || d->grad_stride > (1ll << 32)) return TT_ESHAPE;
  a = {};
  a.n = d->n; a.v = d->v; a.d = d->d; a.wld = d->weight_stride; a.gld = d->grad_stride;
  a.pad = d->padding_idx;
  a.scale = d->scale;
  // few blocks along a row, with as many of a block's lanes in use as can be
  const int64_t cpr = (a.d + 7) / 8;
  int best = 0;
  // (a block that adds its long runs up itself: at least four groups)
  const int64_t most = a.n <= LIST ? 64 : 256;
  for (int64_t chunks = (cpr + most - 1) / most; chunks <= (cpr + 63) / 64; ++chunks) {
    const int lpr = (int)((cpr + chunks - 1) / chunks), used = 256 / lpr * lpr;
    if (used < best + 16) continue;
    best = used;
    a.chunks = (int)chunks;
    a.lpr = lpr;
  }
  // rows enough to pay for finding their tokens, and enough blocks to fill the chip
  const int64_t bytes = a.lpr * 8ll * (d->dtype == TT_DTYPE_F32 ? 4 : 2);
  a.shift = 2;
  while (a.shift < 6 && (bytes << a.shift) < BLOCK_BYTES) ++a.shift;
  while (a.shift < 6 && (a.v >> a.shift) * a.chunks > MOST_BLOCKS) ++a.shift;
  while (a.shift > 2 && (a.v >> a.shift) * a.chunks < 1024) --a.shift;
  a.rows = 1 << a.shift;
  // a long run over several CUs, and over several groups of lanes of each
  const int64_t narrow = searches(a) ? std::max<int64_t>(16, (cpr + 15) / 16) : 64;
  a.long_lpr = (int)std::min<int64_t>({cpr, narrow, 64});
  a.long_chunks = (int)((cpr + a.long_lpr - 1) / a.long_lpr);
  return TT_OK;
}

struct EmbedWs {
  u64 *a, *b;
  int *hist;
  float *part;
  int *first;
  int64_t bytes;
};
struct Digits {
  int passes, bits;
};
static Digits digits(const EmbedArgs &a) {
  int all = 1;
  while (a.v >> all) ++all;  // rows 0 .. v, v standing for none
  const int passes = (all + MAX_BITS - 1) / MAX_BITS;
  return {passes, (all + passes - 1) / passes};
}
// tokens of a workgroup of the sort: few, so that the passes are short, while their counts are few too
static int sort_tile(const EmbedArgs &a) { return a.n <= 1 << 17 ? 1024 : 4096; }

static EmbedWs embed_ws(const EmbedArgs &a, void *ws) {
  EmbedWs w = {};
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    char *p = (char *)ws + off;
    off = round_up(off + bytes, 256);
    return p;
  };
  if (!direct(a)) {
    w.a = (u64 *)take(a.n * 8);
    if (a.n > SMALL_T) {
      w.b = (u64 *)take(a.n * 8);
      w.hist = (int *)take(((a.n + sort_tile(a) - 1) / sort_tile(a) + 1) * (4ll << digits(a).bits));
    }
    if (!searches(a)) {
      w.part = (float *)take(a.n / PIECE_T * a.d * 4);
      w.first = (int *)take(((a.v + a.rows - 1) / a.rows + 1) * 4);
    }
  }
  w.bytes = std::max<int64_t>(off, 256);
  return w;
}

template <class W, class O>
static void go_forward(const EmbedArgs &a, hipStream_t s) {
  const int64_t groups = a.n * ((a.d + 7) / 8);
  auto go = [&](auto *kernel, int u) {
    tt_launch(K_EMBED, kernel,
              dim3((unsigned)std::min<int64_t>((groups + 256 * u - 1) / (256 * u), 1 << 20)),
              dim3(256), 0, s, a);
  };
  if (a.d < 8) return go(k_embed<W, O, true, 1>, 1);
  if (groups < 1 << 21) return go(k_embed<W, O, false, 1>, 1);
  go(k_embed<W, O, false, 4>, 4);
}
template <class W>
static void go_forward(const EmbedArgs &a, int out, hipStream_t s) {
  if (out == TT_DTYPE_F32) go_forward<W, float>(a, s);
  else if (out == TT_DTYPE_BF16) go_forward<W, __bf16>(a, s);
  else go_forward<W, _Float16>(a, s);
}

static hipError_t sort_tokens(const EmbedArgs &a, const EmbedWs &w, const u64 **sorted,
                              hipStream_t s) {
  const Digits g = digits(a);
  if (a.n <= SMALL_T) {
    const int lds = (int)round_up(a.n, 4) * 4;
    tt_launch(K_EMBED_SORT, k_embed_rank<16>, dim3((unsigned)((a.n + 15) / 16)), dim3(256), lds, s, a, w.a);
    *sorted = w.a;
    return hipGetLastError();
  }
  const int tile = sort_tile(a), tiles = (int)((a.n + tile - 1) / tile);
  const u64 *in = nullptr;
  u64 *to = w.a;
  auto passes = [&](auto *hist, auto *scatter) {
    for (int p = 0; p < g.passes; ++p) {
      tt_launch(K_EMBED_SORT, hist, dim3(tiles), dim3(512), 0, s, a, in, w.hist, p * g.bits, g.bits);
      if (tiles > SCAN_TILES)
        tt_launch(K_EMBED_SORT, k_embed_scan, dim3(((1 << g.bits) + 63) / 64), dim3(1024), 0, s, w.hist, tiles, 1 << g.bits);
      tt_launch(K_EMBED_SORT, scatter, dim3(tiles), dim3(512), 0, s, a, in, to, (const int *)w.hist,
                tiles, p * g.bits, g.bits);
      in = to;
      to = to == w.a ? w.b : w.a;
    }
  };
  if (tile == 1024) passes(k_embed_hist<2>, k_embed_scatter<2>);
  else passes(k_embed_hist<8>, k_embed_scatter<8>);
  *sorted = in;
  return hipGetLastError();
}

template <class G, class W, bool NARROW>
static void go_rows(const EmbedArgs &a, hipStream_t s) {
  const unsigned blocks = (unsigned)((a.v + a.rows - 1) / a.rows * a.chunks);
  const unsigned pieces = (unsigned)((a.n + PIECE_T - 1) / PIECE_T), longs = pieces * a.long_chunks;
  auto go = [&](auto *kernel, unsigned grid) { tt_launch(K_EMBED_GRAD, kernel, dim3(grid), dim3(256), 0, s, a); };
  if (direct(a)) return go(k_embed_rows<G, W, NARROW, DIRECT_T>, blocks);
  if (searches(a)) return go(k_embed_rows<G, W, NARROW, SEARCH_T>, longs + blocks);
  tt_launch(K_EMBED_GRAD, k_embed_pieces<G, NARROW>,
            dim3(pieces, (unsigned)std::min<int64_t>((a.d + 2047) / 2048, 64)), dim3(256), 0, s, a);
  go(k_embed_rows<G, W, NARROW, SORTED_T>, longs + blocks);
}
template <class G, class W>
static void go_rows(const EmbedArgs &a, hipStream_t s) {
  if (a.d < 8) go_rows<G, W, true>(a, s);
  else go_rows<G, W, false>(a, s);
}
template <class G>
static void go_rows(const EmbedArgs &a, int w, hipStream_t s) {
  if (w == TT_DTYPE_F32) go_rows<G, float>(a, s);
  else if (w == TT_DTYPE_BF16) go_rows<G, __bf16>(a, s);
  else go_rows<G, _Float16>(a, s);
}

}  // namespace ttb

using namespace ttb;

extern "C" {

int tt_embed_forward(const tt_embed_desc *desc, const int64_t *indices, const void *weight,
                     const float *row_scales, void *out, int32_t *dev_status, void *stream) {
  EmbedArgs a;
  const int rc = embed_args(desc, a);
  if (rc != TT_OK) return rc;
  if (!weight || (a.n && (!indices || !out))) return TT_EINVAL;
  if ((desc->dtype == TT_DTYPE_I8) != (row_scales != nullptr)) return TT_EINVAL;
  if ((uintptr_t)weight % elem_size(desc->dtype) || (uintptr_t)out % elem_size(desc->out_dtype))
    return TT_EINVAL;
  if (row_scales && ((uintptr_t)weight % 16 || a.wld % 16)) return TT_EINVAL;
  if (a.n == 0) return TT_OK;
  a.idx = indices; a.w = weight; a.rs = row_scales; a.out = out; a.status = dev_status;
  hipStream_t s = (hipStream_t)stream;
  if (desc->dtype == TT_DTYPE_F32) go_forward<float>(a, desc->out_dtype, s);
  else if (desc->dtype == TT_DTYPE_BF16) go_forward<__bf16>(a, desc->out_dtype, s);
  else if (desc->dtype == TT_DTYPE_F16) go_forward<_Float16>(a, desc->out_dtype, s);
  else go_forward<int8_t>(a, desc->out_dtype, s);
  return hipGetLastError() == hipSuccess ? TT_OK : TT_EHIP;
}

size_t tt_embed_workspace_size(const tt_embed_desc *desc) {
  EmbedArgs a;
  if (embed_args(desc, a) != TT_OK || desc->dtype == TT_DTYPE_I8 || !launches(a)) return 0;
  return (size_t)embed_ws(a, nullptr).bytes;
}

int tt_embed_backward(const tt_embed_desc *desc, const int64_t *indices, const void *grad_out,
                      void *grad_weight, void *ws, size_t ws_bytes, int32_t *dev_status,
                      void *stream) {
  EmbedArgs a;
  const int rc = embed_args(desc, a);
  if (rc != TT_OK) return rc;
  if (desc->dtype == TT_DTYPE_I8) return TT_EINVAL;
  if (!launches(a)) return TT_ESHAPE;
  if (!grad_weight || (!ws && !direct(a)) || (a.n && (!indices || !grad_out))) return TT_EINVAL;
  if ((uintptr_t)grad_out % elem_size(desc->out_dtype) ||
      (uintptr_t)grad_weight % elem_size(desc->dtype))
    return TT_EINVAL;
  if ((uintptr_t)ws % 256) return TT_EWORKSPACE;
  const EmbedWs w = embed_ws(a, ws);
  if ((size_t)w.bytes > ws_bytes) return TT_EWORKSPACE;
  a.idx = indices; a.w = grad_out; a.out = grad_weight; a.status = dev_status;
  a.part = w.part; a.first = w.first;
  hipStream_t s = (hipStream_t)stream;
  if (!direct(a)) {
    const hipError_t e = sort_tokens(a, w, &a.sorted, s);
    if (e != hipSuccess) return TT_EHIP;
  }
  if (desc->out_dtype == TT_DTYPE_F32) go_rows<float>(a, desc->dtype, s);
  else if (desc->out_dtype == TT_DTYPE_BF16) go_rows<__bf16>(a, desc->dtype, s);
  else go_rows<_Float16>(a, desc->dtype, s);
  return hipGetLastError() == hipSuccess ? TT_OK : TT_EHIP;
}

}  // extern "C"
