// tt_embed.hip -- rows of a dense (or int8) table times a scale, and the table's gradient by
// sorted tokens.
//
//   out[n] = s W[i_n]        dW[v] = s sum over n with i_n = v, in the order of n, of dout[n]
//
// Both are bytes alone.  The forward is a gather: a thread moves groups of eight elements.
// The gradient writes all V rows in one pass (rows that no token names are zeros) and reads
// every gradient row once: the tokens are sorted by row, stably, a block takes R rows of the
// table by LPR groups of eight columns, finds their tokens and adds each row's in their order.
// Runs of one row are cut at multiples of PIECE in the sorted order, and their whole pieces are
// summed beforehand by workgroups of their own, so a token that fills half a batch does not
// leave its row to one wave.  Sums are fp32, their order depends on the tokens alone, and each
// is rounded once.
#include <algorithm>

#include "tt_internal.h"
#include "tt_mfma.h"

namespace ttb {

typedef unsigned long long u64;

constexpr int PIECE_T = 64;      // sorted tokens per piece of a long run
constexpr int LONG_RUN = 2 * PIECE_T;  // from here on a run has a whole piece
constexpr int ROWS_MAX = 64;     // rows of the table per block, at most
constexpr int LIST = 1024;       // tokens of a block's rows that are kept in LDS
constexpr int MAX_BITS = 10;     // of a digit
constexpr int BINS = 1 << MAX_BITS;
constexpr int SORT_ROUNDS = 8;   // elements per thread
constexpr int TILE_T = 512 * SORT_ROUNDS;    // tokens per workgroup of the sort of many
constexpr int SMALL_T = 1024 * SORT_ROUNDS;  // tokens that one workgroup sorts

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
  int lpr, chunks, rows;       // groups of eight columns per block, blocks along a row, rows per block
  const u64 *sorted;           // row << 32 | token; tokens without a row last, as row v
  float *part;                 // [n / PIECE_T][d] sums of the whole pieces
};

template <class T>
struct Eight {
  T x[8];
};
// eight elements at p, of which `left` are there (p on an element's boundary only; int8: on a
// group's)
template <class T>
__device__ __forceinline__ Eight<T> get8(const T *p, int64_t left) {
  Eight<T> r;
  if (left >= 8) {
    struct __attribute__((packed, aligned(sizeof(T) < 2 ? 8 : 2))) any { Eight<T> v; };
    r = ((const any *)p)->v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.x[e] = e < left ? p[e] : (T)0;
  }
  return r;
}
template <class T>
__device__ __forceinline__ void put8(T *p, const Eight<T> &r, int64_t left) {
  if (left >= 8) {
    struct __attribute__((packed, aligned(sizeof(T) < 2 ? 8 : 2))) any { Eight<T> v; };
    any a = {r};
    *(any *)p = a;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = r.x[e];
  }
}

// ---------------------------------------------------------------- forward
template <class W, class O>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a) {
  const int64_t cpr = (a.d + 7) / 8, total = a.n * cpr, st = (int64_t)gridDim.x * 256;
  int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t r = q / cpr, c = q % cpr;
  const int64_t dr = st / cpr, dc = st % cpr;
  for (; q < total; q += st) {
    const int64_t v = a.idx[r];
    const bool in = v >= 0 && v < a.v;
    if (!in && c == 0) set_status(a.status, TT_DEV_BAD_INDEX);
    Eight<O> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.x[e] = (O)0.f;
    if (in) {
      const Eight<W> w = get8((const W *)a.w + v * a.wld + c * 8, a.d - c * 8);
      if constexpr (sizeof(W) == 1) {
        const float t = a.rs[v];
#pragma unroll
        for (int e = 0; e < 8; ++e) o.x[e] = (O)((float)w.x[e] * t * a.scale);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o.x[e] = (O)((float)w.x[e] * a.scale);
      }
    }
    put8((O *)a.out + r * a.d + c * 8, o, a.d - c * 8);
    r += dr;
    c += dc;
    if (c >= cpr) c -= cpr, ++r;
  }
}

// ---------------------------------------------------------------- sort
__device__ __forceinline__ u64 token_key(const EmbedArgs &a, int64_t i, bool tell) {
  const int64_t v = a.idx[i];
  const bool in = v >= 0 && v < a.v;
  if (!in && tell) set_status(a.status, TT_DEV_BAD_INDEX);
  return (u64)(in && v != a.pad ? v : a.v) << 32 | (unsigned)i;
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

// exclusive sums of x over the first `bins` of NT * PER values, thread t holding t, t + NT, ..
// (all threads call it)
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

// All passes of at most SMALL_T tokens, in LDS.
__global__ __launch_bounds__(1024) void k_embed_sort_small(EmbedArgs a, u64 *out, int passes,
                                                           int bits) {
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  u64 *buf = (u64 *)dyn;                                 // [SMALL_T]
  int *count = (int *)(dyn + SMALL_T * sizeof(u64));     // [16][1 << bits]
  __shared__ int s_w[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, n = (int)a.n, bins = 1 << bits;
  // each wave takes as many rounds as the tokens need
  const int rounds = (n + 1023) / 1024;
  const int first = wv * rounds * 64;
  u64 key[SORT_ROUNDS];
  int rank[SORT_ROUNDS];
#pragma unroll
  for (int u = 0; u < SORT_ROUNDS; ++u) {
    const int i = first + u * 64 + lane;
    key[u] = u < rounds && i < n ? token_key(a, i, true) : 0;
  }
  for (int p = 0; p < passes; ++p) {
    for (int i = tid; i < 16 * bins; i += 1024) count[i] = 0;
    __syncthreads();
    rank_rounds(key, first, u64(first) + rounds * 64 < (u64)n ? first + rounds * 64 : n, p * bits, bits,
                count + wv * bins, rank);
    __syncthreads();
    int all = 0;
    if (tid < bins)
      for (int w = 0; w < 16; ++w) {
        const int c = count[w * bins + tid];
        count[w * bins + tid] = all;
        all += c;
      }
    const int base = scan_bins<1024>(all, s_w);
    if (tid < bins)
      for (int w = 0; w < 16; ++w) count[w * bins + tid] += base;
    __syncthreads();
    u64 *to = p == passes - 1 ? out : buf;
#pragma unroll
    for (int u = 0; u < SORT_ROUNDS; ++u)
      if (u < rounds && first + u * 64 + lane < n)
        to[count[wv * bins + digit_of(key[u], p * bits, bits)] + rank[u]] = key[u];
    __syncthreads();
    if (p == passes - 1) break;
#pragma unroll
    for (int u = 0; u < SORT_ROUNDS; ++u) {
      const int i = first + u * 64 + lane;
      if (u < rounds && i < n) key[u] = buf[i];
    }
    __syncthreads();
  }
}

// One pass of more tokens: a tile's digits counted ..
__global__ __launch_bounds__(512) void k_embed_hist(EmbedArgs a, const u64 *in, int *hist, int shift,
                                                    int bits) {
  __shared__ int count[BINS];
  const int tid = threadIdx.x, bins = 1 << bits;
  for (int i = tid; i < bins; i += 512) count[i] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * TILE_T;
#pragma unroll
  for (int u = 0; u < SORT_ROUNDS; ++u) {
    const int64_t i = i0 + u * 512 + tid;
    if (i < a.n) atomicAdd(&count[digit_of(in ? in[i] : token_key(a, i, true), shift, bits)], 1);
  }
  __syncthreads();
  for (int i = tid; i < bins; i += 512) hist[(int64_t)blockIdx.x * bins + i] = count[i];
}
// .. and put behind those of smaller digits and of the same digit in the tiles before
__global__ __launch_bounds__(512) void k_embed_scatter(EmbedArgs a, const u64 *in, u64 *out,
                                                       const int *hist, int tiles, int shift,
                                                       int bits) {
  __shared__ int count[8 * BINS];
  __shared__ int s_w[8];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, bins = 1 << bits;
  for (int i = tid; i < 8 * bins; i += 512) count[i] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * TILE_T + wv * SORT_ROUNDS * 64;
  u64 key[SORT_ROUNDS];
  int rank[SORT_ROUNDS];
#pragma unroll
  for (int u = 0; u < SORT_ROUNDS; ++u) {
    const int64_t i = first + u * 64 + lane;
    key[u] = i < a.n ? (in ? in[i] : token_key(a, i, false)) : 0;
  }
  rank_rounds(key, first, a.n, shift, bits, count + wv * bins, rank);
  __syncthreads();
  int carry = 0;  // of the digits before this block of 512
  for (int d0 = 0; d0 < bins; d0 += 512) {
    const int d = d0 + tid;
    int mine = 0, all = 0;
    if (d < bins) {
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
  for (int u = 0; u < SORT_ROUNDS; ++u)
    if (first + u * 64 + lane < a.n)
      out[count[wv * bins + digit_of(key[u], shift, bits)] + rank[u]] = key[u];
}

// ---------------------------------------------------------------- gradient
template <class G>
__device__ __forceinline__ void add8(float (&acc)[8], const Eight<G> &g) {
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] += (float)g.x[e];
}

// the sums of the pieces whose tokens are all of one row
template <class G>
__global__ __launch_bounds__(256) void k_embed_pieces(EmbedArgs a) {
  const int64_t p = blockIdx.x, s = p * PIECE_T;
  const unsigned row = (unsigned)(a.sorted[s] >> 32);
  if (row != (unsigned)(a.sorted[s + PIECE_T - 1] >> 32) || row >= (u64)a.v) return;
  __shared__ unsigned s_pos[PIECE_T];
  if (threadIdx.x < PIECE_T) s_pos[threadIdx.x] = (unsigned)a.sorted[s + threadIdx.x];
  __syncthreads();
  for (int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8; c < a.d;
       c += (int64_t)gridDim.y * 2048) {
    float acc[8] = {};
    constexpr int U = 8;
    for (int k = 0; k < PIECE_T; k += U) {
      Eight<G> g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = get8((const G *)a.w + (int64_t)s_pos[k + u] * a.gld + c, a.d - c);
#pragma unroll
      for (int u = 0; u < U; ++u) add8(acc, g[u]);
    }
    Eight<float> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.x[e] = acc[e];
    put8(a.part + p * a.d + c, o, a.d - c);
  }
}

// first sorted place whose row is at least r: 64 probes at a time, all lanes of a wave
__device__ __forceinline__ int64_t lower_bound(const u64 *sorted, int64_t n, u64 r) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = n;
  while (len > 0) {
    const int64_t step = (len + 63) / 64, at = lo + lane * step;
    const u64 less = __ballot(at < lo + len && sorted[at] >> 32 < r);
    const int k = __popcll(less);  // probes below r: the place is past the last of them
    if (k == 0) return lo;
    const int64_t from = lo + (k - 1) * step + 1, to = min(lo + k * step, lo + len);
    lo = from;
    len = to - from;
  }
  return lo;
}

// DIRECT: the block looks its tokens up in the unsorted list (at most LIST of them).
template <class G, class W, bool DIRECT>
__global__ __launch_bounds__(256) void k_embed_rows(EmbedArgs a) {
  __shared__ int s_start[ROWS_MAX + 1];
  __shared__ unsigned s_pos[LIST];
  __shared__ short s_row[DIRECT ? LIST : 1];
  __shared__ int s_n[4];
  __shared__ int64_t s_seg[2];
  __shared__ float s_sum[256 * 8];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int chunk = blockIdx.x % a.chunks;
  const int64_t r0 = (int64_t)(blockIdx.x / a.chunks) * a.rows;
  const int R = (int)min<int64_t>(a.rows, a.v - r0);
  int64_t seg = 0;  // the block's first sorted place
  if constexpr (DIRECT) {
    // tokens of these rows in their order
    int found = 0;
    for (int64_t i0 = 0; i0 < a.n; i0 += 256) {
      const int64_t i = i0 + tid;
      const u64 key = i < a.n ? token_key(a, i, blockIdx.x == 0) : (u64)a.v << 32;
      const int64_t r = (int64_t)(key >> 32) - r0;
      const bool on = r >= 0 && r < R;
      const u64 m = __ballot(on);
      if (lane == 0) s_n[wv] = __popcll(m);
      __syncthreads();
      int at = found + __popcll(m & ((1ull << lane) - 1));
      for (int w = 0; w < 4; ++w) {
        if (w < wv) at += s_n[w];
        found += s_n[w];
      }
      if (on) {
        s_row[at] = (short)r;
        s_pos[at] = (unsigned)i;
      }
      __syncthreads();
    }
    // sorted by row: a thread counts, and then moves, one row's
    unsigned own[4];  // (a row's first four; more are looked for again)
    int c = 0;
    if (tid < ROWS_MAX) {
      for (int k = 0; k < found; ++k)
        if (s_row[k] == tid) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c == e) own[e] = k;
          ++c;
        }
      int s = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int m = __shfl_up(s, o);
        if (lane >= o) s += m;
      }
      s_start[tid + 1] = s;
      if (tid == 0) s_start[0] = 0;
    }
    __syncthreads();
    // s_sum is free here: the sorted list goes through it
    unsigned *list = (unsigned *)s_sum;
    if (tid < ROWS_MAX && c > 0) {
      int s = s_start[tid];
      if (c <= 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < c) list[s + e] = s_pos[own[e]];
      } else {
        for (int k = own[0]; k < found; ++k)
          if (s_row[k] == tid) list[s++] = s_pos[k];
      }
    }
    __syncthreads();
    for (int k = tid; k < found; k += 256) s_pos[k] = list[k];
    __syncthreads();
  } else {
    if (wv < 2) {
      const int64_t at = lower_bound(a.sorted, a.n, (u64)(r0 + (wv ? R : 0)));
      if (lane == 0) s_seg[wv] = at;
    }
    __syncthreads();
    seg = s_seg[0];
    const int len = (int)(s_seg[1] - seg);
    if (tid <= R) s_start[tid] = tid == 0 ? 0 : len;
    __syncthreads();
    // a row starts where the sorted row changes; rows without tokens start where the next does
    for (int k = tid; k < len; k += 256) {
      const u64 key = a.sorted[seg + k];
      const int r = (int)((int64_t)(key >> 32) - r0);
      const int before = k == 0 ? -1 : (int)((int64_t)(a.sorted[seg + k - 1] >> 32) - r0);
      for (int u = before + 1; u <= r; ++u) s_start[u] = k;
      if (k < LIST) s_pos[k] = (unsigned)key;
    }
    __syncthreads();
  }
  const int groups = 256 / a.lpr, grp = tid / a.lpr, own = tid % a.lpr;
  const int64_t c = ((int64_t)chunk * a.lpr + own) * 8;
  const bool live = grp < groups && c < a.d;
  const G *src = (const G *)a.w + c;
  const int64_t left = a.d - c;
  auto pos_of = [&](int k) -> int64_t {
    return k < LIST ? s_pos[k] : (unsigned)a.sorted[seg + k];
  };
  auto store = [&](int r, const float (&acc)[8]) {
    Eight<W> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.x[e] = (W)(acc[e] * a.scale);
    put8((W *)a.out + (r0 + r) * a.d + c, o, left);
  };
  constexpr int B = 4, SHORT = 16;
  if (live) {
    // short runs, B rows side by side so that their loads travel together
    for (int rb = grp; rb < R; rb += groups * B) {
      int k[B], e[B], most = 0;
      bool mine[B];
      float acc[B][8] = {};
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int r = rb + j * groups;
        k[j] = r < R ? s_start[r] : 0;
        e[j] = r < R ? s_start[r + 1] : 0;
        mine[j] = r < R && e[j] - k[j] <= SHORT;
        if (!mine[j]) e[j] = k[j];
        most = max(most, e[j] - k[j]);
      }
      for (int m = 0; m < most; ++m) {
        Eight<G> g[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (k[j] + m < e[j]) g[j] = get8(src + pos_of(k[j] + m) * a.gld, left);
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (k[j] + m < e[j]) add8(acc[j], g[j]);
      }
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (mine[j]) store(rb + j * groups, acc[j]);
    }
  }
  // long ones: every group a share of the run, in order, the shares added in order.  A run's
  // items are its tokens up to the first whole piece, the whole pieces, and the rest.
  for (int r = 0; r < R; ++r) {
    const int k0 = s_start[r], k1 = s_start[r + 1];
    if (k1 - k0 <= SHORT) continue;
    const int64_t g0 = seg + k0, g1 = seg + k1;
    int64_t p0 = 0, p1 = 0;
    if (!DIRECT && k1 - k0 >= LONG_RUN) {
      p0 = (g0 + PIECE_T - 1) / PIECE_T;
      p1 = g1 / PIECE_T;
    }
    const int np = (int)(p1 - p0);
    const int head = np ? (int)(p0 * PIECE_T - g0) : k1 - k0;
    const int items = np ? head + np + (int)(g1 - p1 * PIECE_T) : head;
    const int per = (items + groups - 1) / groups;
    float acc[8] = {};
    if (live) {
      const int to = min(items, (grp + 1) * per);
      int m = min(items, grp * per);
      auto tokens = [&](int first, int count) {  // list places [first, first + count)
        constexpr int U = 8;
        int t = 0;
        for (; t + U <= count; t += U) {
          Eight<G> g[U];
#pragma unroll
          for (int u = 0; u < U; ++u) g[u] = get8(src + pos_of(first + t + u) * a.gld, left);
#pragma unroll
          for (int u = 0; u < U; ++u) add8(acc, g[u]);
        }
        for (; t < count; ++t) add8(acc, get8(src + pos_of(first + t) * a.gld, left));
      };
      if (m < head) {
        const int e = min(to, head);
        tokens(k0 + m, e - m);
        m = max(m, e);
      }
      if (m < head + np && m < to) {
        const int e = min(to, head + np);
        const float *p = a.part + (p0 + m - head) * a.d + c;
#pragma unroll 4
        for (; m < e; ++m, p += a.d) add8(acc, get8(p, left));
      }
      if (m < to) tokens((int)(p1 * PIECE_T - seg) + (m - head - np), to - m);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[e * 256 + tid] = acc[e];
    __syncthreads();
    if (live && grp == 0) {
      for (int w = 1; w < groups; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += s_sum[e * 256 + w * a.lpr + tid];
      store(r, acc);
    }
  }
}

// ---------------------------------------------------------------- host
static int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
static int64_t elem_size(int dtype) {
  return dtype == TT_DTYPE_F32 ? 4 : dtype == TT_DTYPE_I8 ? 1 : 2;
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
  const int64_t cpr = (a.d + 7) / 8;
  a.chunks = (int)((cpr + 63) / 64);
  a.lpr = (int)((cpr + a.chunks - 1) / a.chunks);
  // enough blocks to fill the chip, and rows enough to pay for finding their tokens
  a.rows = ROWS_MAX;
  while (a.rows > 8 && (a.v + a.rows - 1) / a.rows * a.chunks < 2048) a.rows /= 2;
  return TT_OK;
}

struct EmbedWs {
  u64 *a, *b;
  int *hist;
  float *part;
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
static bool direct(const EmbedArgs &a) { return a.n <= LIST; }

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
      w.hist = (int *)take((a.n + TILE_T - 1) / TILE_T * (4ll << digits(a).bits));
    }
    w.part = (float *)take(a.n / PIECE_T * a.d * 4);
  }
  w.bytes = std::max<int64_t>(off, 256);
  return w;
}

template <class W, class O>
static void go_forward(const EmbedArgs &a, hipStream_t s) {
  const int64_t groups = a.n * ((a.d + 7) / 8);
  tt_launch(K_EMBED, k_embed<W, O>, dim3((unsigned)std::min<int64_t>((groups + 255) / 256, 1 << 16)),
            dim3(256), 0, s, a);
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
    const int lds = SMALL_T * 8 + (64 << g.bits);
    static const hipError_t e = hipFuncSetAttribute(
        (const void *)k_embed_sort_small, hipFuncAttributeMaxDynamicSharedMemorySize,
        SMALL_T * 8 + (64 << MAX_BITS));
    if (e != hipSuccess) return e;
    tt_launch(K_EMBED_SORT, k_embed_sort_small, dim3(1), dim3(1024), lds, s, a, w.a, g.passes, g.bits);
    *sorted = w.a;
    return hipGetLastError();
  }
  const int tiles = (int)((a.n + TILE_T - 1) / TILE_T);
  const u64 *in = nullptr;
  u64 *to = w.a;
  for (int p = 0; p < g.passes; ++p) {
    tt_launch(K_EMBED_SORT, k_embed_hist, dim3(tiles), dim3(512), 0, s, a, in, w.hist, p * g.bits, g.bits);
    tt_launch(K_EMBED_SORT, k_embed_scatter, dim3(tiles), dim3(512), 0, s, a, in, to,
              (const int *)w.hist, tiles, p * g.bits, g.bits);
    in = to;
    to = to == w.a ? w.b : w.a;
  }
  *sorted = in;
  return hipGetLastError();
}

template <class G, class W>
static void go_rows(const EmbedArgs &a, hipStream_t s) {
  const int64_t blocks = (a.v + a.rows - 1) / a.rows * a.chunks;
  if (direct(a)) {
    tt_launch(K_EMBED_GRAD, k_embed_rows<G, W, true>, dim3((unsigned)blocks), dim3(256), 0, s, a);
    return;
  }
  tt_launch(K_EMBED_GRAD, k_embed_pieces<G>,
            dim3((unsigned)(a.n / PIECE_T), (unsigned)std::min<int64_t>((a.d + 2047) / 2048, 64)),
            dim3(256), 0, s, a);
  tt_launch(K_EMBED_GRAD, k_embed_rows<G, W, false>, dim3((unsigned)blocks), dim3(256), 0, s, a);
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
  if (embed_args(desc, a) != TT_OK || desc->dtype == TT_DTYPE_I8) return 0;
  return (size_t)embed_ws(a, nullptr).bytes;
}

int tt_embed_backward(const tt_embed_desc *desc, const int64_t *indices, const void *grad_out,
                      void *grad_weight, void *ws, size_t ws_bytes, int32_t *dev_status,
                      void *stream) {
  EmbedArgs a;
  const int rc = embed_args(desc, a);
  if (rc != TT_OK) return rc;
  if (desc->dtype == TT_DTYPE_I8) return TT_EINVAL;
  if (!grad_weight || !ws || (a.n && (!indices || !grad_out))) return TT_EINVAL;
  if ((uintptr_t)grad_out % elem_size(desc->out_dtype) ||
      (uintptr_t)grad_weight % elem_size(desc->dtype))
    return TT_EINVAL;
  if ((uintptr_t)ws % 256) return TT_EWORKSPACE;
  const EmbedWs w = embed_ws(a, ws);
  if ((size_t)w.bytes > ws_bytes) return TT_EWORKSPACE;
  if ((a.v + a.rows - 1) / a.rows * a.chunks > 0x7fffffffll) return TT_ESHAPE;
  a.idx = indices; a.w = grad_out; a.out = grad_weight; a.status = dev_status; a.part = w.part;
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
