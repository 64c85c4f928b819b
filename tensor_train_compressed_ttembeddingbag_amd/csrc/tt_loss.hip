// tt_loss.hip -- vocabulary-head losses: the kernels around the products, and the C entry points.
#include "tt_loss.h"

#include <algorithm>
#include <type_traits>

namespace ttb {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// ---------------------------------------------------------------- rows of any alignment
// 8 elements from p (p on an element's boundary only), `left` of them real, the rest 0
template <class S>
__device__ __forceinline__ void load8(const S *p, int64_t left, S (&v)[8]) {
  struct __attribute__((packed, aligned(2))) any { S x[8]; };
  if (left >= 8) {
    const any a = *(const any *)p;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = a.x[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : (S)0.f;
  }
}

// the same where rows are whole groups of eight (WHOLE): without a branch, so that several
// loads of a thread travel together; p0 is the row's start
template <bool WHOLE, class S>
__device__ __forceinline__ void load8_at(const S *p0, int64_t c, int64_t d, bool on, S (&v)[8]) {
  if constexpr (WHOLE) {
    on = on && c < d;
    struct __attribute__((packed, aligned(2))) any { S x[8]; };
    const any a = *(const any *)(p0 + (c < d ? c : 0));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = on ? a.x[e] : (S)0.f;
  } else {
    load8(p0 + c, on ? d - c : 0, v);
  }
}

// 8 fp32 values -> two planes: x s = hi + lo
template <class V8, class S>
__device__ __forceinline__ void two_parts(const S (&v)[8], float scale, V8 &hi, V8 &lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (float)v[e] * scale;
    hi[e] = (_Float16)x;
    lo[e] = (_Float16)(x - (float)hi[e]);
  }
}

// 8 source elements -> planes of 16-bit elements (fp32: two parts, or the halves of x)
template <class S, class E, int PL>
__device__ __forceinline__ void store8(const S (&v)[8], float scale, bool whole, char *dst,
                                       int64_t plane) {
  typename E::v8 h;
  if constexpr (PL == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (typename E::e)v[e];
  } else {
    typename E::v8 l;
    if (whole) {
#pragma unroll
      for (int u = 0; u < 8; u += 4) {
        const float x[4] = {(float)v[u], (float)v[u + 1], (float)v[u + 2], (float)v[u + 3]};
        typename E::v4 a, b;
        halves(x, a, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[u + e] = a[e], l[u + e] = b[e];
      }
    } else {
      two_parts(v, scale, h, l);
    }
    *(typename E::v8 *)(dst + plane) = l;
  }
  *(typename E::v8 *)dst = h;
}

// exponent b of the power of two that puts |x| <= amax below 2^15 (0 for an empty tensor)
__device__ __forceinline__ int plane_exp(float amax) {
  if (!(amax > 0.f)) return 0;
  int e;
  frexpf(amax, &e);  // amax < 2^e
  return 15 - e;
}
// Tiny and huge tensors are multiplied as they are: the scales are taken back as zs 2^-(ew + eh)
// and 2^-(e + ge) of a gradient, which have to be normal numbers whatever T and the gradient.
__device__ __forceinline__ bool plane_exps_in_range(int ew, int eh) {
  return max(max(abs(ew), abs(eh)), abs(ew + eh)) <= 64;
}
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255) - 127; }

// What k_amax found of a tensor, in every lane of a wave.  Two parts hold a value to 22 bits
// down to 2^-17 of the largest and to 2^-40 of the largest below; so they stand for a tensor
// whose values lie near its largest, not for one that a mask or an outlier tops by far.
// `spread` is how many powers of two the values' mean exponent lies below the largest's:
// 4 to 5 for normal values, 12 with outliers of 1000 times the rest, 18 and more with a mask
// of -1e4.  Up to RANGE_BITS the values in the middle keep their 22 bits with some to spare.
struct TensorRange {
  float top, spread;
  __device__ __forceinline__ TensorRange(const float *amax, int lane) {
    float m = 0.f, s = 0.f, n = 0.f;
#pragma unroll
    for (int u = 0; u < AMAX_BLOCKS / 64; ++u) {
      const float *p = amax + u * 64 + lane;
      m = fmaxf(m, p[0]);
      s += p[2 * AMAX_BLOCKS];
      n += p[4 * AMAX_BLOCKS];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor(m, o));
      s += __shfl_xor(s, o);
      n += __shfl_xor(n, o);
    }
    top = m;
    spread = n > 0.f ? exponent(m) - s / n : 0.f;
  }
  __device__ __forceinline__ bool in_parts() const { return top < INFINITY && spread <= RANGE_BITS; }
};

// ---------------------------------------------------------------- distillation entries
// One wave per position: q = softmax(teacher / T) over its entries (index >= 0 and logit
// above -inf), sorted by row, so that repeated rows lie side by side; their q are added into the
// first, so that every (position, row) of G is written once.  (q is the lower half of the key: the order of a sum, and with it
// the result, does not depend on the sort's steps.)  sv.tgt[i]: whether position i has entries.
// pow2: the power of two from k on.
template <class S>
__global__ __launch_bounds__(256) void k_entries(LossArgs a, int pow2) {
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, k = a.k;
  const int64_t i = (int64_t)blockIdx.x * 4 + wv;
  if (i >= a.N) return;  // no workgroup barrier below: waves keep to their own LDS
  struct Entry {
    unsigned q, row;  // bits of q; none: ~0
  };
  union Key {
    Entry e;
    uint64_t u;
  };
  Key *key = (Key *)dyn + wv * pow2;
  const float it = 1.f / a.temp;
  float m = -INFINITY;
  bool bad = false, any = false, nan = false;
  for (int j = lane; j < pow2; j += 64) {
    const int64_t v = j < k ? a.tgt[i * k + j] : -1;
    const float t = j < k ? (float)((const S *)a.tlogits)[i * k + j] * it : -INFINITY;
    bad |= v >= a.V;
    const bool in = v >= 0 && v < a.V && !(t == -INFINITY);
    key[j].e = {__float_as_uint(in ? t : -INFINITY), in ? (unsigned)v : ~0u};
    any |= in;
    nan |= in && t != t;
    if (in) m = fmaxf(m, t);
  }
  if (__any(bad) && lane == 0) set_status(a.status, TT_DEV_BAD_INDEX);
  any = __any(any);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if (__any(nan)) m = __builtin_nanf("");
  float s = 0.f;
  for (int j = lane; j < k; j += 64)
    if (key[j].e.row != ~0u) s += expf(__uint_as_float(key[j].e.q) - m);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  const float ls = logf(s);
  float ent = 0.f;
  for (int j = lane; j < k; j += 64) {
    if (key[j].e.row == ~0u) continue;
    const float lq = __uint_as_float(key[j].e.q) - m - ls, p = expf(lq);
    key[j].e.q = __float_as_uint(p);
    if (!(p == 0.f)) ent += p * lq;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) ent += __shfl_xor(ent, o);
  auto settle = [] {
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
  };
  settle();
  for (int size = 2; size <= pow2; size <<= 1)
    for (int st = size >> 1; st > 0; st >>= 1) {
      for (int x = lane; x < pow2 / 2; x += 64) {
        const int lo = 2 * x - (x & (st - 1)), hi = lo + st;
        const uint64_t p = key[lo].u, q = key[hi].u;
        if ((p > q) == ((lo & size) == 0)) {
          key[lo].u = q;
          key[hi].u = p;
        }
      }
      settle();
    }
  for (int j = lane; j < k; j += 64) {
    const unsigned row = key[j].e.row;
    float p = 0.f;
    if (row != ~0u && (j == 0 || key[j - 1].e.row != row))
      for (int u = j; u < k && key[u].e.row == row; ++u) p += __uint_as_float(key[u].e.q);
    a.sv.eidx[i * k + j] = (int)row;
    a.sv.eq[i * k + j] = p;
  }
  if (lane == 0) {
    a.sv.ent[i] = ent;
    a.sv.tgt[i] = any;
  }
}

// ---------------------------------------------------------------- packing
// amax: the weight (blocks 0 ..) and the positions that count
__global__ __launch_bounds__(256) void k_amax(LossArgs a) {
  const bool w = blockIdx.x < AMAX_BLOCKS;
  const int b = blockIdx.x % AMAX_BLOCKS, tid = threadIdx.x;
  const float *x = (const float *)(w ? a.weight : a.hidden);
  const int64_t rows = w ? a.V : a.N, ld = w ? a.wld : a.hld;
  const int64_t cpr = (a.D + 7) / 8, n = rows * cpr;
  float m = 0.f;
  int es = 0, en = 0;
  int64_t i = (int64_t)b * 256 + tid;
  int64_t r = i / cpr, q = i % cpr;
  const int64_t dr = AMAX_BLOCKS * 256 / cpr, dq = AMAX_BLOCKS * 256 % cpr;
  for (; i < n; i += AMAX_BLOCKS * 256) {
    if (w || counts(a, r)) {
      float v[8];
      load8(x + r * ld + q * 8, a.D - q * 8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m = fmaxf(m, v[e] == v[e] ? fabsf(v[e]) : INFINITY);
        es += v[e] != 0.f ? exponent(v[e]) : 0;
        en += v[e] != 0.f;
      }
    }
    r += dr;
    q += dq;
    if (q >= cpr) q -= cpr, ++r;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  float fs = (float)es, fn = (float)en;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) fs += __shfl_xor(fs, o), fn += __shfl_xor(fn, o);
  __shared__ float s[3][4];
  if ((tid & 63) == 0) s[0][tid >> 6] = m, s[1][tid >> 6] = fs, s[2][tid >> 6] = fn;
  __syncthreads();
  if (tid == 0) {
    float *o = a.amax + blockIdx.x;
    o[0] = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
    o[2 * AMAX_BLOCKS] = s[1][0] + s[1][1] + s[1][2] + s[1][3];
    o[4 * AMAX_BLOCKS] = s[2][0] + s[2][1] + s[2][2] + s[2][3];
  }
}

// counts and its loss has a gradient (one that is not a number is one)
__device__ __forceinline__ bool kept(const LossArgs &a, int64_t i) {
  return a.sv.slot[i] >= 0 && !(gradient_of(a, i) == 0.f);
}

// Positions that count (KEPT: and have a gradient) in each chunk, and (one block) in all chunks
// before each.
template <bool KEPT>
__global__ __launch_bounds__(256) void k_count(LossArgs a) {
  __shared__ int s_n[4];
  const int tid = threadIdx.x;
  const int64_t i0 = (int64_t)blockIdx.x * CHUNK, end = min(i0 + CHUNK, a.N);
  int n = 0;
  for (int64_t i = i0 + tid; i < end; i += 256) n += KEPT ? kept(a, i) : counts(a, i);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if ((tid & 63) == 0) s_n[tid >> 6] = n;
  __syncthreads();
  if (tid == 0) a.chunk[blockIdx.x] = s_n[0] + s_n[1] + s_n[2] + s_n[3];
}
__global__ __launch_bounds__(1024) void k_count_before(LossArgs a, int chunks) {
  __shared__ int s_n[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int before = 0;
  for (int c0 = 0; c0 < chunks; c0 += 1024) {
    const int own = c0 + tid < chunks ? a.chunk[c0 + tid] : 0;
    int n = own;  // up to and with this lane's
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int m = __shfl_up(n, o);
      if (lane >= o) n += m;
    }
    if (lane == 63) s_n[wv] = n;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < 16; ++w) {
      if (w == wv) n += before + all;
      all += s_n[w];
    }
    if (c0 + tid < chunks) a.chunk[c0 + tid] = n - own;
    before += all;
    __syncthreads();
  }
}

// Rows of the hidden states that count, in order, from row 0 of hp on; the rest of hp's first N
// rows are zeros (every position that does not count clears one of them; the backward sums
// over the packed rows 64 at a time), and so are the rows from N to the next multiple of 64.
// A block counts the positions before its own by itself: up to CHUNKS_AT positions reading N / 2
// flags on average in N / 4 blocks costs less than two launches that count them; from there on it
// starts at its chunk.
template <class S, class E, int PL>
__global__ __launch_bounds__(256) void k_pack(LossArgs a) {
  __shared__ int s_n[4], s_slot[PACK_ROWS], s_parts[2];
  __shared__ float s_top[2];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t i0 = (int64_t)blockIdx.x * PACK_ROWS, ib = min(i0, a.N);
  int n = 0;
#pragma unroll 4
  for (int64_t i = (a.chunk ? ib / CHUNK * CHUNK : 0) + tid; i < ib; i += 256) n += counts(a, i);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if (lane == 0) s_n[wv] = n;
  if (PL > 1 && wv < 2) {  // the weight's range, the positions'
    const TensorRange t(a.amax + wv * AMAX_BLOCKS, lane);
    if (lane == 0) s_top[wv] = t.top, s_parts[wv] = t.in_parts();
  }
  __syncthreads();
  const int base = s_n[0] + s_n[1] + s_n[2] + s_n[3] +
                   (a.chunk && i0 < a.N ? a.chunk[i0 / CHUNK] : 0);
  int ew = 0, eh = 0;
  bool whole = false;
  if (PL > 1) {
    whole = !(s_parts[0] && s_parts[1]);
    if (!whole) ew = plane_exp(s_top[0]), eh = plane_exp(s_top[1]);
    if (!plane_exps_in_range(ew, eh)) whole = true, ew = eh = 0;
  }
  if (wv == 0) {
    const int64_t i = i0 + lane;
    const bool own = lane < PACK_ROWS, in = own && i < a.N;
    const bool ok = in && counts(a, i);
    const uint64_t mask = __ballot(ok);
    const int rank = base + __popcll(mask & ((1ull << lane) - 1));
    int slot = -1 - (int)i;  // a row past the last position: zeros
    if (in) {
      slot = ok ? rank : -1 - (int)(a.N - 1 - (i - rank));
      a.sv.slot[i] = slot;
      if (!a.k) {
        const int64_t t = a.tgt[i];
        if (ok) a.sv.tgt[rank] = (int)t;
        else if (bad_target(a, i)) set_status(a.status, TT_DEV_BAD_INDEX);
      }
      if (i == a.N - 1) a.sv.sc->count = rank + ok;
    }
    if (own) s_slot[lane] = slot;
    if (blockIdx.x == 0 && lane == 0) {
      a.sv.sc->zs = ldexpf(LOG2E / a.temp, -(ew + eh));
      a.sv.sc->whole = whole;
      a.sv.sc->ge = whole ? 0 : g_exp(a.dtype);
      a.sv.sc->ew = ew;
      a.sv.sc->eh = eh;
      a.sv.sc->ticket = 0;
    }
  }
  __syncthreads();
  const float scale = ldexpf(1.f, eh);
  const int cpr = (int)(a.Dp / 8);
  const int64_t last = a.twin ? a.twin : (a.N + GK - 1) / GK * GK;
  auto copy = [&](auto eights) {  // rows of whole groups of eight
    constexpr int U = 4;  // groups of eight in flight per thread
    for (int q0 = tid; q0 < PACK_ROWS * cpr; q0 += 256 * U) {
      S v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = min(q0 + 256 * u, PACK_ROWS * cpr - 1), r = q / cpr, c = (q - r * cpr) * 8;
        // a block of past-the-end rows copies none: any row's address will do
        load8_at<decltype(eights)::value>((const S *)a.hidden + min(i0 + r, a.N - 1) * a.hld, c,
                                         a.D, s_slot[r] >= 0, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + 256 * u, r = q / cpr, c = (q - r * cpr) * 8;
        if (q >= PACK_ROWS * cpr) continue;
        const int slot = s_slot[r];
        const int64_t row = slot < 0 ? -1 - slot : slot;
        if (row >= last) continue;
        char *o = a.sv.hp + (row * PL * a.Dp + c) * 2;
        store8<S, E, PL>(v[u], scale, whole, o, a.Dp * 2);
        if (PL == 1 && a.twin) store8<S, E, PL>(v[u], scale, whole, o + a.twin * a.Dp * 2, 0);
      }
    }
  };
  if (a.D % 8 == 0) copy(std::true_type());
  else copy(std::false_type());
}

// The same from rows that are packed, for the positions that are kept; their target and statistics
// move with them.  (8000 x 4096 bf16, 131 MB: 46 us.)
__global__ __launch_bounds__(256) void k_keep(LossArgs a, LossSaved to, int64_t row_bytes) {
  __shared__ int s_n[4], s_slot[PACK_ROWS];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t i0 = (int64_t)blockIdx.x * PACK_ROWS, ib = min(i0, a.N);
  int n = 0;
#pragma unroll 4
  for (int64_t i = (a.chunk ? ib / CHUNK * CHUNK : 0) + tid; i < ib; i += 256) n += kept(a, i);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if (lane == 0) s_n[wv] = n;
  __syncthreads();
  const int base = s_n[0] + s_n[1] + s_n[2] + s_n[3] +
                   (a.chunk && i0 < a.N ? a.chunk[i0 / CHUNK] : 0);
  if (wv == 0) {
    const int64_t i = i0 + lane;
    const bool own = lane < PACK_ROWS, in = own && i < a.N;
    const bool ok = in && kept(a, i);
    const uint64_t mask = __ballot(ok);
    const int rank = base + __popcll(mask & ((1ull << lane) - 1));
    if (in) {
      to.slot[i] = ok ? rank : -1 - (int)(a.N - 1 - (i - rank));
      if (ok) {
        const int from = a.sv.slot[i];
        to.tgt[rank] = a.sv.tgt[from];
        to.mx[rank] = a.sv.mx[from];
        to.lg[rank] = a.sv.lg[from];
      }
      if (i == a.N - 1) to.sc->count = rank + ok;
    }
    if (own) s_slot[lane] = in ? to.slot[i] : -1 - (int)i;
    if (blockIdx.x == 0 && lane == 0) {
      to.sc->zs = a.sv.sc->zs;
      to.sc->whole = a.sv.sc->whole;
      to.sc->ge = a.sv.sc->ge;
      to.sc->ew = a.sv.sc->ew;
      to.sc->eh = a.sv.sc->eh;
    }
  }
  __syncthreads();
  const int64_t last = (a.N + GK - 1) / GK * GK;
  const int cpr = (int)(row_bytes / 16);
  constexpr int U = 4;
  for (int q0 = tid; q0 < PACK_ROWS * cpr; q0 += 256 * U) {
    i32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = min(q0 + 256 * u, PACK_ROWS * cpr - 1), r = q / cpr, c = q - r * cpr;
      const int64_t from = s_slot[r] >= 0 ? a.sv.slot[i0 + r] : 0;
      v[u] = *(const i32x4 *)(a.sv.hp + from * row_bytes + c * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + 256 * u, r = q / cpr, c = q - r * cpr;
      if (q >= PACK_ROWS * cpr) continue;
      const int64_t row = s_slot[r] < 0 ? -1 - s_slot[r] : s_slot[r];
      if (row < last) *(i32x4 *)(to.hp + row * row_bytes + c * 16) = s_slot[r] < 0 ? i32x4{} : v[u];
    }
  }
}

// rows [v0, v0 + nv) of the weight -> wp (a copy: 32000 x 1024 fp32 in 41 us, 6.4 TB/s)
template <class S, class E, int PL>
__global__ __launch_bounds__(256) void k_pack_w(LossArgs a, int64_t v0, int64_t nv) {
  const bool whole = PL > 1 && a.sv.sc->whole;
  const float scale = PL > 1 ? ldexpf(1.f, a.sv.sc->ew) : 1.f;
  const int64_t cpr = a.Dp / 8, n = nv * cpr, st = (int64_t)gridDim.x * 256;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < n; q += st) {
    const int64_t r = q / cpr, c = (q - r * cpr) * 8;
    S v[8];
    load8((const S *)a.weight + (v0 + r) * a.wld + c, a.D - c, v);
    store8<S, E, PL>(v, scale, whole, a.wp + (r * PL * a.Dp + c) * 2, a.Dp * 2);
  }
}

// ---------------------------------------------------------------- loss
// packed row of a position, or below 0
__device__ __forceinline__ int slot_of(const LossArgs &a, int64_t i) {
  return a.direct ? (counts(a, i) ? (int)i : -1) : a.sv.slot[i];
}

// the rows' losses added in a fixed order, in fp64; NT threads, s_d: a double per wave
template <int NT>
__device__ __forceinline__ void sum_rows(const LossArgs &a, double *s_d) {
  const int tid = threadIdx.x;
  double d = 0.0;
  int n = 0;
  if (a.direct)  // at most 64 positions
    n = __popcll(__ballot((tid & 63) < a.N && counts(a, tid & 63)));
  else
    n = a.sv.sc->count;
  for (int64_t r = tid; r < a.N; r += NT)
    d += (double)__hip_atomic_load(&a.rowloss[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) d += __shfl_xor(d, o);
  if ((tid & 63) == 0) s_d[tid >> 6] = d;
  __syncthreads();
  if (tid == 0) {
    d = 0.0;
    for (int w = 0; w < NT / 64; ++w) d += s_d[w];
    a.loss[0] = (float)(a.reduction == TT_REDUCE_MEAN ? d / max(n, 1) : d);
  }
}

// Statistics of a position over part of the weight's rows: its largest sum of products, the sum
// of 2^((sum of products - largest) zs), the sum of its logits.
struct Stats {
  float m, s, z;
};
// slots [t0, t1) of a position, every step-th one from this lane on, and then the wave's lanes
__device__ __forceinline__ Stats wave_stats(const LossArgs &a, int64_t slot, int t0, int t1,
                                            int step, float zs) {
  Stats w = {-INFINITY, 0.f, 0.f};
  const int64_t row = slot * a.ptiles;
  for (int t = t0; t < t1; t += step) {
    const float2 v = a.part[row + t];
    const float n = fmaxf(w.m, v.x), n0 = n == -INFINITY ? 0.f : n;
    w.s = w.s * __builtin_amdgcn_exp2f((w.m - n0) * zs) + v.y * __builtin_amdgcn_exp2f((v.x - n0) * zs);
    w.m = n;
    if (a.smoothing > 0.f) w.z += a.zpart[row + t];
  }
  float m = w.m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  w.s *= __builtin_amdgcn_exp2f((w.m - (m == -INFINITY ? 0.f : m)) * zs);
  w.m = m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    w.s += __shfl_xor(w.s, o);
    w.z += __shfl_xor(w.z, o);
  }
  return w;
}

// Where the statistics of all tiles would not fit (see ws_layout): those of a piece of the
// vocabulary, slots 1 .. tiles, are added to the position's in slot 0.
__global__ __launch_bounds__(256) void k_fold(LossArgs a, int tiles, int first) {
  const int lane = threadIdx.x & 63;
  const int64_t count = a.direct ? a.N : a.sv.sc->count;
  const float zs = a.direct ? LOG2E / a.temp : a.sv.sc->zs;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < count; r += gridDim.x * 4) {
    const Stats w = wave_stats(a, r, first + lane, tiles + 1, 64, zs);
    if (lane == 0) {
      a.part[r * a.ptiles] = make_float2(w.m, w.s);
      if (a.smoothing > 0.f) a.zpart[r * a.ptiles] = w.z;
    }
  }
}

// The sums of products of 16 entries of position i, from entry j0 on: lane 16 g + c has those of
// entries 4 g .. + 3 (the same for every c).  They are the very sums that k_logits has of these
// rows: the same instructions on the same k in the same order, the rows of the weight gathered
// in place of 16 that follow each other, and the position's row in all 16 columns.  So what the
// products' rounding does to a logit is the same in it and in lse, and cancels where an entry
// holds most of the probability; a dot product of its own, however exact, would not.
// The gather is its time: 2048 x 32 rows of 2048 fp16 in 41 us, 4096 x 64 of
// 2048 bf16 in 138 us, out of the last-level cache.  (Entries picked out of the tiles of k_logits
// cost 30 and 160 us there, and 45 us of 100 with rows of 256.)
template <class S, class E, bool EIGHTS>
__device__ __forceinline__ f4 entry_sums(const LossArgs &a, int64_t i, int j0, int lane) {
  constexpr int U = 8;  // times 32 k in flight
  const int g = lane >> 4, v = a.sv.eidx[i * a.k + min(j0 + (lane & 15), a.k - 1)];
  const S *w = (const S *)a.weight + max(v, 0) * a.wld;  // no entry: any row, not used
  const S *h = (const S *)a.hidden + i * a.hld;
  f4 acc = zero4();
  for (int64_t k0 = 0; k0 < a.D; k0 += 32 * U) {
    S x[U][8], y[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load8_at<EIGHTS>(w, k0 + 32 * u + 8 * g, a.D, true, x[u]);
      load8_at<EIGHTS>(h, k0 + 32 * u + 8 * g, a.D, true, y[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      typename E::v8 p, q;
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = x[u][e], q[e] = y[u][e];
      acc = E::mfma(p, q, acc);
    }
  }
  return acc;
}
// fp32: the planes as k_logits reads them, but the rows of the weight from the caller's where the
// packed ones are of the vocabulary's last piece only
template <bool EIGHTS>
__device__ __forceinline__ f4 entry_sums_fp32(const LossArgs &a, int64_t i, int slot, int j0,
                                              int lane) {
  constexpr int U = 4;
  const bool packed = a.piece >= a.V, whole = a.sv.sc->whole;
  const float scale = ldexpf(1.f, a.sv.sc->ew);
  const int g = lane >> 4;
  const int64_t v = max(a.sv.eidx[i * a.k + min(j0 + (lane & 15), a.k - 1)], 0), row = a.Dp * 4;
  const char *w = packed ? a.wp + v * row : (const char *)a.weight + v * a.wld * 4;
  const char *h = a.sv.hp + slot * row;
  union Eight {  // values, or their two planes
    float x[8];
    hf8 p[2];
  };
  auto load16 = [](const char *p) {
    struct __attribute__((packed, aligned(2))) any { hf8 v; };
    return ((const any *)p)->v;
  };
  f4 acc = zero4();
  for (int64_t k0 = 0; k0 < a.D; k0 += 32 * U) {
    Eight x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = k0 + 32 * u + 8 * g;
      const int64_t at = c < a.Dp ? c * 2 : 0;
      y[u].p[0] = load16(h + at);
      y[u].p[1] = load16(h + row / 2 + at);
      if (c >= a.Dp) y[u].p[0] = y[u].p[1] = hf8{};
      if (EIGHTS || packed) {
        const bool in = c < (packed ? a.Dp : a.D);
        const char *p = w + (in ? c * (packed ? 2 : 4) : 0);
        x[u].p[0] = load16(p);
        x[u].p[1] = load16(p + (packed ? row / 2 : 16));
        if (!in) x[u].p[0] = x[u].p[1] = hf8{};
      } else {
        load8((const float *)w + c, a.D - c, x[u].x);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
              packed ? ttb::whole(x[u].p[0], x[u].p[1], e) : x[u].x[e],
              ttb::whole(y[u].p[0], y[u].p[1], e), acc, 0, 0, 0);
        continue;
      }
      hf8 hi = x[u].p[0], lo = x[u].p[1];
      if (!packed) two_parts(x[u].x, scale, hi, lo);
      acc = Fp16::mfma(hi, y[u].p[0], acc);
      acc = Fp16::mfma(hi, y[u].p[1], acc);
      acc = Fp16::mfma(lo, y[u].p[0], acc);
    }
  }
  return acc;
}
template <class S, class E, int PL, bool EIGHTS>
__device__ __forceinline__ f4 sums_of(const LossArgs &a, int64_t i, int slot, int j0, int lane) {
  if constexpr (PL > 1) return entry_sums_fp32<EIGHTS>(a, i, slot, j0, lane);
  else return entry_sums<S, E, EIGHTS>(a, i, j0, lane);
}

// NW waves per position: the tiles' statistics become its lse.  The logits of the target and
// of the entries are the ones in these sums (a small loss is the difference of large terms);
// the sum over the entries is taken in fp64.
// ENTRIES (distillation) is a variant of its own, because the gather's registers halve the
// occupancy.
template <class S, class E, int PL, int NW, bool ENTRIES>
__global__ __launch_bounds__(256) void k_loss(LossArgs a, int ticket) {
  __shared__ float s_m[4], s_s[4], s_z[4];
  __shared__ double s_d[4], s_q[4];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, part = wv % NW;
  const int64_t i = (int64_t)blockIdx.x * (4 / NW) + wv / NW;
  const int slot = i < a.N ? slot_of(a, i) : -1;
  if (a.direct && !a.k && slot < 0 && i < a.N && lane == 0 && bad_target(a, i))
    set_status(a.status, TT_DEV_BAD_INDEX);
  const float zs = a.direct ? LOG2E / a.temp : a.sv.sc->zs;
  float out = 0.f, wm = -INFINITY, s = 0.f, z = 0.f;
  if (slot >= 0) {
    const Stats w = wave_stats(a, slot, part * 64 + lane, a.fold ? 1 : a.ptiles, 64 * NW, zs);
    wm = w.m, s = w.s, z = w.z;
  }
  if constexpr (NW > 1) {
    if (lane == 0) s_m[wv] = wm, s_s[wv] = s, s_z[wv] = z;
    __syncthreads();
    const int w0 = wv - part;
    wm = s_m[w0];
    for (int w = 1; w < NW; ++w) wm = fmaxf(wm, s_m[w0 + w]);
    const float m0 = wm == -INFINITY ? 0.f : wm;
    s = z = 0.f;
    for (int w = w0; w < w0 + NW; ++w) {
      s += s_s[w] * __builtin_amdgcn_exp2f((s_m[w] - m0) * zs);
      z += s_z[w];
    }
  }
  const float mx = wm == -INFINITY ? 0.f : wm, lg = log2f(s);
  double qd = 0.0;  // sum over the entries of q (lse - logit), base 2
  float far = fabsf(mx);
  if (ENTRIES && slot >= 0) {
    for (int j0 = part * 16; j0 < a.k; j0 += 16 * NW) {
      if (a.sv.eidx[i * a.k + j0] < 0) break;  // the empty ones are last
      const f4 sums = a.D % 8 == 0 ? sums_of<S, E, PL, true>(a, i, slot, j0, lane)
                                   : sums_of<S, E, PL, false>(a, i, slot, j0, lane);
      const int c = lane & 15, j = j0 + 4 * (lane >> 4) + c;
      const int64_t t = i * a.k + j;
      if (c >= 4 || j >= a.k || a.sv.eidx[t] < 0) continue;
      const float z = c == 0 ? sums[0] : c == 1 ? sums[1] : c == 2 ? sums[2] : sums[3];
      const float q = a.sv.eq[t];
      const double lp = ((double)z - mx) * zs - lg;
      if (!(q == 0.f)) qd -= q * lp, far = fmaxf(far, fabsf(z));
      a.sv.ez[t] = (float)lp;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) qd += __shfl_xor(qd, o);
  }
  if (NW > 1 && ENTRIES) {
    if (lane == 0) s_q[wv] = qd;
    __syncthreads();
    qd = 0.0;
    for (int w = 0; w < NW; ++w) qd += s_q[wv - part + w];
  }
  const bool first = lane == 0 && part == 0 && i < a.N;
  if (slot >= 0 && !ENTRIES) far = fmaxf(far, fabsf(a.sv.zt[slot]));
  if (a.dtype == TT_DTYPE_BF16 && !a.direct && slot >= 0 && !(far < G_PLAIN))
    atomicMin(&a.sv.sc->ge, 0);
  if (slot >= 0 && first) {
    a.sv.mx[slot] = mx;
    a.sv.lg[slot] = lg;
    if (ENTRIES) {
      out = (float)((double)(a.temp * a.temp) * (a.sv.ent[i] + qd * LN2));
    } else {
      const float nll = (mx - a.sv.zt[slot]) * zs + lg;  // no difference of large sums
      out = a.smoothing > 0.f ? (1.f - a.smoothing) * nll +
                                    a.smoothing * (mx * zs + lg - z / (float)a.V)
                              : nll;
      out *= LN2;
    }
  }
  if (a.reduction == TT_REDUCE_NONE) {
    if (first) a.loss[i] = out;
    return;
  }
  if (!ticket) {
    if (first) a.rowloss[i] = out;
    return;
  }
  // The block that ends last adds the rows up.  A row is written through to memory by its own
  // scope and the ticket waits for these stores alone (a fence would write back the XCD's
  // whole L2, in every block).
  if (first) __hip_atomic_store(&a.rowloss[i], out, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  vmem_drain();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.sv.sc->ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (s_last) sum_rows<256>(a, s_d);
}

// the rows' sum in a launch of its own
__global__ __launch_bounds__(1024) void k_loss_sum(LossArgs a) {
  __shared__ double s_d[16];
  sum_rows<1024>(a, s_d);
}

// ---------------------------------------------------------------- backward, around the products
// With a gradient per position: the factor of every packed row's g.  G in fp16 needs |factor|
// <= 1 (2^14 g fits), so the factors are divided by the power of two above the largest finite
// one; light ones come in two parts, see LIGHT.  The blocks find the largest for themselves, from
// FACTORS_AT positions on from what k_row_max found.
__device__ __forceinline__ float block_max_factor(const LossArgs &a, int64_t i0, int64_t step) {
  __shared__ float s_m[4];
  const int tid = threadIdx.x;
  float m = 0.f;
#pragma unroll 4
  for (int64_t i = i0 + tid; i < a.N; i += step) {
    const float u = fabsf(gradient_of(a, i));
    if (u < INFINITY && a.sv.slot[i] >= 0) m = fmaxf(m, u);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((tid & 63) == 0) s_m[tid >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
}
__global__ __launch_bounds__(256) void k_row_max(LossArgs a) {
  const float m = block_max_factor(a, (int64_t)blockIdx.x * 256, 256 * gridDim.x);
  if (threadIdx.x == 0) a.upmax[blockIdx.x] = m;
}
__global__ __launch_bounds__(256) void k_row_factors(LossArgs a) {
  const int tid = threadIdx.x;
  float cm = 1.f;
  const bool scaled = a.dtype != TT_DTYPE_BF16 && !a.sv.sc->whole;
  if (scaled) {
    float m;
    if (a.upmax) {
      m = 0.f;
      for (int b = tid & 63; b < FACTOR_BLOCKS; b += 64) m = fmaxf(m, a.upmax[b]);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    } else {
      m = block_max_factor(a, 0, 256);
    }
    if (m > 0.f) {
      int e;
      frexpf(m, &e);
      cm = ldexpf(1.f, max(e, -120));
    }
  }
  if (blockIdx.x == 0 && tid == 0) *a.cm = cm;
  for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < a.N; i += (int64_t)gridDim.x * 256) {
    const int slot = a.sv.slot[i];
    if (slot < 0) continue;
    const float f = gradient_of(a, i) / cm;
    int e = 0;
    if (scaled && fabsf(f) < INFINITY) {
      frexpf(f, &e);
      e = min(e + LIGHT, 0);
    }
    a.rowf[slot] = ldexpf(f, -e);
    a.rowe[slot] = e;
  }
}

// G of the light rows at its right size, for dweight: blockIdx.y takes LIGHT_BYTES of a row
constexpr int LIGHT_BYTES = 16 * 256 * 4;
__global__ __launch_bounds__(256) void k_light_rows(LossArgs a) {
  const int count = a.sv.sc->count;
  const int64_t c0 = (int64_t)blockIdx.y * (LIGHT_BYTES / 16), c1 = min(c0 + LIGHT_BYTES / 16, a.ldG / 16);
  for (int64_t r = blockIdx.x; r < count; r += gridDim.x) {
    const int e = a.rowe[r];
    if (e == 0) continue;
    const float s = ldexpf(1.f, e);
    for (int part = 0; part < (a.twin ? 2 : 1); ++part) {
      hf8 *g = (hf8 *)(a.G + (r + part * a.twin) * a.ldG);
#pragma unroll 4
      for (int64_t c = c0 + threadIdx.x; c < c1; c += 256) {
        hf8 v = g[c];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = (_Float16)((float)v[u] * s);
        g[c] = v;
      }
    }
  }
}

// G at the entries of this piece: (p - q) from the entry's own logit, rounded like the rest
template <class E, int PL>
__global__ __launch_bounds__(256) void k_entries_g(LossArgs a, int64_t v0, int64_t nv) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.N * a.k) return;
  const int64_t i = t / a.k;
  const int slot = a.sv.slot[i];
  const int64_t v = a.sv.eidx[t] - v0;
  if (slot < 0 || a.sv.eidx[t] < 0 || v < 0 || v >= nv) return;
  if (t > i * a.k && a.sv.eidx[t - 1] == a.sv.eidx[t]) return;  // its row's first has all of q
  const bool whole = PL > 1 && a.sv.sc->whole;
  const int x = a.sv.sc->ge;
  const float q = ldexpf(__builtin_amdgcn_exp2f(0.5f * a.sv.ez[t]), x / 2);
  const float g = (q * q - ldexpf(a.sv.eq[t], x)) *
                  (a.reduction == TT_REDUCE_NONE ? a.rowf[slot] : 1.f);
  char *o = a.G + slot * a.ldG + v * 2;
  if (whole) {
    *(unsigned short *)o = (unsigned short)(__float_as_uint(g) >> 16);
    *(unsigned short *)(o + a.Gplane) = (unsigned short)__float_as_uint(g);
    return;
  }
  const typename E::e h = (typename E::e)g;
  *(typename E::e *)o = h;
  if (PL > 1 || a.twin) *(typename E::e *)(o + a.Gplane) = (typename E::e)(g - (float)h);
}

// dh: the splits added in order (2048 x 2048, four splits: 84 MB in 22 us), scaled, rounded once, put back at the position's row
template <class O>
__global__ __launch_bounds__(256) void k_dhidden_out(LossArgs a, DhPlan plan, GradScale scale) {
  const int rows = a.twin ? 2 * a.twin : a.sv.sc->count;
  const int ns = dh_splits(plan, rows, threadIdx.x & 63);
  const int64_t st = dh_split_stride(rows, plan.by, a.Dp);
  const float c_dh = scale.get(a.sv.sc->ew);
  const int per = (int)((a.D + 1023) / 1024);
  for (int64_t b = blockIdx.x; b < a.N * per; b += gridDim.x) {
    const int64_t i = b / per, c = ((b - i * per) * 256 + threadIdx.x) * 4;
    if (c >= a.D) continue;
    const int slot = a.sv.slot[i];
    f4 v = zero4();
    if (slot >= 0) {
      const float *p = a.dhp + (int64_t)slot * a.Dp + c;
#pragma unroll 4
      for (int k = 0; k < ns; ++k) v += *(const f4 *)(p + k * st);
      if (a.twin) {
        f4 w = zero4();
#pragma unroll 4
        for (int k = 0; k < ns; ++k) w += *(const f4 *)(p + a.twin * a.Dp + k * st);
        v += w;
      }
      v *= c_dh;
      if (a.reduction == TT_REDUCE_NONE) {
        const int e = a.rowe[slot];
        if (e)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = ldexpf(v[r], e);
      }
    }
    O *o = (O *)a.dh + i * a.D + c;
    typedef O o4 __attribute__((ext_vector_type(4)));
    struct __attribute__((packed, aligned(2))) any { o4 v; };
    any w;
#pragma unroll
    for (int r = 0; r < 4; ++r) w.v[r] = (O)v[r];
    if (c + 4 <= a.D) {
      *(any *)o = w;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c + r < a.D) o[r] = w.v[r];
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_fill0(T *x, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    x[i] = (T)0.f;
}

// ---------------------------------------------------------------- plan
// Which tiles, by the rounds they take on the CUs.  A round of 256 x 256 tiles (one per CU)
// runs at about 1.45 PFLOP/s; 128 x 128 tiles reach 1.03 with two on every CU and 0.86 with
// one (the products 4096 x 2048 x 2048 and 2048 x 2048 x 2048: half a round and a fourth).  So
// a last round of few large tiles is cheaper in small ones: 784 tiles on 256 CUs take 3 + 0.42
// rounds instead of 4.
int64_t large_tiles(int64_t along, int64_t across, int cus) {
  auto rounds = [&](int64_t n) { return (double)((n + cus - 1) / cus); };
  const int64_t keep = along * across / cus * cus / across;  // tiles of the whole rounds
  const int64_t small = 4 * (along - keep) * across;
  const double cut = rounds(keep * across) + (small <= cus ? 0.42 : 0.7 * rounds((small + 1) / 2));
  return cut + 0.05 < rounds(along * across) ? keep : along;
}

// Smaller ones, so that few tiles still fill the CUs: 1024 x 1024 x 2048 runs at 0.23 PFLOP/s
// in 64 tiles of 128 x 128, 0.24 in 128 of half that and 0.29 in 256 of a fourth.
GemmShape gemm_shape(int64_t x, int64_t y, int cus) {
  const int64_t m = ((x + 127) / 128) * ((y + 127) / 128);
  if (y <= 64) return m > cus / 2 ? GemmShape{2, 128, 64} : GemmShape{4, 64, 64};
  if (m <= cus / 4) return {4, 64, 64};
  if (x <= 64 || m <= cus / 2) return {3, 64, 128};
  return m <= cus ? GemmShape{5, 128, 128} : GemmShape{1, 128, 128};
}

// dh's tiles are few where positions and width are; the vocabulary is split then
GemmShape dh_shape(const LossArgs &a) {
  const int64_t rows = dh_rows(a), big = ((a.D + 255) / 256) * ((rows + 255) / 256);
  if (rows > 128 && a.D > 128 && big * std::min<int64_t>(DH_SPLITS, a.piece / 512) >= 128)
    return {0, 256, 256};
  if (a.D <= 64 && rows > 64) return {3, 64, 128};
  return rows > 64 ? GemmShape{1, 128, 128} : GemmShape{2, 128, 64};
}

// Memory for one piece of the vocabulary: G of every position, and the packed weight.  256
// MiB each keeps a piece about the size of the last-level cache; it is the whole of what the
// backward holds beside its outputs, whatever V is.
constexpr int64_t PIECE_BYTES = 256ll << 20;

static int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct Bump {
  char *base;
  int64_t off = 0;
  template <class T>
  void take(T *&p, int64_t n) {
    p = (T *)(base + off);
    off = round_up(off + n * (int64_t)sizeof(T), 256);
  }
};

int64_t saved_layout(LossArgs &a, void *saved) {
  Bump b{(char *)saved};
  b.take(a.sv.sc, 1);
  if (!a.direct) b.take(a.sv.hp, a.Npad * a.Dp * 2 * a.planes);
  b.take(a.sv.slot, a.N);
  b.take(a.sv.tgt, a.N);
  b.take(a.sv.mx, a.N);
  b.take(a.sv.lg, a.N);
  b.take(a.sv.zt, a.k ? 0 : a.N);
  if (a.k) {
    b.take(a.sv.ent, a.N);
    b.take(a.sv.eidx, a.N * a.k);
    b.take(a.sv.eq, a.N * a.k);
    b.take(a.sv.ez, a.N * a.k);
  }
  return b.off;
}

// elements between rows that tiles are loaded from: 256 of them inside one buffer descriptor
constexpr int64_t MAX_STRIDE = 1 << 21;

static int64_t elem_size(int dtype) { return dtype == TT_DTYPE_F32 ? 4 : 2; }

// Positions past which k_count goes before k_pack.  A loss alone of n x 200 x 64, without and
// with it: 4096 18 and 21 us, 8192 25 and 24, 16384 43 and 31, 131072 1025 and 126, 2^20 76 ms
// and 0.8 ms.
constexpr int64_t CHUNKS_AT = 8192;
// Positions past which k_row_max goes before k_row_factors (the backward of n x 200 x 64 for dhidden:
// 16384 64 us without and 66 with it, 32768 99 and 77, 131072 426 and 228, 2^20 4.1 and 1.7 ms).
constexpr int64_t FACTORS_AT = 16384;

// mode: TT_LOSS_FORWARD, _BACKWARD or _ONLY (what is saved otherwise is in the workspace then)
int64_t ws_layout(LossArgs &a, void *ws, int mode) {
  const bool grad = mode == TT_LOSS_BACKWARD;
  Bump b{(char *)ws};
  if (mode == TT_LOSS_ONLY) {
    // up to 64 positions fill one tile whether they count or not: nothing to pack, if whole
    // 16-byte groups make up their rows (and a tile of them fits a descriptor)
    a.direct = a.N <= 64 && a.D % 8 == 0 && a.planes == 1 && a.hld <= MAX_STRIDE;
    // fp32 rows of the weight are read once that way, and four times where they are packed (64 x 32000 x
    // 1024: 52 us of products in fp32, and 102 us of the tensors' range, packing and products)
    if (a.few32 && a.planes == 2 && !a.k && a.N <= 64 && a.hld <= MAX_STRIDE / 2 && a.wld <= MAX_STRIDE / 2) {
      a.direct = a.f32 = 1;
      a.planes = 1;
      a.pack_w = 0;
    }
    b.off = saved_layout(a, ws);
  }
  b.take(a.amax, grad || a.planes == 1 ? 0 : 3 * 2 * AMAX_BLOCKS);
  int64_t rows = a.V;
  const int64_t wrow = a.Dp * 2 * a.planes, grow = a.Npad * 2 * a.planes;
  int64_t lim = (1ll << 38) / std::max<int64_t>(a.Npad, 256);  // tiles of one launch
  if (a.pack_w) lim = std::min(lim, PIECE_BYTES / wrow);
  if (grad) lim = std::min(lim, PIECE_BYTES / grow);
  if (lim < rows) {  // pieces of near-equal size, whole tiles each
    const int64_t n = (rows + std::max<int64_t>(lim, 256) - 1) / std::max<int64_t>(lim, 256);
    rows = round_up((rows + n - 1) / n, 256);
  }
  a.piece = rows;
  if (a.pack_w) b.take(a.wp, rows * wrow);
  if (grad) {
    b.take(a.cm, 1);
    b.take(a.rowf, a.reduction == TT_REDUCE_NONE ? a.Npad : 0);
    b.take(a.rowe, a.reduction == TT_REDUCE_NONE ? a.Npad : 0);
    if (a.N > FACTORS_AT && a.reduction == TT_REDUCE_NONE && a.dtype != TT_DTYPE_BF16)
      b.take(a.upmax, FACTOR_BLOCKS);
    a.Gplane = round_up(std::min(rows, a.V), 256) * 2;
    a.ldG = a.Gplane * a.planes;
    if (a.twin) a.Gplane = a.twin * a.ldG;
    b.take(a.G, a.Npad * a.ldG);
    const GemmShape t = dh_shape(a);
    a.dh_bx = t.bx; a.dh_by = t.by;
    const int64_t ty = (dh_rows(a) + t.by - 1) / t.by, tx = (a.D + t.bx - 1) / t.bx;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(DH_SPLITS, rows / 512));
    b.take(a.dhp, std::max(ty, std::min<int64_t>(DH_TILES / tx, most * ty)) * t.by * a.Dp);
  } else {
    // statistics of all tiles where they fit, else of a piece's at a time
    const int64_t most = PIECE_BYTES / (a.Npad * (a.smoothing > 0.f ? 12 : 8));
    auto tiles = [&]() {
      int64_t n = 0;
      for (int64_t v0 = 0; v0 < a.V; v0 += a.piece) n += logits_cut(a, std::min(a.piece, a.V - v0)).tiles;
      return n;
    };
    int64_t all = tiles();
    a.fold = all > most;
    if (a.fold) {
      auto widest = [&]() {  // of a whole piece and the last one
        const int64_t last = a.V - (a.V - 1) / a.piece * a.piece;
        return std::max(logits_cut(a, std::min(a.piece, a.V)).tiles, logits_cut(a, last).tiles);
      };
      while (a.piece > 256 && widest() + 1 > most) a.piece = round_up(a.piece / 2, 256);
      all = widest() + 1;
    }
    a.ptiles = (int)all;
    b.take(a.part, a.Npad * a.ptiles);
    b.take(a.zpart, a.smoothing > 0.f ? a.Npad * a.ptiles : 0);
    b.take(a.rowloss, a.N);
    if (a.N > CHUNKS_AT) b.take(a.chunk, (a.N + CHUNK - 1) / CHUNK);
    if (a.N > CHUNKS_AT) b.take(a.chunk, (a.N + CHUNK - 1) / CHUNK);
  }
  return b.off;
}

int loss_args(const tt_loss_desc *d, const void *weight, LossArgs &a) {
  if (!d) return TT_EINVAL;
  if (d->n < 0 || d->v < 1 || d->d < 1 || d->k < 0) return TT_EINVAL;
  if (d->dtype < TT_DTYPE_F32 || d->dtype > TT_DTYPE_F16) return TT_EINVAL;
  if (d->teacher_dtype < TT_DTYPE_F32 || d->teacher_dtype > TT_DTYPE_F16) return TT_EINVAL;
  if (d->reduction < TT_REDUCE_NONE || d->reduction > TT_REDUCE_SUM) return TT_EINVAL;
  if (!(d->label_smoothing >= 0.f && d->label_smoothing <= 1.f)) return TT_EINVAL;
  if (!(d->temperature > 0.f && d->temperature < INFINITY)) return TT_EINVAL;
  if (d->k ? d->label_smoothing != 0.f : d->temperature != 1.f) return TT_EINVAL;
  if (d->hidden_stride < d->d || d->weight_stride < d->d) return TT_EINVAL;
  // 32-bit places of positions, rows and entries; a tile's rows inside one descriptor
  if (d->n > (1 << 23) || d->v > (1 << 30) || d->d > (1 << 20) || d->k > 2048) return TT_ESHAPE;
  if (d->weight_stride > MAX_STRIDE) return TT_ESHAPE;
  if (d->n * std::max(d->k, 1) > (1ll << 31)) return TT_ESHAPE;
  a = {};
  a.N = d->n; a.V = d->v; a.D = d->d; a.hld = d->hidden_stride; a.wld = d->weight_stride;
  a.dtype = d->dtype; a.tdtype = d->teacher_dtype; a.reduction = d->reduction; a.k = d->k;
  a.ignore = d->ignore_index; a.smoothing = d->label_smoothing; a.temp = d->temperature;
  a.weight = weight;
  a.Npad = round_up(std::max<int64_t>(a.N, 1), a.N > 128 ? 256 : a.N > 64 ? 128 : 64);
  a.Dp = round_up(a.D, 64);
  a.planes = a.dtype == TT_DTYPE_F32 ? 2 : 1;
  a.cus = std::max(device_cus(), 1);
  // G rounded to 16 bits adds to the gradients' error as much as their own rounding does where
  // many roundings average out, and half as much again where few do.  Up to 32 positions a
  // tile of 64 has room for what the rounding left.
  a.twin = a.planes == 1 && a.N <= 32 ? 32 : 0;
  // 16-bit rows of odd length are read as they lie, and the last tile of k is put right in LDS
  // for every tile of positions; where positions are many for the width, packing the weight
  // is cheaper (1294 x 99003 x 1389: 1205 us as they lie, 1420 packed; 3855 x 41825 x 124:
  // 312 and 298)
  a.pack_w = a.planes > 1 || (a.D % 8 && a.N >= 16 * a.D);
  return TT_OK;
}

template <class S, class E, int PL>
static hipError_t pack_h(const LossArgs &a, hipStream_t s) {
  tt_launch(K_LOSS_PACK, k_pack<S, E, PL>, dim3((unsigned)((a.Npad + PACK_ROWS - 1) / PACK_ROWS)),
            dim3(256), 0, s, a);
  return hipGetLastError();
}
template <class S, class E, int PL>
static hipError_t pack_w(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s) {
  const int64_t n = nv * (a.Dp / 8);
  tt_launch(K_LOSS_PACK, k_pack_w<S, E, PL>, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)),
            dim3(256), 0, s, a, v0, nv);
  return hipGetLastError();
}
static hipError_t launch_pack(const LossArgs &a, hipStream_t s) {
  if (a.chunk) {
    const int chunks = (int)((a.N + CHUNK - 1) / CHUNK);
    tt_launch(K_LOSS_PACK, k_count<false>, dim3(chunks), dim3(256), 0, s, a);
    tt_launch(K_LOSS_PACK, k_count_before, dim3(1), dim3(1024), 0, s, a, chunks);
  }
  if (a.dtype == TT_DTYPE_F32) {
    tt_launch(K_LOSS_PACK, k_amax, dim3(2 * AMAX_BLOCKS), dim3(256), 0, s, a);
    return pack_h<float, Fp16, 2>(a, s);
  }
  if (a.dtype == TT_DTYPE_BF16) return pack_h<__bf16, Bf16, 1>(a, s);
  return pack_h<_Float16, Fp16, 1>(a, s);
}
static hipError_t launch_pack_w(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s) {
  if (!a.pack_w) return hipSuccess;
  if (a.dtype == TT_DTYPE_F32) return pack_w<float, Fp16, 2>(a, v0, nv, s);
  if (a.dtype == TT_DTYPE_BF16) return pack_w<__bf16, Bf16, 1>(a, v0, nv, s);
  return pack_w<_Float16, Fp16, 1>(a, v0, nv, s);
}

static hipError_t launch_entries(const LossArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 3) / 4));
  int pow2 = 1;
  while (pow2 < a.k) pow2 *= 2;
  const size_t lds = (size_t)pow2 * 32;  // at most 64 KiB
  if (a.tdtype == TT_DTYPE_F32) tt_launch(K_LOSS_ROWS, k_entries<float>, grid, dim3(256), lds, s, a, pow2);
  else if (a.tdtype == TT_DTYPE_BF16) tt_launch(K_LOSS_ROWS, k_entries<__bf16>, grid, dim3(256), lds, s, a, pow2);
  else tt_launch(K_LOSS_ROWS, k_entries<_Float16>, grid, dim3(256), lds, s, a, pow2);
  return hipGetLastError();
}

// A sum of up to LOSS_TICKETS rows is taken by k_loss's last block; the tickets of all blocks
// go through one address at some 13 ns each (8192 rows: 140 us, of which 100 waited for
// them), so more rows are added in a launch of its own (about 5 us).
constexpr int64_t LOSS_TICKETS = 256;

static hipError_t launch_fold(const LossArgs &a, int tiles, int first, hipStream_t s) {
  tt_launch(K_LOSS_ROWS, k_fold, dim3((unsigned)std::min<int64_t>((a.N + 3) / 4, 1 << 16)),
            dim3(256), 0, s, a, tiles, first);
  return hipGetLastError();
}

template <class S, class E, int PL, bool ENTRIES>
static void launch_loss(const LossArgs &a, int ticket, hipStream_t s) {
  // few statistics: a wave per position and group of 16 entries
  const bool few = a.fold || a.ptiles <= 256;
  auto go = [&](auto *kernel, int nw) {
    tt_launch(K_LOSS_ROWS, kernel, dim3((unsigned)((a.N * nw + 3) / 4)), dim3(256), 0, s, a, ticket);
  };
  if (few && a.k <= 16) return go(k_loss<S, E, PL, 1, ENTRIES>, 1);
  if constexpr (ENTRIES)
    if (few && a.k <= 32) return go(k_loss<S, E, PL, 2, ENTRIES>, 2);
  go(k_loss<S, E, PL, 4, ENTRIES>, 4);
}

static hipError_t launch_loss(const LossArgs &a, hipStream_t s) {
  const int ticket = a.N <= LOSS_TICKETS && !a.direct;  // (k_pack clears the ticket)
  if (!a.k) launch_loss<_Float16, Fp16, 1, false>(a, ticket, s);  // (of any type)
  else if (a.dtype == TT_DTYPE_F32) launch_loss<float, Fp16, 2, true>(a, ticket, s);
  else if (a.dtype == TT_DTYPE_BF16) launch_loss<__bf16, Bf16, 1, true>(a, ticket, s);
  else launch_loss<_Float16, Fp16, 1, true>(a, ticket, s);
  if (a.reduction != TT_REDUCE_NONE && !ticket)
    tt_launch(K_LOSS_ROWS, k_loss_sum, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

static hipError_t launch_entries_g(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s) {
  if (!a.k) return hipSuccess;
  const dim3 grid((unsigned)((a.N * a.k + 255) / 256));
  if (a.dtype == TT_DTYPE_F32) tt_launch(K_LOSS_ROWS, k_entries_g<Fp16, 2>, grid, dim3(256), 0, s, a, v0, nv);
  else if (a.dtype == TT_DTYPE_BF16) tt_launch(K_LOSS_ROWS, k_entries_g<Bf16, 1>, grid, dim3(256), 0, s, a, v0, nv);
  else tt_launch(K_LOSS_ROWS, k_entries_g<Fp16, 1>, grid, dim3(256), 0, s, a, v0, nv);
  return hipGetLastError();
}

static hipError_t launch_dhidden_out(const LossArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(a.N * ((a.D + 1023) / 1024), 1 << 20));
  if (a.dtype == TT_DTYPE_F32) tt_launch(K_LOSS_ROWS, k_dhidden_out<float>, grid, dim3(256), 0, s, a, dh_plan(a), grad_scale(a));
  else if (a.dtype == TT_DTYPE_BF16) tt_launch(K_LOSS_ROWS, k_dhidden_out<__bf16>, grid, dim3(256), 0, s, a, dh_plan(a), grad_scale(a));
  else tt_launch(K_LOSS_ROWS, k_dhidden_out<_Float16>, grid, dim3(256), 0, s, a, dh_plan(a), grad_scale(a));
  return hipGetLastError();
}

static hipError_t launch_light_rows(const LossArgs &a, hipStream_t s) {
  if (a.reduction != TT_REDUCE_NONE || a.dtype == TT_DTYPE_BF16) return hipSuccess;
  const int64_t y = (a.ldG + LIGHT_BYTES - 1) / LIGHT_BYTES;
  tt_launch(K_LOSS_ROWS, k_light_rows,
            dim3((unsigned)std::min<int64_t>(a.N, std::max<int64_t>(1, 4096 / y)), (unsigned)y), dim3(256), 0, s, a);
  return hipGetLastError();
}

static hipError_t fill0(void *x, int64_t bytes, hipStream_t s) {
  if (bytes == 0) return hipSuccess;
  const int64_t n = bytes / 2;  // every output here has elements of 2 or 4 bytes
  hipLaunchKernelGGL(k_fill0<_Float16>, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)),
                     dim3(256), 0, s, (_Float16 *)x, n);
  return hipGetLastError();
}

hipError_t loss_forward(const LossArgs &a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.k) e = launch_entries(a, s);
  if (e == hipSuccess && !a.direct) e = launch_pack(a, s);
  int tile0 = 0;
  for (int64_t v0 = 0; v0 < a.V && e == hipSuccess; v0 += a.piece) {
    const int64_t nv = std::min(a.piece, a.V - v0);
    e = launch_pack_w(a, v0, nv, s);
    const int tiles = logits_cut(a, nv).tiles;
    if (e == hipSuccess) e = launch_logits(a, v0, nv, a.fold ? 1 : tile0, false, s);
    if (e == hipSuccess && a.fold) e = launch_fold(a, tiles, v0 == 0, s);
    tile0 += tiles;
  }
  return e == hipSuccess ? launch_loss(a, s) : e;
}

int64_t kept_layout(const LossArgs &a, void *p, Kept &k) {
  Bump b{(char *)p};
  k = {};
  b.take(k.to.sc, 1);
  b.take(k.to.hp, a.Npad * a.Dp * 2 * a.planes);
  b.take(k.to.slot, a.N);
  b.take(k.to.tgt, a.N);
  b.take(k.to.mx, a.N);
  b.take(k.to.lg, a.N);
  if (a.N > CHUNKS_AT) b.take(k.chunk, (a.N + CHUNK - 1) / CHUNK);
  return b.off;
}

hipError_t keep_rows(LossArgs &a, const Kept &k, hipStream_t s) {
  a.chunk = k.chunk;
  if (a.chunk) {
    const int chunks = (int)((a.N + CHUNK - 1) / CHUNK);
    tt_launch(K_LOSS_PACK, k_count<true>, dim3(chunks), dim3(256), 0, s, a);
    tt_launch(K_LOSS_PACK, k_count_before, dim3(1), dim3(1024), 0, s, a, chunks);
  }
  tt_launch(K_LOSS_PACK, k_keep, dim3((unsigned)((a.Npad + PACK_ROWS - 1) / PACK_ROWS)), dim3(256), 0, s, a,
            k.to, a.Dp * 2 * a.planes);
  a.sv = k.to;
  return hipGetLastError();
}

hipError_t loss_backward(const LossArgs &a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.N == 0) return a.dw ? fill0(a.dw, a.V * a.D * elem_size(a.dtype), s) : e;
  if (!a.dh && !a.dw) return e;
  if (a.reduction == TT_REDUCE_NONE) {
    if (a.upmax) tt_launch(K_LOSS_ROWS, k_row_max, dim3(FACTOR_BLOCKS), dim3(256), 0, s, a);
    tt_launch(K_LOSS_ROWS, k_row_factors, dim3((unsigned)std::min<int64_t>((a.N + 255) / 256, 1024)),
              dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  for (int64_t v0 = 0; v0 < a.V && e == hipSuccess; v0 += a.piece) {
    const int64_t nv = std::min(a.piece, a.V - v0);
    e = launch_pack_w(a, v0, nv, s);
    if (e == hipSuccess) e = launch_logits(a, v0, nv, 0, true, s);
    if (e == hipSuccess) e = launch_entries_g(a, v0, nv, s);
    if (e == hipSuccess && a.dh) e = launch_dhidden(a, v0, nv, s);
    if (e == hipSuccess && a.dw) e = launch_light_rows(a, s);
    if (e == hipSuccess && a.dw) e = launch_dweight(a, v0, nv, s);
  }
  return e == hipSuccess && a.dh ? launch_dhidden_out(a, s) : e;
}

}  // namespace ttb

using namespace ttb;

extern "C" {

size_t tt_loss_saved_size(const tt_loss_desc *desc) {
  LossArgs a;
  return loss_args(desc, nullptr, a) == TT_OK ? (size_t)saved_layout(a, nullptr) : 0;
}

size_t tt_loss_workspace_size(const tt_loss_desc *desc, const void *weight, int mode) {
  LossArgs a;
  if (mode < TT_LOSS_FORWARD || mode > TT_LOSS_ONLY) return 0;
  return loss_args(desc, weight, a) == TT_OK ? (size_t)ws_layout(a, nullptr, mode) : 0;
}

int tt_loss_forward(const tt_loss_desc *desc, const void *hidden, const void *weight,
                    const int64_t *targets, const void *teacher_logits, float *loss, void *saved,
                    size_t saved_bytes, void *ws, size_t ws_bytes, int32_t *dev_status,
                    void *stream) {
  LossArgs a;
  const int rc = loss_args(desc, weight, a);
  if (rc != TT_OK) return rc;
  if (!weight || !ws) return TT_EINVAL;
  if (!loss && (a.N || a.reduction != TT_REDUCE_NONE)) return TT_EINVAL;
  if (a.N && (!hidden || !targets || (a.k && !teacher_logits))) return TT_EINVAL;
  if ((uintptr_t)weight % elem_size(a.dtype) || (uintptr_t)hidden % elem_size(a.dtype)) return TT_EINVAL;
  if ((uintptr_t)saved % 256 || (uintptr_t)ws % 256) return TT_EWORKSPACE;
  if (saved && (size_t)saved_layout(a, saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)ws_layout(a, ws, saved ? TT_LOSS_FORWARD : TT_LOSS_ONLY) > ws_bytes) return TT_EWORKSPACE;
  a.hidden = hidden; a.tgt = targets; a.tlogits = teacher_logits; a.loss = loss;
  a.status = dev_status;
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (a.N > 0) e = loss_forward(a, s);
  else if (a.reduction != TT_REDUCE_NONE) e = fill0(loss, 4, s);  // a sum or mean of nothing is 0
  return e == hipSuccess ? TT_OK : TT_EHIP;
}

int tt_loss_backward(const tt_loss_desc *desc, const void *hidden, const void *weight,
                     const void *saved, size_t saved_bytes, const float *grad_loss,
                     void *grad_hidden, void *grad_weight, void *ws, size_t ws_bytes,
                     void *stream) {
  LossArgs a;
  const int rc = loss_args(desc, weight, a);
  if (rc != TT_OK) return rc;
  if (!weight || !saved || !ws || (a.N && (!hidden || !grad_loss))) return TT_EINVAL;
  if ((uintptr_t)weight % elem_size(a.dtype) || (uintptr_t)hidden % elem_size(a.dtype) ||
      (uintptr_t)grad_hidden % elem_size(a.dtype) || (uintptr_t)grad_weight % elem_size(a.dtype))
    return TT_EINVAL;
  if ((uintptr_t)saved % 256 || (uintptr_t)ws % 256) return TT_EWORKSPACE;
  if ((size_t)saved_layout(a, (void *)saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)ws_layout(a, ws, TT_LOSS_BACKWARD) > ws_bytes) return TT_EWORKSPACE;
  a.hidden = hidden; a.up = grad_loss; a.dh = grad_hidden; a.dw = grad_weight;
  return loss_backward(a, (hipStream_t)stream) == hipSuccess ? TT_OK : TT_EHIP;
}

}  // extern "C"
