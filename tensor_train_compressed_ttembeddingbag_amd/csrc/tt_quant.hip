// tt_quant.hip -- tables in 8-bit integers with a scale for each row, and their product with
// hidden states that get a scale for each token:
//   s_i = max |x_i| / 127,  q_i = round(x_i / s_i) to even,   out_iv = s_i t_v sum_k q_ik w_vk
// The sum is one of whole numbers, exact in 32 bits up to 131072 columns; the two scales are
// multiplied onto it in fp32 and the result is rounded once.
//
// The product runs on the tiles of tt_gemm.h: v_mfma_i32_16x16x64_i8 has the operand layout of the
// 16-bit instructions byte for byte, at twice the operations, so a row of d bytes is one of d / 2
// 16-bit columns there.
#include "tt_gemm.h"
#include "tt_internal.h"
#include "tt_loss.h"
#include "tt_rows.h"

#include <algorithm>

namespace ttb {

struct QuantArgs {
  int64_t n, d, ld, pitch;  // ld in elements, pitch in bytes
  const void *x;
  int8_t *q;
  float *s;
};

// A row with a value that is not finite gets the scale NaN and zeros, one whose scale would be below the
// normal numbers the scale 0 and zeros.
__device__ __forceinline__ float row_max(float m, float x) {
  const float f = fabsf(x);
  return f <= m ? m : f == f ? f : INFINITY;
}
__device__ __forceinline__ float row_scale(float m) {
  const float s = m / 127.f;
  return !(m < INFINITY) ? __builtin_nanf("") : s < 0x1p-126f ? 0.f : s;
}
__device__ __forceinline__ int8_t row_value(float x, float s) {
  return s > 0.f ? (int8_t)(int)fminf(fmaxf(rintf(x / s), -127.f), 127.f) : (int8_t)0;
}

// NT lanes a row; U groups of eight of each stay in registers between the maximum and the rounding,
// wider rows are read twice.
template <class S, int NT, bool NARROW>
__global__ __launch_bounds__(256) void k_quantize(QuantArgs a) {
  constexpr int U = 4;
  __shared__ float s_m[4];
  const int tid = threadIdx.x % NT, lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT;
  const bool on = r < a.n;
  const S *x = (const S *)a.x + (on ? r : 0) * a.ld;
  const int64_t cpr = (a.d + 7) / 8;
  Eight<S> v[U];
  auto load = [&](int64_t g0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = get8<NARROW>(x + column<NARROW>(min(g0 + u * NT + tid, cpr - 1), a.d), a.d);
  };
  float m = 0.f;
  for (int64_t g0 = 0; g0 < cpr; g0 += U * NT) {
    load(g0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = row_max(m, (float)v[u].x[e]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if constexpr (NT > 64) {
    if (lane == 0) s_m[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  }
  if (!on) return;
  const float s = row_scale(m);
  if (tid == 0) a.s[r] = s;
  int8_t *q = a.q + r * a.pitch;
  for (int64_t g0 = 0; g0 < cpr; g0 += U * NT) {
    if (cpr > U * NT) load(g0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * NT + tid;
      if (g >= cpr) break;
      Eight<int8_t> o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o.x[e] = row_value((float)v[u].x[e], s);
      put8<NARROW>(q + column<NARROW>(g, a.d), o, a.d);
    }
  }
  for (int64_t c = a.d + tid; c < a.pitch; c += NT) q[c] = 0;
}

// Rows that come in 8 bits, with the bytes behind them cleared: a product runs over whole groups of
// 16, and the table's may hold anything there.
__global__ __launch_bounds__(256) void k_pad_rows(QuantArgs a) {
  const int8_t *x = (const int8_t *)a.x;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n * a.pitch; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / a.pitch, c = i - r * a.pitch;
    a.q[i] = c < a.d ? x[r * a.ld + c] : (int8_t)0;
  }
}

template <class O>
struct Int8Out {
  O *out;
  const float *s, *t;  // a scale per token, per row of the table
  int64_t ld;
  int n, v;
};

// A tile with room for a wave's results on their way out: 16 tokens by ROW bytes, as much as leaves the tile
// its place beside another one on the CU.
template <class O, class T>
struct WithRows : T {
  static constexpr int MOST = T::X == 256 ? 256 : 128;
  static constexpr int ROW = T::wx * (int)sizeof(O) < MOST ? T::wx * (int)sizeof(O) : MOST;
  static constexpr int EXTRA = T::NT / 64 * 16 * ROW;
  static constexpr int LDS = T::LDS - T::EXTRA + EXTRA;
  // 16-byte group k of row r, permuted so that neither writes nor reads meet in a bank
  static __device__ __forceinline__ int at(int r, int k) {
    return r * ROW + (k ^ (r * ROW / 256 & (ROW / 16 - 1))) * 16;
  }
};

// A lane's results are four columns of one token.  Stored from there they are 64 bytes of each of 16 rows
// at a time; they go through LDS instead, for each wave by itself, and leave as whole rows of up to 256
// bytes: 4096 x 50021 x 2048 to bf16 500 -> 403 us, to fp32 645 -> 514, with 50048 rows 428 -> 390.
template <class O, class T>
__global__ __launch_bounds__(T::NT) void k_int8(GemmArgs a, Int8Out<O> ep) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int C = 16 / sizeof(O);                 // columns of 16 bytes
  constexpr int W = T::ROW / (int)sizeof(O);          // columns that go together
  typedef O o4 __attribute__((ext_vector_type(4)));
  gemm_tiles<Int8, T, 1, false, false, false, false>(
      a, lds, [&](const TileAt &at, i32x4 (&acc)[T::MI][T::NI], char *tmp) {
        const int tid = own_thread(), lane = tid & 63, wv = tid >> 6, g = lane >> 4, c = lane & 15;
        const int x = at.ix * T::X + (wv % T::NWX) * T::wx;
        const int y = at.iy * T::Y + (wv / T::NWX) * T::wy;
        char *rows = tmp + wv * 16 * T::ROW;
        // all scales at once: one wait for memory, not one for each pair of columns
        float s[T::NI], t[T::MI][4];
#pragma unroll
        for (int j = 0; j < T::NI; ++j) s[j] = ep.s[min(y + 16 * j + c, ep.n - 1)];
        if (at.ix * T::X + T::X <= ep.v) {
          struct __attribute__((packed, aligned(4))) any { f4 v; };
#pragma unroll
          for (int i = 0; i < T::MI; ++i) {
            const f4 v = ((const any *)(ep.t + x + 16 * i + 4 * g))->v;
#pragma unroll
            for (int r = 0; r < 4; ++r) t[i][r] = v[r];
          }
        } else {
#pragma unroll
          for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) t[i][r] = ep.t[min(x + 16 * i + 4 * g + r, ep.v - 1)];
        }
#pragma unroll
        for (int j = 0; j < T::NI; ++j)
#pragma unroll
          for (int i0 = 0; i0 < T::MI; i0 += W / 16) {
#pragma unroll
            for (int i = 0; i < W / 16; ++i) {
              o4 v;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                // (kept: fp32 by itself, not one rounding with the conversion to fp16)
                const float z = keep((float)acc[i0 + i][j][r] * s[j] * t[i0 + i][r]);
                v[r] = (O)z;
              }
              const int col = 16 * i + 4 * g;
              *(o4 *)(rows + T::at(c, col / C) + col % C * sizeof(O)) = v;
            }
            wave_lds_sync();
            constexpr int LPR = W / C;  // lanes of a row
#pragma unroll
            for (int p = 0; p < LPR / 4; ++p) {
              const int r = p * (64 / LPR) + lane / LPR, k = lane % LPR;
              const i32x4 v = *(const i32x4 *)(rows + T::at(r, k));
              const int col = x + 16 * i0 + k * C, left = ep.v - col;
              if (y + 16 * j + r >= ep.n || left <= 0) continue;
              O *o = ep.out + (int64_t)(y + 16 * j + r) * ep.ld + col;
              if (left >= C) {
                struct __attribute__((packed, aligned(2))) any { i32x4 v; };
                ((any *)o)->v = v;
              } else {
                union {
                  i32x4 v;
                  O e[C];
                } u = {v};
#pragma unroll
                for (int e = 0; e < C; ++e)
                  if (e < left) o[e] = u.e[e];
              }
            }
            wave_lds_sync();
          }
      });
}

// A few tokens in one launch: every workgroup quantises them for itself, into LDS, while its first rows of
// the table travel.  A wave takes 16 rows of the table at a time, straight from memory to the registers of
// v_mfma_i32_16x16x64_i8 (a lane has 16 bytes of a row), U loads ahead of the products.
// Bound by the table's bytes; what one launch less saves is 4 us of 15 (1 x 32000 x 1024).
constexpr int FEW_TOKENS = 16, FEW_VALUES = 4096;
constexpr int64_t FEW_BYTES = 48 << 20;
struct FewArgs {
  int64_t d, hld, pitch, wpitch, v;
  int n, lp;               // tokens; bytes between them in LDS
  const void *x;
  const int8_t *w;
  const float *t;
  void *out;
};
template <class S, class O, bool NARROW>
__global__ __launch_bounds__(256) void k_int8_few(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char q[];  // [n][lp], zeros behind d
  __shared__ float s_s[FEW_TOKENS];
  constexpr int U = 8;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int nk = (int)((a.d + 64 * U - 1) / (64 * U));  // loads of U x 64 bytes along a row
  const int64_t tiles = (a.v + 15) / 16, stride = (int64_t)gridDim.x * 4;
  int64_t tile = (int64_t)blockIdx.x * 4 + wv;
  i32x4 p[2][U];
  auto load = [&](int64_t tile, int kk, i32x4 (&to)[U]) {
    const int8_t *row = a.w + min(tile * 16 + c, a.v - 1) * a.wpitch;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = ((int64_t)kk * U + u) * 64 + 16 * g;
      to[u] = *(const i32x4 *)(row + (k < a.pitch ? k : 0));  // past the row: its q are zeros
    }
  };
  if (tile < tiles) load(tile, 0, p[0]);
  const int64_t cpr = (a.d + 7) / 8;
  for (int i = wv; i < a.n; i += 4) {
    const S *x = (const S *)a.x + i * a.hld;
    float m = 0.f;
#pragma unroll 4
    for (int64_t r = lane; r < cpr; r += 64) {
      const Eight<S> v = get8<NARROW>(x + column<NARROW>(r, a.d), a.d);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = row_max(m, (float)v.x[e]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float s = row_scale(m);
    if (lane == 0) s_s[i] = s;
    char *o = q + i * a.lp;
    for (int64_t k = a.d + lane; k < a.lp; k += 64) o[k] = 0;
#pragma unroll 4
    for (int64_t r = lane; r < cpr; r += 64) {
      const int64_t col = column<NARROW>(r, a.d);
      const Eight<S> v = get8<NARROW>(x + col, a.d);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!NARROW || e < a.d) o[col + e] = row_value((float)v.x[e], s);
    }
  }
  __syncthreads();
  const char *qc = q + min(c, a.n - 1) * a.lp + 16 * g;
  const float sc = s_s[min(c, a.n - 1)];
  auto multiply = [&](const i32x4 (&from)[U], int kk, i32x4 &acc) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      acc = Int8::mfma(from[u], *(const i32x4 *)(qc + (kk * U + u) * 64), acc);
  };
  for (; tile < tiles; tile += stride) {
    i32x4 acc = {};
    // pairs of loads, so that the register sets have their names at compile time
    for (int kk = 0; kk < nk; kk += 2) {
      if (kk + 1 < nk) load(tile, kk + 1, p[1]);
      else if (tile + stride < tiles) load(tile + stride, 0, p[1]);
      multiply(p[0], kk, acc);
      if (kk + 1 < nk) {
        if (kk + 2 < nk) load(tile, kk + 2, p[0]);
        else if (tile + stride < tiles) load(tile + stride, 0, p[0]);
        multiply(p[1], kk + 1, acc);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) p[0][u] = p[1][u];
      }
    }
    const int64_t row = tile * 16 + 4 * g;
    if (c < a.n) {
      O *o = (O *)a.out + c * a.v + row;
      O v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float z = keep((float)acc[r] * sc * a.t[min(row + r, a.v - 1)]);
        v[r] = (O)z;
      }
      if (row + 4 <= a.v) {
        struct __attribute__((packed, aligned(2))) any { O v[4]; };
        *(any *)o = {{v[0], v[1], v[2], v[3]}};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row + r < a.v) o[r] = v[r];
      }
    }
  }
}

// ---------------------------------------------------------------- host
// A launch has less than 2^32 threads: rows past what these workgroups take have launches of their own.  (A loop
// over rows in the kernel: 131072 x 4096 bf16 479 -> 494 us.)
constexpr int64_t MOST_BLOCKS = 1 << 20;
template <class S, bool NARROW>
static void go_quantize(const QuantArgs &all, hipStream_t s) {
  // a wave a row where it holds one in registers, or where rows are many
  const bool wave = all.d <= 1024 || (all.d <= 2048 && all.n >= 1024);
  const int64_t most = wave ? 4 * MOST_BLOCKS : MOST_BLOCKS;
  for (int64_t r = 0; r < all.n; r += most) {
    QuantArgs a = all;
    a.n = std::min(all.n - r, most);
    a.x = (const S *)all.x + r * all.ld;
    a.q += r * all.pitch;
    a.s += r;
    if (wave)
      tt_launch(K_INT8_QUANT, k_quantize<S, 64, NARROW>, dim3((unsigned)((a.n + 3) / 4)), dim3(256), 0, s, a);
    else
      tt_launch(K_INT8_QUANT, k_quantize<S, 256, NARROW>, dim3((unsigned)a.n), dim3(256), 0, s, a);
  }
}
template <class S>
static void go_quantize(const QuantArgs &a, hipStream_t s) {
  if (a.d < 8) go_quantize<S, true>(a, s);
  else go_quantize<S, false>(a, s);
}
static hipError_t quantize(const QuantArgs &a, int dtype, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  if (dtype == TT_DTYPE_F32) go_quantize<float>(a, s);
  else if (dtype == TT_DTYPE_BF16) go_quantize<__bf16>(a, s);
  else go_quantize<_Float16>(a, s);
  return hipGetLastError();
}

template <class O, class Plain>
static hipError_t go_int8(const GemmArgs &g, const Int8Out<O> &ep, int cus, hipStream_t s) {
  typedef WithRows<O, Plain> T;
  const hipError_t e = lds_limit<T>(&k_int8<O, T>);
  if (e != hipSuccess) return e;
  const int64_t tiles = (int64_t)g.tx * g.ty, most = (int64_t)cus * (160 * 1024 / T::LDS);
  tt_launch(K_INT8, k_int8<O, T>, dim3((unsigned)std::min(tiles, most)), dim3(T::NT), T::LDS, s, g, ep);
  return hipGetLastError();
}

struct Int8Args {
  int64_t n, v, d, wpitch, pitch, qpitch;  // bytes; pitch: d in whole groups of 16
  const int8_t *w, *q;
  const float *s, *t;
  void *out;
};

template <class O>
static hipError_t product(const Int8Args &a, hipStream_t s) {
  const int cus = std::max(device_cus(), 1);
  int64_t large = 0;
  if (a.n > 128 && a.v > 128)
    large = std::min(a.v, large_tiles((a.v + 255) / 256, (a.n + 255) / 256, cus) * 256);
  hipError_t e = hipSuccess;
  auto part = [&](int64_t r0, int64_t rows, GemmShape t) {  // rows of the table
    if (rows <= 0 || e != hipSuccess) return;
    GemmArgs g = {};
    g.P.p = (const char *)a.w + r0 * a.wpitch; g.P.ld = a.wpitch; g.P.rows = rows; g.P.cols = a.pitch / 2;
    g.Q.p = (const char *)a.q; g.Q.ld = a.qpitch; g.Q.rows = a.n; g.Q.cols = a.pitch / 2;
    g.K = a.pitch / 2;
    g.xn = (int)rows; g.yn = (int)a.n;
    g.tx = (int)((rows + t.bx - 1) / t.bx); g.ty = (int)((a.n + t.by - 1) / t.by);
    g.splits = 1;
    Int8Out<O> ep = {(O *)a.out + r0, a.s, a.t + r0, a.v, (int)a.n, (int)rows};
    if (t.cfg == 0) e = go_int8<O, TileL>(g, ep, cus, s);
    else if (t.cfg == 1) e = go_int8<O, TileM>(g, ep, cus, s);
    else if (t.cfg == 3) e = go_int8<O, TileN>(g, ep, cus, s);
    else if (t.cfg == 4) e = go_int8<O, TileT>(g, ep, cus, s);
    else if (t.cfg == 5) e = go_int8<O, TileM1>(g, ep, cus, s);
    else e = go_int8<O, TileS>(g, ep, cus, s);
  };
  part(0, large, {0, 256, 256});
  part(large, a.v - large, gemm_shape(a.v - large, a.n, cus));
  return e;
}

template <class S, class O>
static void go_few(const FewArgs &a, int cus, hipStream_t s) {
  const int64_t blocks = ((a.v + 15) / 16 + 3) / 4;
  auto go = [&](auto *kernel) {
    tt_launch(K_INT8, kernel, dim3((unsigned)std::min<int64_t>(blocks, 8 * cus)), dim3(256), a.n * a.lp, s, a);
  };
  if (a.d < 8) go(k_int8_few<S, O, true>);
  else go(k_int8_few<S, O, false>);
}
template <class S>
static void go_few(const FewArgs &a, int out, int cus, hipStream_t s) {
  if (out == TT_DTYPE_F32) go_few<S, float>(a, cus, s);
  else if (out == TT_DTYPE_BF16) go_few<S, __bf16>(a, cus, s);
  else go_few<S, _Float16>(a, cus, s);
}

static int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
static int64_t elem_size(int dtype) {
  return dtype == TT_DTYPE_F32 ? 4 : dtype == TT_DTYPE_I8 ? 1 : 2;
}
constexpr int64_t MAX_INT8_D = 1 << 17;  // 127 128 2^17 < 2^31: a token that is quantised has no -128

static int int8_args(const tt_int8_desc *d, Int8Args &a) {
  if (!d) return TT_EINVAL;
  if (d->n < 0 || d->v < 1 || d->d < 1) return TT_EINVAL;
  if (d->dtype < TT_DTYPE_F32 || d->dtype > TT_DTYPE_I8) return TT_EINVAL;
  if (d->out_dtype < TT_DTYPE_F32 || d->out_dtype > TT_DTYPE_F16) return TT_EINVAL;
  a = {};
  a.n = d->n; a.v = d->v; a.d = d->d; a.wpitch = d->weight_pitch;
  a.pitch = round_up(a.d, 16);
  if (d->hidden_stride < d->d || a.wpitch < a.pitch || a.wpitch % 16) return TT_EINVAL;
  if (d->dtype == TT_DTYPE_I8 && (d->hidden_stride < a.pitch || d->hidden_stride % 16)) return TT_EINVAL;
  if (a.n > (1 << 23) || a.v > (1 << 30) || a.d > MAX_INT8_D || a.n * a.v > (1ll << 40)) return TT_ESHAPE;
  // one that is given may have, as its row: 128^2 2^17 = 2^31
  if (d->dtype == TT_DTYPE_I8 && a.d == MAX_INT8_D) return TT_ESHAPE;
  // a tile's rows inside one buffer descriptor
  if (a.wpitch > (1 << 22) || (d->dtype == TT_DTYPE_I8 && d->hidden_stride > (1 << 22)) ||
      d->hidden_stride > (1ll << 32))
    return TT_ESHAPE;
  return TT_OK;
}
// Tokens that are quantised in the product's own launch.  us of this launch and of the two with the tiles, tables
// that are not in a cache, without the host: 1 x 8000 x 1024 7.7 and 10.9, 1 or 4 x 32000 x 1024 11.2 and 14.4, 4 x 48000 x
// 1024 13.7 and 18.9, 1 x 16000 x 2048 12.3 and 14.0.  More tokens are quantised too often: 8 x 32000 x 1024 14.6 and 14.6, 16
// of them 19.2 and 15.0, 8 x 16000 x 2048 16.5 and 14.9 (in between, 4 x 16000 x 2048, 12.8 and 14.7).  Larger tables go either
// way up to some 100 MB (4 x 64000 x 1024 22.0 and 21.5, 1 x 32000 x 2048 17.4 and 19.1, 1 x 50000 x 2048 32.4 and 30.5) and
// are read faster by the tiles beyond (1 x 131072 x 4096 131 and 111).
static bool few(const tt_int8_desc *d, const Int8Args &a) {
  return d->dtype != TT_DTYPE_I8 && a.n <= FEW_TOKENS && a.n * a.d <= FEW_VALUES && a.v * a.wpitch <= FEW_BYTES;
}
static int64_t int8_ws(const tt_int8_desc *d, const Int8Args &a) {
  if (few(d, a) || (d->dtype == TT_DTYPE_I8 && a.d % 16 == 0)) return 256;  // none
  return round_up(std::max<int64_t>(a.n, 1) * a.pitch, 256) + round_up(std::max<int64_t>(a.n, 1) * 4, 256);
}

}  // namespace ttb

using namespace ttb;

extern "C" {

int tt_int8_quantize(int64_t n, int64_t d, int32_t dtype, const void *x, int64_t stride,
                     int8_t *values, int64_t pitch, float *scales, void *stream) {
  if (n < 0 || d < 1 || dtype < TT_DTYPE_F32 || dtype > TT_DTYPE_F16) return TT_EINVAL;
  if (stride < d || pitch < round_up(d, 16) || pitch % 16) return TT_EINVAL;
  if (n > (1 << 30) || d > (1 << 20) || stride > (1ll << 32) || pitch > (1ll << 32)) return TT_ESHAPE;
  if (n && (!x || !values || !scales)) return TT_EINVAL;
  if ((uintptr_t)x % elem_size(dtype) || (uintptr_t)values % 16 || (uintptr_t)scales % 4) return TT_EINVAL;
  QuantArgs a = {n, d, stride, pitch, x, values, scales};
  return quantize(a, dtype, (hipStream_t)stream) == hipSuccess ? TT_OK : TT_EHIP;
}

size_t tt_int8_workspace_size(const tt_int8_desc *desc) {
  Int8Args a;
  return int8_args(desc, a) == TT_OK ? (size_t)int8_ws(desc, a) : 0;
}

int tt_int8_linear(const tt_int8_desc *desc, const void *hidden, const float *hidden_scales,
                   const int8_t *weight, const float *weight_scales, void *out, void *ws,
                   size_t ws_bytes, void *stream) {
  Int8Args a;
  const int rc = int8_args(desc, a);
  if (rc != TT_OK) return rc;
  const bool given = desc->dtype == TT_DTYPE_I8;
  if (!weight || !weight_scales || (a.n && (!hidden || !out))) return TT_EINVAL;
  if (given != (hidden_scales != nullptr) || (!ws && int8_ws(desc, a) > 256)) return TT_EINVAL;
  if ((uintptr_t)weight % 16 || (uintptr_t)weight_scales % 4 || (uintptr_t)hidden_scales % 4 ||
      (uintptr_t)hidden % (given ? 16 : elem_size(desc->dtype)) ||
      (uintptr_t)out % elem_size(desc->out_dtype))
    return TT_EINVAL;
  if ((uintptr_t)ws % 256) return TT_EWORKSPACE;
  if ((size_t)int8_ws(desc, a) > ws_bytes) return TT_EWORKSPACE;
  if (a.n == 0) return TT_OK;
  hipStream_t s = (hipStream_t)stream;
  a.w = weight; a.t = weight_scales; a.out = out;
  if (few(desc, a)) {
    // LDS rows of whole loads, and 16 bytes off each other's banks
    const FewArgs f = {a.d, desc->hidden_stride, a.pitch, a.wpitch, a.v, (int)a.n,
                       (int)(round_up(a.d, 512) + 16), hidden, weight, weight_scales, out};
    const int cus = std::max(device_cus(), 1);
    if (desc->dtype == TT_DTYPE_F32) go_few<float>(f, desc->out_dtype, cus, s);
    else if (desc->dtype == TT_DTYPE_BF16) go_few<__bf16>(f, desc->out_dtype, cus, s);
    else go_few<_Float16>(f, desc->out_dtype, cus, s);
    return hipGetLastError() == hipSuccess ? TT_OK : TT_EHIP;
  }
  QuantArgs q = {a.n, a.d, desc->hidden_stride, a.pitch, hidden, (int8_t *)ws,
                 (float *)((char *)ws + round_up(a.n * a.pitch, 256))};
  a.q = q.q; a.qpitch = a.pitch; a.s = given ? hidden_scales : q.s;
  if (given && a.d % 16 == 0) {
    a.q = (const int8_t *)hidden;
    a.qpitch = a.n > 1 ? desc->hidden_stride : a.pitch;
  } else if (given) {
    tt_launch(K_INT8_QUANT, k_pad_rows, dim3((unsigned)std::min<int64_t>((a.n * a.pitch + 255) / 256, 4096)),
              dim3(256), 0, s, q);
    if (hipGetLastError() != hipSuccess) return TT_EHIP;
  } else if (quantize(q, desc->dtype, s) != hipSuccess) {
    return TT_EHIP;
  }
  hipError_t e;
  if (desc->out_dtype == TT_DTYPE_F32) e = product<float>(a, s);
  else if (desc->out_dtype == TT_DTYPE_BF16) e = product<__bf16>(a, s);
  else e = product<_Float16>(a, s);
  return e == hipSuccess ? TT_OK : TT_EHIP;
}

}  // extern "C"
