// tt_gemm.h -- the 16-bit matrix-core product that the vocabulary-head losses are built of (and, on
// bytes in pairs, the 8-bit one of int8 tables).
//
// out[y][x] = sum_k P(x, k) Q(y, k): P's index x runs along the contiguous axis of the
// result, Q's index y along its rows.  v_mfma_f32_16x16x32 (fp16 or bf16 in, fp32 sums) takes
// 8 consecutive k per lane of each operand and leaves a lane with four consecutive x of one
// y: lane = 16 g + c holds out[16 ni + c][16 mi + 4 g + r], r = 0..3.
//
// Each operand is either "row" (its rows run along k, so a lane's 8 values are 16 bytes of a
// row) or "col" (its rows run along x or y; the transposing LDS read ds_read_b64_tr_b16
// hands a lane four k of one column).  That way the three products of a linear loss --
// logits W h^T, dh = G W, dW = G^T h -- read W, h and G as they lie, with no transposed copy.
//
// Tiles of 64 k go from memory to LDS by bounds-checked buffer loads that bypass registers
// (rows past the end arrive as zeros), S tiles deep, with one barrier per tile.  These loads
// fill LDS in lane order, 16 bytes a lane, so the swizzle that keeps the reads free of bank
// conflicts is put on the memory side: a lane fetches the chunk that its LDS place stands for.
//
// fp32 operands come as two fp16 planes (x s = hi + lo, s a power of two that puts the
// tensor's largest value below 2^15: 22 bits of every value within 2^17 of the largest, an
// absolute 2^-39 of the largest below that), side by side in a row.  Their tiles hold 32 k of
// both planes, and hi hi, hi lo and lo hi go into the same sums: three products for the LDS
// traffic of two.
//
// What two parts cannot stand for goes through the same tiles WHOLE: the planes hold the upper
// and the lower halves of the values' bits, which are put together again in registers, and
// v_mfma_f32_16x16x4 multiplies them, fp32 as it is.  An infinity is such a value: it would
// meet the other operand's lo part as inf x 0 or inf - inf.  So are the rest of a tensor that a
// few values top by far.  (A step of 1024 x 32000 x 1024:
// 2.4 ms, of two parts 0.84 ms.)
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tt_mfma.h"

namespace ttb {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef _Float16 hf4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// the thread's index, as a value that the compiler takes to be new at each place: what is
// derived from it for one stage of a kernel does not occupy registers in the others
__device__ __forceinline__ int own_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

struct Bf16 {
  typedef __bf16 e;
  typedef bf8 v8;
  typedef bf4 v4;
  typedef f4 acc4;
  static __device__ __forceinline__ f4 mfma(v8 a, v8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
struct Fp16 {
  typedef _Float16 e;
  typedef hf8 v8;
  typedef hf4 v4;
  typedef f4 acc4;
  static __device__ __forceinline__ f4 mfma(v8 a, v8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// v_mfma_i32_16x16x64_i8: sixteen 8-bit integers a lane where the others have eight 16-bit values, so
// an operand of 2 c columns of 8 bits is one of c columns here, and lies in tiles and registers the
// same way (both operands name the same k of a lane's 16 bytes, whatever its order).
struct Int8 {
  typedef i32x4 v8;
  typedef i32x4 acc4;
  static __device__ __forceinline__ i32x4 mfma(v8 a, v8 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// fp32 rows as they lie, four values a lane where the others have eight of 16 bits (columns of k count
// 16 bits here too): element e of a lane's four is one product over the four lane groups' k.
struct Fp32 {
  typedef f4 v8;
  typedef f4 acc4;
  static __device__ __forceinline__ f4 mfma(v8 a, v8 b, f4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

// element e of eight fp32 values whose upper and lower halves lie in two fragments
template <class V8>
__device__ __forceinline__ float whole(V8 hi, V8 lo, int e) {
  union {
    V8 v;
    unsigned u[4];
  } a, b;
  a.v = hi;
  b.v = lo;
  return __uint_as_float(
      __builtin_amdgcn_perm(a.u[e / 2], b.u[e / 2], e % 2 ? 0x07060302u : 0x05040100u));
}
// the halves of four fp32 values, as 16-bit patterns
template <class V4>
__device__ __forceinline__ void halves(const float (&v)[4], V4 &hi, V4 &lo) {
  union {
    V4 v;
    unsigned short u[4];
  } a, b;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    a.u[r] = (unsigned short)(__float_as_uint(v[r]) >> 16);
    b.u[r] = (unsigned short)__float_as_uint(v[r]);
  }
  hi = a.v;
  lo = b.v;
}

constexpr int GK = 64;                        // k per tile (over all planes)
constexpr unsigned BUF_MAX = 0x7fffffffu;     // largest extent of one buffer descriptor
constexpr unsigned BUF_OUT = 0x80000000u;     // an offset past every extent: reads as zeros

// One operand in memory: `rows` rows of `cols` elements, ld bytes apart; with two planes, the
// second one's row lies `plane` bytes behind the first one's.  "row" operands have rows = x or
// y, cols = k; "col" ones the reverse.
struct Operand {
  const char *p;
  int64_t ld, plane;
  int64_t rows, cols;
};

struct GemmArgs {
  Operand P, Q;
  int64_t K;            // k in all
  int xn, yn;           // x and y in all
  const int *kcount;    // device word that bounds K (rounded up to 64), or null
  const int *ycount;    // device word that bounds yn, or null
  int tx, ty, splits;   // tiles along x and y, pieces of k
};

// ---------------------------------------------------------------- memory -> LDS
__device__ __forceinline__ i32x4 buf_desc(uint64_t base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : (bytes > (int64_t)BUF_MAX ? (int64_t)BUF_MAX : bytes);
  i32x4 r;
  r.x = __builtin_amdgcn_readfirstlane((int)(unsigned)base);
  r.y = __builtin_amdgcn_readfirstlane((int)((unsigned)(base >> 32) & 0xffffu));
  r.z = __builtin_amdgcn_readfirstlane((int)n);
  r.w = 0x00020000;  // raw buffer, dword format
  return r;
}

// 64 lanes x 16 bytes from desc[voff] to LDS bytes [lds, lds + 1024) in lane order.  The load
// has no register result; its end is counted by vmcnt.
__device__ __forceinline__ void load_lds(i32x4 desc, unsigned voff, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(voff), "s"(desc)
               : "memory");
}

// every wave's LDS reads are done and all but the last N loads have arrived, in all waves
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// swizzle of "col" tiles: the 16-byte chunks of row k are permuted by XOR with this.  A
// transposing read touches 32 bytes of each of the rows k0 + {0..3, 8..11} in one pass, which
// this spreads over the 64 banks (rows of 128 bytes alternate bank halves by themselves).
template <int ROWS>
__device__ __forceinline__ int col_swz(int k) {
  return ROWS >= 128 ? 2 * ((k & 3) + 4 * ((k >> 3) & 1))
                     : 2 * (((k >> 1) & 1) + 2 * ((k >> 3) & 1));
}

// The tile of ROWS x (or y) by 64 / PL k of one operand: where its lanes read and where it is
// next.  Two planes: "row" tiles hold k of the first plane in the front half of a row and of
// the second in the rear half, "col" tiles have the second plane's rows below the first's.
template <int ROWS, bool COL, int PL, int NT>
struct Feed {
  static constexpr int KT = GK / PL;
  static constexpr int L = ROWS * 8 / NT;  // loads per thread and tile
  unsigned voff[L];
  uint64_t base;
  int64_t rem, step;        // bytes from base to the operand's end; bytes per tile of k
  int64_t kleft;            // "row": elements of k left
  int chunk;                // "row": this lane's first element of k inside the tile

  __device__ __forceinline__ void init(const Operand &o, int64_t x0, int64_t k0, int tid) {
    const int64_t r = COL ? k0 : x0, c = COL ? x0 : k0;
    base = (uint64_t)o.p + r * o.ld + c * 2;
    rem = (o.rows - 1 - r) * o.ld + (PL > 1 ? o.plane : 0) + (o.cols - c) * 2;
    step = COL ? KT * o.ld : KT * 2;
    kleft = o.cols - k0;
    if constexpr (COL) {
      constexpr int CPR = ROWS / 8;
      const int k = tid / CPR, pc = tid % CPR;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int kk = k + j * (NT / CPR);
        voff[j] = (unsigned)((kk % KT) * o.ld + (kk / KT) * o.plane +
                             (pc ^ col_swz<ROWS>(kk)) * 16);
      }
      chunk = 0;
    } else {
      const int row = tid / 8, c8 = (tid % 8) ^ (row & 7);
#pragma unroll
      for (int j = 0; j < L; ++j)
        voff[j] = (unsigned)((row + j * (NT / 8)) * o.ld + (c8 * 8 / KT) * o.plane +
                             (c8 * 8 % KT) * 2);
      chunk = c8 * 8 % KT;
    }
  }
  __device__ __forceinline__ void issue(unsigned lds, bool live) {
    const i32x4 d = buf_desc(base, live ? rem : 0);
    const bool whole = COL || kleft >= KT;
    if (whole) {
#pragma unroll
      for (int j = 0; j < L; ++j) load_lds(d, voff[j], lds + j * (NT * 16));
    } else {  // the last, partial tile of a row: chunks past the row's end read as zeros
      const bool in = chunk < kleft;
#pragma unroll
      for (int j = 0; j < L; ++j) load_lds(d, in ? voff[j] : BUF_OUT, lds + j * (NT * 16));
    }
    base += step;
    rem -= step;
    kleft -= KT;
  }

  // What the loads get wrong in the last tile of k where the rows of o are of any alignment,
  // put right in LDS (all threads; the tile has arrived, its readers wait for a barrier):
  //  - "row": the group of eight across the end of k holds the next row's first elements,
  //    which have to be zeros (the other operand is zero there, but 0 x inf is not);
  //  - the bounds check goes by dwords from the load's start, so the very last element of an
  //    operand of odd length is dropped.
  static __device__ __forceinline__ void mend(const Operand &o, char *t, int64_t x0, int64_t k0) {
    const int tid = own_thread();
    if constexpr (!COL) {
      const int in = (int)(o.cols - k0);  // elements of k in this tile
      for (int r = tid; r < ROWS; r += NT) {
        union {
          i32x4 v;
          unsigned short e[8];
        } u;
        i32x4 *at = (i32x4 *)(t + r * 128 + (((in >> 3) ^ (r & 7)) << 4));
        u.v = *at;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= (in & 7)) u.e[e] = 0;
        if ((in & 1) && x0 + r == o.rows - 1) {
          const unsigned short last =
              *(const unsigned short *)(o.p + (o.rows - 1) * o.ld + (o.cols - 1) * 2);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e == (in & 7) - 1) u.e[e] = last;
        }
        *at = u.v;
      }
    } else if (tid == 0 && (o.cols & 1)) {
      const int64_t k = o.rows - 1 - k0, x = o.cols - 1 - x0;
      if (k >= 0 && k < GK && x >= 0 && x < ROWS)
        *(unsigned short *)(t + k * ROWS * 2 + (((int)(x >> 3)) ^ col_swz<ROWS>((int)k)) * 16 +
                            (x & 7) * 2) =
            *(const unsigned short *)(o.p + (o.rows - 1) * o.ld + (o.cols - 1) * 2);
    }
  }
};

// ---------------------------------------------------------------- LDS -> registers
// Fragments of 16 x (or y) at x0 of the tile at `t`: k = 32 kk + 8 g .. + 8, with two planes
// k = 8 g .. + 8 of plane kk
template <class E, int ROWS, bool COL>
__device__ __forceinline__ typename E::v8 frag(const char *t, int x0, int kk, int lane) {
  const int g = lane >> 4, c = lane & 15;
  if constexpr (!COL) {
    return *(const typename E::v8 *)(t + (x0 + c) * 128 + ((((kk << 2) + g) ^ (lane & 7)) << 4));
  } else {
    constexpr int RB = ROWS * 2;
    const int q = c >> 2, s = col_swz<ROWS>(8 * g + q);
    const char *a = t + (8 * g + q) * RB + (((x0 >> 3) + ((c & 3) >> 1)) ^ s) * 16 + (c & 1) * 8 +
                    kk * 32 * RB;
    typedef __attribute__((address_space(3))) s16x4 lds_v;
    union {
      s16x4 h[2];
      typename E::v8 v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)a);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)(a + 4 * RB));
    return u.v;
  }
}

// One tile of the result: (x tile, y tile, split) and its tiles of k.
struct TileAt {
  int ix, iy, is, nk;
  int64_t k0;
};

// The walk of a workgroup over the tiles.  Ids go round the XCDs (workgroup b runs on XCD
// b mod 8), so the ids of one XCD are made consecutive; within them 8 x-tiles by all y-tiles
// are walked together, so the 32 CUs of an XCD share the rows of few tiles of both operands
// in its L2.
struct TileWalk {
  int tx, ty, splits, total, KT, yn;
  int64_t K, kper;

  template <int BY>
  __device__ __forceinline__ void init(const GemmArgs &a, int kt) {
    KT = kt;
    tx = a.tx;
    yn = a.ycount ? min(a.yn, *a.ycount) : a.yn;
    ty = min(a.ty, (yn + BY - 1) / BY);
    splits = a.splits;
    K = a.kcount ? (int64_t)((*a.kcount + GK - 1) / GK) * GK : a.K;
    kper = ((K + splits - 1) / splits + GK - 1) / GK * GK;
    total = tx * ty * splits;
  }
  __device__ __forceinline__ bool at(int id, TileAt &t) const {
    if (id >= total) return false;
    const int q = total / 8, r = total % 8, xcd = id % 8;
    id = xcd * q + min(xcd, r) + id / 8;
    const int per = tx * ty;
    t.is = id / per;
    id -= t.is * per;
    const int grp = id / (8 * ty), x0 = grp * 8, w = min(8, tx - x0), in = id - grp * 8 * ty;
    t.ix = x0 + in % w;
    t.iy = in / w;
    t.k0 = t.is * kper;
    const int64_t n = min(kper, K - t.k0);
    t.nk = n > 0 ? (int)((n + KT - 1) / KT) : 0;
    return true;
  }
};

template <int BX, int BY, int WX, int WY, int S>
struct Tile {
  static constexpr int X = BX, Y = BY, NWX = BX / WX, NWY = BY / WY;
  static constexpr int NT = NWX * NWY * 64, MI = WX / 16, NI = WY / 16, STAGES = S;
  static constexpr int EXTRA = NWX * BY * 12;  // scratch for the results
  static constexpr int LDS = (BX + BY) * GK * 2 * S + EXTRA;
  static constexpr int wx = WX, wy = WY;
};

// All tiles of this workgroup (id blockIdx.x, + gridDim.x, ...): the sums of each are handed
// to done(tile, sums, scratch), scratch being T::EXTRA bytes of LDS beside the tiles'.  The
// loads run on from one tile into the next, so the next tile's first data travel while this
// one's results are worked off; done() may use its scratch freely between two of its own
// barriers.
// MEND: P's rows do not end with whole 16-byte groups (see Feed::mend); a variant of its own,
// because the test for it in the loop cost the others 1 to 7 %.
// WHOLE: the two planes are the halves of fp32 values.
template <class E, class T, int PL, bool PC, bool QC, bool MEND, bool WHOLE, class Done>
__device__ __forceinline__ void gemm_tiles(const GemmArgs &a, char *lds, Done done) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int px = (wv % T::NWX) * T::wx, qy = (wv / T::NWX) * T::wy;
  TileWalk walk;
  walk.init<T::Y>(a, GK / PL);
  TileAt now, ahead;
  int id = blockIdx.x, ida = id;
  if (!walk.at(id, now)) return;

  Feed<T::X, PC, PL, T::NT> fp;
  Feed<T::Y, QC, PL, T::NT> fq;
  constexpr int PB = T::X * GK * 2, QB = T::Y * GK * 2, SB = PB + QB;
  const unsigned lbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds +
                         wv * 1024;
  int ik = 0;  // the next tile of k to load, of tile `ahead`
  bool live = true;
  auto aim = [&]() {  // at the first tile from ida on that has any k
    while ((live = walk.at(ida, ahead)) && ahead.nk == 0) ida += gridDim.x;
    if (live) {
      const int tid = own_thread();
      fp.init(a.P, (int64_t)ahead.ix * T::X, ahead.k0, tid);
      fq.init(a.Q, (int64_t)ahead.iy * T::Y, ahead.k0, tid);
    }
  };
  auto load = [&](int buf) {
    const unsigned l = __builtin_amdgcn_readfirstlane(lbase + buf * SB);
    fp.issue(l, live);  // past the last tile: zeros
    fq.issue(l + PB, live);
    if (live && ++ik >= ahead.nk) {
      ik = 0;
      ida += gridDim.x;
      aim();
    }
  };
  aim();
  constexpr int LPT = Feed<T::X, PC, PL, T::NT>::L + Feed<T::Y, QC, PL, T::NT>::L;
  typename E::acc4 acc[T::MI][T::NI];
  // fp32 as it lies: 128 k are summed by themselves and then added, because every 4 k of one chain are
  // rounded at the size of the whole sum (6 positions x 5392 x 1216, logits up to 14: log-probabilities of
  // relative error 3.7e-7 in one chain, 0.9e-7 by 32 k, 0.8e-7 by 128; 64 x 32000 x 1024: 52.0, 56.7, 53.7 us)
  constexpr bool APART = std::is_same<E, Fp32>::value;
  typename E::acc4 some[APART ? T::MI : 1][APART ? T::NI : 1];
  typename E::v8 p[2][T::MI], q[2][T::NI];
  auto read_p = [&](int set, int buf) {
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
      p[set][i] = frag<E, T::X, PC>(lds + buf * SB, px + 16 * i, set, lane);
  };
  auto read_q = [&](int set, int buf) {
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
      q[set][j] = frag<E, T::Y, QC>(lds + buf * SB + PB, qy + 16 * j, set, lane);
  };
  auto mul = [&](int sp, int sq) {
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        typename E::acc4 &c = *(APART ? &some[APART ? i : 0][APART ? j : 0] : &acc[i][j]);
        c = E::mfma(p[sp][i], q[sq][j], c);
      }
  };
  auto gather = [&]() {
#pragma unroll
    for (int i = 0; APART && i < T::MI; ++i)
#pragma unroll
      for (int j = 0; APART && j < T::NI; ++j) {
        acc[i][j] += some[i][j];
        some[i][j] = typename E::acc4{};
      }
  };
  // fp32: lane group g holds k = 8 g + e of both operands, so element e of all four is one
  // product over four k.  The reads wait for their use here: both register sets beside the
  // accumulators and the joined values do not fit.
  auto mul_whole = [&](int buf) {
    if constexpr (!WHOLE) return;
    else {
    read_q(0, buf);
    read_q(1, buf);
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
      const typename E::v8 hi = frag<E, T::X, PC>(lds + buf * SB, px + 16 * i, 0, lane),
                           lo = frag<E, T::X, PC>(lds + buf * SB, px + 16 * i, 1, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < T::NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              whole(hi, lo, e), whole(q[0][j], q[1][j], e), acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    }
  };
  // one LDS read to every few products, so that neither unit waits for the other's burst
  auto pace = [&]() {
#pragma unroll
    for (int u = 0; u < T::MI + T::NI; ++u) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, T::MI * T::NI / (T::MI + T::NI), 0);
    }
  };
  // The two halves of a tile (32 k each, or the two planes of 32 k) take turns in two register
  // sets: while one is multiplied the other is read.  The barrier sits between them: there every wave has read
  // all of this tile, whose buffer the next load may take, and the next tile is complete, so
  // its first half is read under the second half's products.  (Reads right behind the
  // barrier, with one register set, ran at 1.25 PFLOP/s on 16384 x 8192 x 4096; this runs at
  // 1.35 in all three layouts.)
#pragma unroll
  for (int s = 0; s < T::STAGES; ++s) load(s);
  int buf = 0;
  for (;;) {
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        acc[i][j] = typename E::acc4{};
        if (APART) some[i][j] = typename E::acc4{};
      }
    const int steps = now.nk;
    auto mend = [&](int b) {
      const int64_t k0 = now.k0 + (int64_t)(now.nk - 1) * (GK / PL);
      Feed<T::X, PC, PL, T::NT>::mend(a.P, lds + b * SB, (int64_t)now.ix * T::X, k0);
      if constexpr (std::is_same<E, Fp32>::value)  // Q lies as it came, too: 0 x inf is not 0
        Feed<T::Y, QC, PL, T::NT>::mend(a.Q, lds + b * SB + PB, (int64_t)now.iy * T::Y, k0);
      lds_barrier();
    };
    // a wave whose part of a ragged tile lies outside has its loads and barriers only (1800
    // positions: the eighth row of tiles, with 8 of 256, costs half)
    if (now.ix * T::X + px >= a.xn || now.iy * T::Y + qy >= walk.yn) {
      if (steps > 0) {
        wait_barrier<(T::STAGES - 1) * LPT>();
        if (MEND && steps == 1) mend(buf);
      }
      for (int st = 0; st < steps; ++st) {
        const int next = buf + 1 == T::STAGES ? 0 : buf + 1;
        wait_barrier<(T::STAGES - 2) * LPT>();
        if (MEND && st + 2 == steps) mend(next);
        load(buf);
        buf = next;
      }
    } else {
      if (steps > 0) {
        wait_barrier<(T::STAGES - 1) * LPT>();
        if (MEND && steps == 1) mend(buf);
        if constexpr (!WHOLE) {
          read_q(0, buf);
          read_p(0, buf);
        }
      }
      for (int st = 0; st < steps; ++st) {
        const int next = buf + 1 == T::STAGES ? 0 : buf + 1;
        if constexpr (WHOLE) {
          mul_whole(buf);
        } else {
          read_q(1, buf);
          read_p(1, buf);
          if (APART && st > 0 && st % 4 == 0) gather();
          mul(0, 0);
          pace();
        }
        wait_barrier<(T::STAGES - 2) * LPT>();
        if (MEND && st + 2 == steps) mend(next);
        load(buf);
        if constexpr (PL == 1) {
          read_q(0, next);
          read_p(0, next);
          mul(1, 1);
          pace();
        } else if constexpr (!WHOLE) {  // hi lo and lo hi; each operand's next front half follows its last use
          mul(0, 1);
          read_p(0, next);
          mul(1, 0);
          read_q(0, next);
        }
        buf = next;
      }
    }
    gather();
    done(now, acc, lds + T::STAGES * SB);
    id += gridDim.x;
    if (!walk.at(id, now)) break;
  }
  // the zeros of loads past the last tile must not land in another workgroup's LDS
  wait_barrier<0>();
}

// 4 + 4 sixteen-bit values of a lane, from two result tiles 16 x apart, to 8 consecutive ones
// per lane: swapping the odd 16-lane rows of one register with the even ones of the other
// leaves lane groups 0..3 with x = 0, 16, 8, 24 and on.  o: x = 0 of the pair.
// o may lie on any boundary of two bytes.
template <class V4>
__device__ __forceinline__ void store_pair_if(bool in, char *o, V4 a, V4 b, int g) {
  union {
    V4 v[2];
    unsigned u[4];
  } s;
  s.v[0] = a;
  s.v[1] = b;
  const auto lo = __builtin_amdgcn_permlane16_swap(s.u[0], s.u[2], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(s.u[1], s.u[3], false, false);
  struct __attribute__((packed, aligned(2))) any { i32x4 v; };
  any v = {{(int)lo[0], (int)hi[0], (int)lo[1], (int)hi[1]}};
  if (in) *(any *)(o + ((g & 1) * 16 + (g >> 1) * 8) * 2) = v;
}
template <class V4>
__device__ __forceinline__ void store_pair(char *o, V4 a, V4 b, int g) {
  store_pair_if(true, o, a, b, g);
}

}  // namespace ttb
