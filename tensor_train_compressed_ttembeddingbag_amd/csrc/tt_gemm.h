// tt_gemm.h -- the 16-bit matrix-core product that the vocabulary-head losses are built of.
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
// (rows past the end arrive as zeros), S tiles deep, with one barrier per tile: the load of
// tile k + S - 1 goes into the buffer of tile k - 1 once every wave has passed the barrier
// of step k.  These loads fill LDS in lane order, 16 bytes a lane, so the swizzle that keeps
// the reads free of bank conflicts is put on the memory side: a lane fetches the chunk that
// its LDS place stands for.
//
// fp32 operands come as two fp16 planes (x s = hi + lo, s a power of two that puts the
// tensor's largest value below 2^15: 22 bits of every value within 2^17 of the largest, an
// absolute 2^-39 of the largest below that); lo hi + hi lo + hi hi are three runs over k into
// the same sums.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tt_mfma.h"

namespace ttb {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef _Float16 hf4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Bf16 {
  typedef __bf16 e;
  typedef bf8 v8;
  typedef bf4 v4;
  static __device__ __forceinline__ f4 mfma(v8 a, v8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
struct Fp16 {
  typedef _Float16 e;
  typedef hf8 v8;
  typedef hf4 v4;
  static __device__ __forceinline__ f4 mfma(v8 a, v8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

constexpr int GK = 64;                        // k per tile
constexpr unsigned BUF_MAX = 0x7fffffffu;     // largest extent of one buffer descriptor
constexpr unsigned BUF_OUT = 0x80000000u;     // an offset past every extent: reads as zeros

// One operand in memory: `rows` rows of `cols` elements, ld bytes apart, `planes` copies
// plane bytes apart.  "row" operands have rows = x or y, cols = k; "col" ones the reverse.
struct Operand {
  const char *p;
  int64_t ld, plane;
  int64_t rows, cols;
};

struct GemmArgs {
  Operand P, Q;
  int64_t K;            // k in all
  int64_t kper;         // k per split (a multiple of 64)
  const int *kcount;    // device word that bounds K (rounded up to 64), or null
  const int *ycount;    // device word: tiles of y from it on have nothing to do, or null
  int nseg;             // 1, or 3 for two-plane operands
  int tx, ty, splits;   // tiles along x and y, pieces of k
  const int *dsplits;   // device word: the pieces of k (over the tiles of ycount), or null
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

// The 64-k tile of ROWS x (or y) of one operand: where its lanes read and where it is next.
template <int ROWS, bool COL, int NT>
struct Feed {
  static constexpr int L = ROWS * 8 / NT;  // loads per thread and tile
  unsigned voff[L];
  uint64_t base0, base;
  int64_t rem0, rem, step;  // bytes from base to the operand's end; bytes per tile of k
  int64_t kleft0, kleft;    // "row": elements of k left
  int chunk;                // "row": this lane's first element of k inside the tile

  __device__ __forceinline__ void init(const Operand &o, int64_t x0, int64_t k0, int tid) {
    const int64_t r = COL ? k0 : x0, c = COL ? x0 : k0;
    base0 = (uint64_t)o.p + r * o.ld + c * 2;
    rem0 = (o.rows - 1 - r) * o.ld + (o.cols - c) * 2;
    step = COL ? GK * o.ld : GK * 2;
    kleft0 = o.cols - k0;
    if constexpr (COL) {
      constexpr int CPR = ROWS / 8;
      const int k = tid / CPR, pc = tid % CPR;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int kk = k + j * (NT / CPR);
        voff[j] = (unsigned)(kk * o.ld + (pc ^ col_swz<ROWS>(kk)) * 16);
      }
      chunk = 0;
    } else {
      const int row = tid / 8, c8 = (tid % 8) ^ (row & 7);
#pragma unroll
      for (int j = 0; j < L; ++j) voff[j] = (unsigned)((row + j * (NT / 8)) * o.ld + c8 * 16);
      chunk = c8 * 8;
    }
    seek(0);
  }
  __device__ __forceinline__ void seek(int64_t plane) {
    base = base0 + plane;
    rem = rem0;
    kleft = kleft0;
  }
  __device__ __forceinline__ void issue(unsigned lds, bool live) {
    const i32x4 d = buf_desc(base, live ? rem : 0);
    const bool whole = COL || kleft >= GK;
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
    kleft -= GK;
  }
};

// ---------------------------------------------------------------- LDS -> registers
// Fragments of 16 x (or y) at x0 of the tile at `t`, k = 32 kk + 8 g .. + 8
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

// tile index -> (x tile, y tile, split).  Workgroups go to the 8 XCDs in turn, so the ids of
// one XCD are made consecutive; within them 8 x-tiles by all y-tiles are walked together, so
// the 32 CUs of an XCD share the rows of few tiles of both operands in its L2.
// Returns false for a workgroup without a tile.
template <int BY>
__device__ __forceinline__ bool tile_of(GemmArgs &a, int &ix, int &iy, int &is) {
  if (a.dsplits) {
    a.splits = *a.dsplits;
    a.ty = (*a.ycount + BY - 1) / BY;
    a.kper = ((a.K + a.splits - 1) / a.splits + GK - 1) / GK * GK;
  }
  const int total = a.tx * a.ty * a.splits;
  int id = blockIdx.x;
  if (id >= total) return false;
  const int q = total / 8, r = total % 8, xcd = id % 8, loc = id / 8;
  id = xcd * q + min(xcd, r) + loc;
  const int per = a.tx * a.ty;
  is = id / per;
  id -= is * per;
  const int grp = id / (8 * a.ty), x0 = grp * 8, w = min(8, a.tx - x0), in = id - grp * 8 * a.ty;
  ix = x0 + in % w;
  iy = in / w;
  return true;
}

template <int BX, int BY, int WX, int WY, int S>
struct Tile {
  static constexpr int X = BX, Y = BY, NWX = BX / WX, NWY = BY / WY;
  static constexpr int NT = NWX * NWY * 64, MI = WX / 16, NI = WY / 16, STAGES = S;
  static constexpr int LDS = (BX + BY) * GK * 2 * S;
  static constexpr int wx = WX, wy = WY;
};

// The sums of this workgroup's tile; returns false if it has nothing to do.
template <class E, class T, bool PC, bool QC>
__device__ __forceinline__ bool gemm_tile(const GemmArgs &a, char *lds, int ix, int iy, int is,
                                          f4 (&acc)[T::MI][T::NI]) {
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int px = (wv % T::NWX) * T::wx, qy = (wv / T::NWX) * T::wy;
  if (a.ycount && iy * T::Y >= *a.ycount) return false;
  int64_t K = a.K;
  if (a.kcount) K = (int64_t)((*a.kcount + GK - 1) / GK) * GK;
  const int64_t k0 = is * a.kper, k1 = k0 + a.kper < K ? k0 + a.kper : K;
  const int nk = k1 > k0 ? (int)((k1 - k0 + GK - 1) / GK) : 0, steps = nk * a.nseg;
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = zero4();

  Feed<T::X, PC, T::NT> fp;
  Feed<T::Y, QC, T::NT> fq;
  fp.init(a.P, (int64_t)ix * T::X, k0, tid);
  fq.init(a.Q, (int64_t)iy * T::Y, k0, tid);
  constexpr int PB = T::X * GK * 2, QB = T::Y * GK * 2, SB = PB + QB;
  const unsigned lbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds +
                         wv * 1024;
  int ik = 0, seg = 0;  // the next tile to load
  auto load = [&](int buf) {
    if (ik == 0 && a.nseg > 1) {  // lo hi, hi lo, hi hi: the small terms first
      fp.seek(seg == 0 ? a.P.plane : 0);
      fq.seek(seg == 1 ? a.Q.plane : 0);
    }
    const bool live = seg < a.nseg && nk > 0;
    const unsigned l = __builtin_amdgcn_readfirstlane(lbase + buf * SB);
    fp.issue(l, live);
    fq.issue(l + PB, live);
    if (++ik >= nk) {
      ik = 0;
      ++seg;
    }
  };
  constexpr int LPT = Feed<T::X, PC, T::NT>::L + Feed<T::Y, QC, T::NT>::L;
  typename E::v8 p[2][T::MI], q[2][T::NI];
  auto read = [&](int set, int buf, int kk) {
    const char *tp = lds + buf * SB, *tq = tp + PB;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) q[set][j] = frag<E, T::Y, QC>(tq, qy + 16 * j, kk, lane);
#pragma unroll
    for (int i = 0; i < T::MI; ++i) p[set][i] = frag<E, T::X, PC>(tp, px + 16 * i, kk, lane);
  };
  auto mul = [&](int set) {
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
      for (int j = 0; j < T::NI; ++j) acc[i][j] = E::mfma(p[set][i], q[set][j], acc[i][j]);
    // one LDS read to every few products, so that neither unit waits for the other's burst
#pragma unroll
    for (int u = 0; u < T::MI + T::NI; ++u) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, T::MI * T::NI / (T::MI + T::NI), 0);
    }
  };
  // The two halves of a tile (32 k each) take turns in two register sets: while one is
  // multiplied the other is read.  The barrier sits between them: there every wave has read
  // all of this tile, whose buffer the next load may take, and the next tile is complete, so
  // its first half is read under the second half's products.  (Reads right behind the
  // barrier, with one register set, ran at 1.25 PFLOP/s on 16384 x 8192 x 4096; this runs at
  // 1.35 in all three layouts.)
#pragma unroll
  for (int s = 0; s < T::STAGES; ++s) load(s);
  wait_barrier<(T::STAGES - 1) * LPT>();
  read(0, 0, 0);
  int buf = 0;
  for (int st = 0; st < steps; ++st) {
    const int next = buf + 1 == T::STAGES ? 0 : buf + 1;
    read(1, buf, 1);
    mul(0);
    wait_barrier<(T::STAGES - 2) * LPT>();
    load(buf);
    read(0, next, 0);
    mul(1);
    buf = next;
  }
  // loads issued past the end write zeros: none may land in LDS that an epilogue uses
  wait_barrier<0>();
  return true;
}

}  // namespace ttb
