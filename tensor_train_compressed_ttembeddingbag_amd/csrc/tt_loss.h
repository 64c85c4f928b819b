// tt_loss.h -- shared declarations of the vocabulary-head losses (not installed).
//
// Losses of hidden [N, D] against a weight [V, D] whose [N, V] logits are never kept:
//   z_iv = <hidden_i, weight_v> / T,  lse_i = log sum_v exp z_iv
//   cross entropy  loss_i = lse_i - (1 - e) z_i,t - (e / V) sum_v z_iv
//   distillation   loss_i = T^2 (sum_j q_ij log q_ij - sum_j q_ij z_i,idx(ij) + lse_i)
//   dloss_i/d<hidden_i, weight_v> = s g_iv,  g_iv = exp(z_iv - lse_i) - e / V - sum of the
//   position's q on v (the target's q is 1 - e), s = 1 or T.
//
// forward:  k_entries (distillation: q, sorted, repeated rows merged) -> k_pack (positions that
//           count, packed) -> k_logits (running maximum and sum per position and tile of the
//           weight, the targets' logits) -> k_loss (lse, the entries' logits, loss).  A loss alone of up to 64 positions
//           leaves k_pack out.
// backward: per piece of the vocabulary k_logits (G = row factor * g, in 16 bits), k_entries_g
//           (distillation: the entries of G), k_dhidden (split over the vocabulary, fp32),
//           k_light_rows (a gradient per position), k_dweight; k_dhidden_out adds the splits.
//
// The logits are worked out twice (8 N V D operations where 6 would do): keeping them, or the
// 16-bit G of all pieces, is the [N, V] array that these losses are there to avoid.  (Where G is
// one piece, it exists for the length of the backward.)
#pragma once
#include "tt_gemm.h"
#include "tt_internal.h"

namespace ttb {

constexpr int PACK_ROWS = 4;    // positions per block of k_pack
constexpr int AMAX_BLOCKS = 1024;
constexpr int FACTOR_BLOCKS = 256;  // of k_row_max
constexpr int CHUNK = 1024;     // positions that k_count counts together
constexpr int RANGE_BITS = 14;  // see TensorRange

// scalars that the device works out in the forward
struct LossScalars {
  int count;       // positions that count
  int whole;       // fp32: the planes are the halves of the values' bits, see tt_gemm.h
  int ew, eh;      // exponents of the planes' scales, weight and hidden states (else 0)
  int ge;          // exponent of the scale of G, see g_exp
  float zs;        // logits from sums of products: log2(e) / T over the planes' scales
  int ticket;      // blocks of k_loss that are done
};

// saved by the forward for the backward (one buffer, see saved_layout)
struct LossSaved {
  LossScalars *sc;
  int *slot;       // [N] position -> packed row, or -1 - (a packed row of zeros)
  char *hp;        // packed positions: [row][plane][Dp]
  int *tgt;        // [N] packed row -> target row of the weight (cross entropy)
  float *mx, *lg;  // [N] packed row -> its largest sum of products, and log2 of the sum of
                   // 2^((sum of products - mx) zs): lse in base 2 is mx zs + lg.  In two parts,
                   // because exp(z - lse) and a small loss lose what their rounded sum loses
  float *zt;       // [N] packed row -> the target's sum of products (cross entropy)
  int *eidx;       // [N][k] distillation entries by row of the weight, the empty ones (-1) last
  float *eq, *ez;  // their q (of a repeated row at its first entry, 0 behind) and their log2 p
  float *ent;      // [N] sum_j q log q
};

struct LossArgs {
  // problem
  int64_t N, V, D, hld, wld;  // ld in elements
  int dtype, tdtype, reduction, k;
  int64_t ignore;
  float smoothing, temp;
  const void *hidden, *weight;
  const int64_t *tgt;      // targets [N] or teacher indices [N][k]
  const void *tlogits;     // teacher logits [N][k]
  float *loss;
  const float *up;         // gradient of the loss
  void *dh, *dw;
  int32_t *status;
  // plan
  int64_t Npad, Dp;        // packed rows and their pitch (elements)
  int planes;              // 2 for fp32
  int pack_w;              // the weight is packed too (fp32, odd widths)
  int twin;                // 16-bit, up to 32 positions: G's rows are followed, twin rows on, by
                           // what their rounding left (hp's by themselves); else 0
  int direct;              // loss alone, few positions: the hidden rows as they lie, all of them
  int64_t piece;           // rows of the weight per piece
  int ptiles;              // running statistics per position
  int fold;                // those of a piece are added up into slot 0
  int dh_bx, dh_by, cus;   // k_dhidden's tile, compute units
  LossSaved sv;
  // workspace
  float *amax;             // [3][2 * AMAX_BLOCKS] (fp32) per block of the weight and of the positions:
                           // largest |x| (infinite where a value is not finite), sum of the
                           // exponents of the values that are not 0, how many these are
  char *wp;                // packed piece of the weight: [row][plane][Dp]
  int *chunk;              // [N / CHUNK] positions that count before each chunk, or null, see CHUNKS_AT
  float2 *part;            // [Npad][ptiles] (max, sum) in base 2
  float *zpart;            // [Npad][ptiles] sums of logits (label smoothing)
  float *rowloss;          // [N]
  float *rowf;             // [Npad] factor of a packed row's g (a gradient per row; else null)
  int *rowe;               // [Npad] exponent that a light row's factor leaves out, see LIGHT
  float *upmax;            // [FACTOR_BLOCKS] largest factors, or null, see FACTORS_AT
  float *cm;               // what the factors were divided by
  char *G;                 // [Npad][planes][piece]
  int64_t ldG, Gplane;     // bytes; Gplane: to the second part of a row of G (plane or twin)
  float *dhp;              // [splits][tiles of positions that count][Dp]
};

// A gradient per position in fp16 G: factors down to 2^-LIGHT of the largest go into G, whose
// range has that much to spare.  A smaller one would push its row's G below fp16's steps, and
// with it all of the position's dh: it goes into G times a power of two, which dh's sums take
// back.  dweight adds the positions up, so there G gets its right size first (k_light_rows,
// which reads and writes such rows only: 4096 x 32000 x 2048 fp16, 1840 us with none or with
// factors spread evenly over 0 .. 1, 1871 with half of the rows light, 1907 with all but one).
constexpr int LIGHT = 4;

constexpr int DH_SPLITS = 64;   // most splits of the vocabulary in k_dhidden: a lane each
constexpr int DH_TILES = 1024;  // most tiles of it where there are several splits

// Splits of the vocabulary in k_dhidden for `count` positions (known on the device only): the
// number with the least estimated time.  A tile of 256 x 256 does 64 k in about 1.8 us on one
// CU, the tiles come in rounds over the CUs (smaller tiles: two workgroups per CU, at half
// the rate each), and each split's sums cost a write and a read at some 4 TB/s.
struct DhPlan {
  int tx, bx, by, K, cus, planes;  // tiles along the width, tile, rows per piece, ...
};
__device__ __forceinline__ int dh_splits(const DhPlan &d, int count, int lane) {
  const int tiles = d.tx * ((max(count, 1) + d.by - 1) / d.by), K = d.K, s = lane + 1;
  const int slots = d.bx == 256 ? d.cus : 2 * d.cus;
  const float area = d.bx * d.by / 65536.f;
  const float step = 1.8f * area * (d.planes > 1 ? 3.f : 1.f) * (d.bx == 256 ? 1.f : 2.f);
  float t = (float)((s * tiles + slots - 1) / slots) * step * ((K + 64 * s - 1) / (64 * s)) +
            0.13f * s * tiles * area;
  if (s > 1 && (s * tiles > DH_TILES || K / s < 512)) t = INFINITY;
  float least = t;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) least = fminf(least, __shfl_xor(least, o));
  // lane s - 1 holds s
  return __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(t == least)));
}

// rows of G that k_dhidden takes
inline int64_t dh_rows(const LossArgs &a) { return a.twin ? 2 * a.twin : a.N; }
inline DhPlan dh_plan(const LossArgs &a) {
  return {(int)((a.D + a.dh_bx - 1) / a.dh_bx), a.dh_bx, a.dh_by,
          (int)(a.piece < a.V ? a.piece : a.V), a.cus, a.planes};
}
// floats between two splits of dh
__device__ __forceinline__ int64_t dh_split_stride(int count, int by, int64_t ld) {
  return (int64_t)((count + by - 1) / by) * by * ld;
}

// G is held times 2^14 in fp16 and times 2^32 in bf16, as small probabilities are most of a
// vocabulary and |g| <= 1 keeps both in range.  The matrix cores keep subnormal inputs, so a g
// is off by half a step of 2^-38 or 2^-165 at least.  (LossScalars::ge: bf16 values near the
// type's largest would overflow with this scale on G; where a position's largest sum of
// products or its target's passes G_PLAIN, which tells, G is held as it is.)
__host__ __device__ inline int g_exp(int dtype) { return dtype == TT_DTYPE_BF16 ? 32 : 14; }
constexpr float G_PLAIN = 0x1p90f;

// What the gradients' sums of products are multiplied by: the gradient of the loss (a mean's
// over the positions that count; with a gradient per row, what the factors were divided by)
// over the scales that G and the other operand carry.
struct GradScale {
  const float *up;
  const LossScalars *sc;
  float base;
  int mean;
  __device__ __forceinline__ float get(int e) const {
    const float c = base * *up / (mean ? (float)max(sc->count, 1) : 1.f);
    return ldexpf(c, -e - sc->ge);
  }
};
inline GradScale grad_scale(const LossArgs &a) {
  return {a.reduction == TT_REDUCE_NONE ? a.cm : a.up, a.sv.sc, a.k ? a.temp : 1.f,
          a.reduction == TT_REDUCE_MEAN};
}

// tile shapes (x by y): 0 = 256 x 256, 1 = 128 x 128 for two on a CU, 2 = 128 x 64,
// 3 = 64 x 128, 4 = 64 x 64, 5 = 128 x 128 for one on a CU
struct GemmShape {
  int cfg, bx, by;
};
GemmShape gemm_shape(int64_t x, int64_t y, int cus);  // of products without large tiles
GemmShape dh_shape(const LossArgs &a);
// of `along` large tiles by `across` others, how many of the first to take in large tiles
int64_t large_tiles(int64_t along, int64_t across, int cus);

// A piece of nv rows of the vocabulary in k_logits: the first `large` rows in large tiles, the
// rest in tiles of `rest`; tiles in all.
struct LogitsCut {
  int64_t large;
  GemmShape rest;
  int tiles;
};
inline LogitsCut logits_cut(const LossArgs &a, int64_t nv) {
  LogitsCut c = {0, {}, 0};
  if (a.N > 128 && nv > 128) {
    const int64_t n = large_tiles((nv + 255) / 256, (a.N + 255) / 256, a.cus) * 256;
    c.large = n < nv ? n : nv;
  }
  c.rest = gemm_shape(nv - c.large, a.N, a.cus);
  c.tiles = (int)((c.large + 255) / 256 + (nv - c.large + c.rest.bx - 1) / c.rest.bx);
  return c;
}

hipError_t launch_logits(const LossArgs &a, int64_t v0, int64_t nv, int tile0, bool grad,
                         hipStream_t s);
hipError_t launch_dhidden(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s);
hipError_t launch_dweight(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s);

// the weight's rows [v0, v0 + nv) as an operand: the caller's memory or the packed piece
inline Operand weight_operand(const LossArgs &a, int64_t v0, int64_t nv) {
  Operand o;
  if (a.pack_w) {
    o.p = a.wp; o.ld = a.Dp * 2 * a.planes; o.plane = a.Dp * 2; o.rows = nv; o.cols = a.Dp;
  } else {
    o.p = (const char *)a.weight + v0 * a.wld * 2; o.ld = a.wld * 2; o.plane = 0;
    o.rows = a.V - v0; o.cols = a.D;
  }
  return o;
}
inline Operand hidden_operand(const LossArgs &a) {
  Operand o;
  if (a.direct) {
    o.p = (const char *)a.hidden; o.ld = a.hld * 2; o.plane = 0; o.rows = a.N; o.cols = a.D;
    return o;
  }
  o.p = a.sv.hp; o.ld = a.Dp * 2 * a.planes; o.plane = a.Dp * 2; o.rows = a.Npad; o.cols = a.Dp;
  return o;
}
inline Operand g_operand(const LossArgs &a, int64_t nv) {
  Operand o;
  o.p = a.G; o.ld = a.ldG; o.plane = a.Gplane; o.rows = a.Npad;
  o.cols = (nv + GK - 1) / GK * GK;
  return o;
}

template <class T, class F>
inline hipError_t lds_limit(F *f) {
  static const hipError_t e = hipFuncSetAttribute(
      (const void *)f, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
  return e;
}

// workgroups of a product with that many tiles: as many as the CUs hold at once
template <class T>
inline unsigned gemm_grid(const LossArgs &a, int64_t tiles) {
  const int64_t most = (int64_t)a.cus * (160 * 1024 / T::LDS);
  return (unsigned)(tiles < most ? tiles : most);
}

typedef Tile<256, 256, 128, 64, 2> TileL;
typedef Tile<128, 128, 64, 32, 2> TileM;
typedef Tile<128, 64, 32, 64, 3> TileS;
typedef Tile<64, 128, 32, 64, 3> TileN;
typedef Tile<64, 64, 32, 32, 4> TileT;
typedef Tile<128, 128, 32, 64, 3> TileM1;

}  // namespace ttb
