// tt_loss_logits.hip -- logits of a piece of the vocabulary, a tile at a time: their running
// statistics for the forward, or the gradient G in 16 bits for the two products that follow.
//
// x = rows of the weight, y = packed positions, so a lane holds 4 consecutive vocabulary rows
// of one position: statistics are sums over a lane's own registers, then over the 4 lane
// groups, then over the waves that share the positions.  Statistics and exponentials are fp32
// in base 2 (the logits are scaled by log2 e once).
//
// Bound by the matrix cores from some 200 positions on, below that by the weight's bytes.
// Measured (MI355X): 8192 x 131072 x 4096 bf16, statistics 6.4 ms = 1.37 PFLOP/s; a piece of
// G (16384 rows of the vocabulary) 0.83 ms = 1.33 PFLOP/s (without its results 1.52: the
// exponentials and 128 KiB of stores per tile are not hidden); 1024 x 32000 x 1024 fp32, 160
// and 175 us (1.26 and 1.15 PFLOP/s over three products); 48 x 131072 x 2048 fp16, 107 us = 5.0
// TB/s of weight.
#include "tt_loss.h"

namespace ttb {

struct LogitsEpi {
  const LossScalars *sc;   // null: n positions and the scale zs
  int n;
  float zs;
  int64_t v0, nv;          // the piece
  float2 *part;
  float *zpart;
  int ptiles, tile0;
  char *G;
  int64_t ldG, Gplane;
  const float *mx, *lg, *rowf;
  const int *tgt;          // null with distillation
  const int64_t *tgt64;    // the caller's targets instead (loss alone), or null
  float *zt;
  int twin;
  float one_e, e_v;        // 1 - e, e / V
};

template <class E, class T, int PL, bool GRAD, bool MEND, bool WHOLE>
__device__ __forceinline__ void logits_tiles(const GemmArgs &a, const LogitsEpi &ep, char *lds) {
  gemm_tiles<E, T, PL, false, false, MEND, WHOLE>(a, lds, [&](const TileAt &t, f4 (&acc)[T::MI][T::NI], char *tmp) {
    const int tid = own_thread(), lane = tid & 63, wv = tid >> 6, g = lane >> 4, c = lane & 15;
    const int px = (wv % T::NWX) * T::wx, qy = (wv / T::NWX) * T::wy;
    const float zs = ep.sc ? ep.sc->zs : ep.zs;
    const int count = ep.sc ? ep.sc->count : ep.n;
    const int ix = t.ix, iy = t.iy;
    const int xl = (int)min<int64_t>(ep.nv - (int64_t)ix * T::X, T::X);  // rows of this tile
    const int xb = px + 4 * g;
    const bool full = xl == T::X;  // no rows of the tile past the vocabulary
    if constexpr (!GRAD) {
      float2 *sm = (float2 *)tmp;                       // [NWX][Y]
      float *sz = (float *)(tmp + T::NWX * T::Y * 8);   // [NWX][Y]
      int d_[T::NI];  // the target's place from this lane's first row, or -1
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        const int pos = iy * T::Y + qy + 16 * j + c;
        const int64_t first = ep.v0 + (int64_t)ix * T::X + xb;
        const int64_t t = !ep.zt || pos >= count ? -1 : ep.tgt64 ? ep.tgt64[pos] : ep.tgt[pos];
        d_[j] = (int)max<int64_t>(min<int64_t>(t - first, 1 << 20), -1);
      }
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        float m = -INFINITY, zsum = 0.f;
        // the target's logit is the one that the sum below has in it
        if (__any(d_[j] >= 0 && d_[j] < 16 * T::MI)) {
#pragma unroll
          for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (d_[j] == 16 * i + r && d_[j] + xb < xl)
                ep.zt[iy * T::Y + qy + 16 * j + c] = acc[i][j][r];
        }
        if (ep.zpart) {
#pragma unroll
          for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) zsum += xb + 16 * i + r < xl ? acc[i][j][r] : 0.f;
          zsum *= zs;
        }
        if (!full) {
#pragma unroll
          for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (xb + 16 * i + r >= xl) acc[i][j][r] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float m0 = m == -INFINITY ? 0.f : m;  // nothing but -inf: every term is 0
        // the difference first: m zs overflows where all rows hold a type's lowest value
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) s += __builtin_amdgcn_exp2f((acc[i][j][r] - m0) * zs);
        s = sum_lane_groups(s);
        if (ep.zpart) zsum = sum_lane_groups(zsum);
        if (g == 0) {
          sm[(wv % T::NWX) * T::Y + qy + 16 * j + c] = make_float2(m, s);
          if (ep.zpart) sz[(wv % T::NWX) * T::Y + qy + 16 * j + c] = zsum;
        }
      }
      lds_barrier();
      for (int y = tid; y < T::Y; y += T::NT) {
        const int pos = iy * T::Y + y;
        if (pos >= count) continue;
        float m = -INFINITY, s = 0.f, z = 0.f;
#pragma unroll
        for (int w = 0; w < T::NWX; ++w) m = fmaxf(m, sm[w * T::Y + y].x);
        const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < T::NWX; ++w) {
          const float2 q = sm[w * T::Y + y];
          s += q.y * __builtin_amdgcn_exp2f((q.x - m0) * zs);
          if (ep.zpart) z += sz[w * T::Y + y];
        }
        const int64_t at = (int64_t)pos * ep.ptiles + ep.tile0 + ix;
        ep.part[at] = make_float2(m, s);
        if (ep.zpart) ep.zpart[at] = z;
      }
      lds_barrier();
    } else {
      // p 2^g_exp as the square of exp2 of half the logit, times the row's factor: v_exp_f32
      // itself ends at 2^-126, bf16 and the gradients do not
      const float zh = 0.5f * zs, gs = ldexpf(1.f, ep.sc->ge);
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        const int pos = iy * T::Y + qy + 16 * j + c;
        const bool live = pos < count;
        if (ep.twin && qy + 16 * j >= ep.twin) continue;
        const float mx = live ? ep.mx[pos] : 0.f, lg = live ? 0.5f * ep.lg[pos] : 0.f,
                    f = live ? (ep.rowf ? ep.rowf[pos] : 1.f) * gs : 0.f;
        const float ef = ep.e_v * f;
        const int64_t first = ep.v0 + (int64_t)ix * T::X + xb;
        const int d = live && ep.tgt ? (int)(ep.tgt[pos] - first) : -1;
        // few tiles hold the target of one of a wave's 16 positions
        const bool hit = __any(d >= 0 && d < 16 * T::MI);
        char *o = ep.G + pos * ep.ldG + ((int64_t)ix * T::X + px) * 2;
#pragma unroll
        for (int i0 = 0; i0 < T::MI; i0 += 2) {
          typename E::v4 h[2], l[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = i0 + u;
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float q = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r] - mx, zh, -lg));
              v[r] = __builtin_fmaf(q * q, f, -ef);
            }
            if (hit) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (d == 16 * i + r) v[r] -= ep.one_e * f;
            }
            if (!full) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (xb + 16 * i + r >= xl) v[r] = 0.f;
            }
            if (!live) v[0] = v[1] = v[2] = v[3] = 0.f;
            if constexpr (WHOLE) {
              halves(v, h[u], l[u]);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r) h[u][r] = (typename E::e)v[r];
#pragma unroll
              for (int r = 0; r < 4; ++r) l[u][r] = (typename E::e)(v[r] - (float)h[u][r]);
            }
          }
          store_pair(o + 32 * i0, h[0], h[1], g);
          if (PL > 1 || ep.twin) store_pair(o + ep.Gplane + 32 * i0, l[0], l[1], g);
        }
      }
    }
  });
}

template <class E, class T, int PL, bool GRAD, bool MEND>
__global__ __launch_bounds__(T::NT) void k_logits(GemmArgs a, LogitsEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if constexpr (PL > 1)
    if (ep.sc->whole) return logits_tiles<E, T, PL, GRAD, MEND, true>(a, ep, lds);
  logits_tiles<E, T, PL, GRAD, MEND, false>(a, ep, lds);
}

template <class E, class T, int PL, bool GRAD, bool MEND>
static hipError_t go(const LossArgs &a, const GemmArgs &g, const LogitsEpi &ep, hipStream_t s) {
  const hipError_t e = lds_limit<T>(&k_logits<E, T, PL, GRAD, MEND>);
  if (e != hipSuccess) return e;
  tt_launch(GRAD ? K_LOSS_G : K_LOSS_LOGITS, k_logits<E, T, PL, GRAD, MEND>,
            dim3(gemm_grid<T>(a, (int64_t)g.tx * g.ty)), dim3(T::NT), T::LDS, s, g, ep);
  return hipGetLastError();
}

template <class E, int PL, bool GRAD, bool MEND>
static hipError_t pick(int cfg, const LossArgs &a, const GemmArgs &g, const LogitsEpi &ep,
                       hipStream_t s) {
  if (cfg == 0) return go<E, TileL, PL, GRAD, MEND>(a, g, ep, s);
  if (cfg == 1) return go<E, TileM, PL, GRAD, MEND>(a, g, ep, s);
  if (cfg == 3) return go<E, TileN, PL, GRAD, MEND>(a, g, ep, s);
  if (cfg == 4) return go<E, TileT, PL, GRAD, MEND>(a, g, ep, s);
  if (cfg == 5) return go<E, TileM1, PL, GRAD, MEND>(a, g, ep, s);
  return go<E, TileS, PL, GRAD, MEND>(a, g, ep, s);
}

template <class E, int PL, bool MEND>
static hipError_t pick(bool grad, int cfg, const LossArgs &a, const GemmArgs &g,
                       const LogitsEpi &ep, hipStream_t s) {
  return grad ? pick<E, PL, true, MEND>(cfg, a, g, ep, s)
              : pick<E, PL, false, MEND>(cfg, a, g, ep, s);
}

template <class E, int PL>
static hipError_t pick(bool grad, int cfg, const LossArgs &a, const GemmArgs &g,
                       const LogitsEpi &ep, hipStream_t s) {
  if constexpr (PL == 1)
    if (!a.pack_w && a.D % 8) return pick<E, PL, true>(grad, cfg, a, g, ep, s);
  return pick<E, PL, false>(grad, cfg, a, g, ep, s);
}

hipError_t launch_logits(const LossArgs &a, int64_t v0, int64_t nv, int tile0, bool grad,
                         hipStream_t s) {
  LogitsEpi ep = {};
  ep.sc = a.direct ? nullptr : a.sv.sc;
  ep.n = (int)a.N;
  ep.zs = 1.4426950408889634f / a.temp;
  ep.part = a.part; ep.zpart = a.smoothing > 0.f ? a.zpart : nullptr;
  ep.ptiles = a.ptiles; ep.tile0 = tile0;
  ep.twin = a.twin;
  ep.ldG = a.ldG; ep.Gplane = a.Gplane;
  ep.mx = a.sv.mx; ep.lg = a.sv.lg; ep.rowf = a.reduction == TT_REDUCE_NONE ? a.rowf : nullptr;
  ep.tgt = a.k ? nullptr : a.sv.tgt;
  ep.tgt64 = a.direct ? a.tgt : nullptr;
  ep.zt = a.k || grad ? nullptr : a.sv.zt;
  ep.one_e = 1.f - a.smoothing;
  ep.e_v = a.smoothing / (float)a.V;
  const LogitsCut cut = logits_cut(a, nv);
  hipError_t e = hipSuccess;
  // rows [r0, r0 + n) of the piece in tiles of t
  auto part = [&](int64_t r0, int64_t n, GemmShape t) {
    if (n <= 0 || e != hipSuccess) return;
    GemmArgs g = {};
    g.P = weight_operand(a, v0, nv);
    g.P.p += r0 * g.P.ld;
    g.P.rows -= r0;
    g.Q = hidden_operand(a);
    g.K = a.pack_w ? a.Dp : a.D;
    g.xn = (int)n;
    g.yn = (int)a.N;
    // twin rows of G are used whole, so all are written
    g.ycount = a.direct || (grad && a.twin) ? nullptr : &a.sv.sc->count;
    g.tx = (int)((n + t.bx - 1) / t.bx);
    g.ty = (int)((a.N + t.by - 1) / t.by);
    g.splits = 1;
    ep.v0 = v0 + r0;
    ep.nv = n;
    ep.G = a.G + r0 * 2;
    if (a.dtype == TT_DTYPE_BF16) e = pick<Bf16, 1>(grad, t.cfg, a, g, ep, s);
    else if (a.dtype == TT_DTYPE_F16) e = pick<Fp16, 1>(grad, t.cfg, a, g, ep, s);
    else e = pick<Fp16, 2>(grad, t.cfg, a, g, ep, s);
    ep.tile0 += g.tx;
  };
  part(0, cut.large, {0, 256, 256});
  part(cut.large, nv - cut.large, cut.rest);
  return e;
}

}  // namespace ttb
