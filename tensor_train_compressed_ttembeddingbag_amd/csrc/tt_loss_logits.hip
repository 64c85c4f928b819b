// tt_loss_logits.hip -- logits of a piece of the vocabulary, a tile at a time: their running
// statistics for the forward, or the gradient G in 16 bits for the two products that follow.
//
// x = rows of the weight, y = packed positions, so a lane holds 4 consecutive vocabulary rows
// of one position: statistics are sums over a lane's own registers, then over the 4 lane
// groups, then over the waves that share the positions.  Statistics and exponentials are fp32
// in base 2 (the logits are scaled by log2 e once).
#include "tt_loss.h"

namespace ttb {

struct LogitsEpi {
  const LossScalars *sc;
  const int *count;
  int64_t v0, nv;          // the piece
  float2 *part;
  float *zpart;
  int ptiles, tile0;
  char *G;
  int64_t ldG, Gplane;
  const float *lse, *rowf;
  const int *tgt;          // null with distillation
  float one_e, e_v, ghalf; // (1 - e) and e / V times G's factor 2^g_exp; the root of that
  int planes;
};

template <class E, class T, bool GRAD>
__global__ __launch_bounds__(T::NT) void k_logits(GemmArgs a, LogitsEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  int ix, iy, is;
  if (!tile_of<T::Y>(a, ix, iy, is)) return;
  f4 acc[T::MI][T::NI];
  if (!gemm_tile<E, T, false, false>(a, lds, ix, iy, is, acc)) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, g = lane >> 4, c = lane & 15;
  const int px = (wv % T::NWX) * T::wx, qy = (wv / T::NWX) * T::wy;
  const float zs = ep.sc->zs;
  const int count = *ep.count;
  const int xl = (int)min<int64_t>(ep.nv - (int64_t)ix * T::X, T::X);  // rows of this tile
  const int xb = px + 4 * g;
  if constexpr (!GRAD) {
    float2 *sm = (float2 *)lds;                       // [NWX][Y]
    float *sz = (float *)(lds + T::NWX * T::Y * 8);   // [NWX][Y]
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      float m = -INFINITY, zsum = 0.f;
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool in = xb + 16 * i + r < xl;
          const float u = acc[i][j][r] * zs;
          zsum += in ? u : 0.f;
          acc[i][j][r] = in ? u : -INFINITY;
          m = fmaxf(m, acc[i][j][r]);
        }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float m0 = m == -INFINITY ? 0.f : m;  // nothing but -inf: every term is 0
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) s += __builtin_amdgcn_exp2f(acc[i][j][r] - m0);
      s = sum_lane_groups(s);
      if (ep.zpart) zsum = sum_lane_groups(zsum);
      if (g == 0) {
        sm[(wv % T::NWX) * T::Y + qy + 16 * j + c] = make_float2(m, s);
        if (ep.zpart) sz[(wv % T::NWX) * T::Y + qy + 16 * j + c] = zsum;
      }
    }
    __syncthreads();
    for (int y = tid; y < T::Y; y += T::NT) {
      const int pos = iy * T::Y + y;
      if (pos >= count) break;
      float m = -INFINITY, s = 0.f, z = 0.f;
#pragma unroll
      for (int w = 0; w < T::NWX; ++w) m = fmaxf(m, sm[w * T::Y + y].x);
      const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < T::NWX; ++w) {
        const float2 q = sm[w * T::Y + y];
        s += q.y * __builtin_amdgcn_exp2f(q.x - m0);
        if (ep.zpart) z += sz[w * T::Y + y];
      }
      const int64_t at = (int64_t)pos * ep.ptiles + ep.tile0 + ix;
      ep.part[at] = make_float2(m, s);
      if (ep.zpart) ep.zpart[at] = z;
    }
  } else {
    const float zh = 0.5f * zs;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int pos = iy * T::Y + qy + 16 * j + c;
      const bool live = pos < count;
      const float lse = live ? 0.5f * ep.lse[pos] : 0.f, f = live ? ep.rowf[pos] : 0.f;
      const int64_t first = ep.v0 + (int64_t)ix * T::X + xb;
      const int d = live && ep.tgt ? (int)(ep.tgt[pos] - first) : -1;
      char *o = ep.G + pos * ep.ldG + ((int64_t)ix * T::X + xb) * 2;
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // as the square of exp2 of half: v_exp_f32 itself ends at 2^-126
          const float q = __builtin_amdgcn_exp2f(acc[i][j][r] * zh - lse) * ep.ghalf;
          float p = q * q - ep.e_v;
          if (d == 16 * i + r) p -= ep.one_e;
          v[r] = live && xb + 16 * i + r < xl ? p * f : 0.f;
        }
        typename E::v4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = (typename E::e)v[r];
        *(typename E::v4 *)(o + 32 * i) = h;
        if (ep.planes > 1) {
          typename E::v4 l;
#pragma unroll
          for (int r = 0; r < 4; ++r) l[r] = (typename E::e)(v[r] - (float)h[r]);
          *(typename E::v4 *)(o + ep.Gplane + 32 * i) = l;
        }
      }
    }
  }
}

template <class E, class T, bool GRAD>
static hipError_t go(const GemmArgs &g, const LogitsEpi &ep, hipStream_t s) {
  const hipError_t e = lds_limit<T>(&k_logits<E, T, GRAD>);
  if (e != hipSuccess) return e;
  tt_launch(GRAD ? K_LOSS_G : K_LOSS_LOGITS, k_logits<E, T, GRAD>, dim3(g.tx * g.ty), dim3(T::NT),
            T::LDS, s, g, ep);
  return hipGetLastError();
}

template <class E, bool GRAD>
static hipError_t pick(int cfg, const GemmArgs &g, const LogitsEpi &ep, hipStream_t s) {
  if (cfg == 0) return go<E, TileL, GRAD>(g, ep, s);
  if (cfg == 1) return go<E, TileM, GRAD>(g, ep, s);
  return go<E, TileS, GRAD>(g, ep, s);
}

hipError_t launch_logits(const LossArgs &a, int64_t v0, int64_t nv, int tile0, bool grad,
                         hipStream_t s) {
  GemmArgs g = {};
  g.P = weight_operand(a, v0, nv);
  g.Q = hidden_operand(a);
  g.K = g.kper = a.pack_w ? a.Dp : a.D;
  g.kper = (g.K + GK - 1) / GK * GK;
  g.ycount = a.sv.count;
  g.nseg = a.planes > 1 ? 3 : 1;
  const GemmShape t = gemm_shape(a.V < a.piece ? a.V : a.piece, a.N);
  g.tx = (int)((nv + t.bx - 1) / t.bx);
  g.ty = (int)((a.N + t.by - 1) / t.by);
  g.splits = 1;
  LogitsEpi ep = {};
  ep.sc = a.sc; ep.count = a.sv.count;
  ep.v0 = v0; ep.nv = nv;
  ep.part = a.part; ep.zpart = a.smoothing > 0.f ? a.zpart : nullptr;
  ep.ptiles = a.ptiles; ep.tile0 = tile0;
  ep.G = a.G; ep.ldG = a.ldG; ep.Gplane = a.Gplane;
  ep.lse = a.sv.lse; ep.rowf = a.rowf;
  ep.tgt = a.k ? nullptr : a.sv.tgt;
  ep.ghalf = ldexpf(1.f, g_exp(a.dtype) / 2);
  ep.one_e = ldexpf(1.f - a.smoothing, g_exp(a.dtype));
  ep.e_v = ldexpf(a.smoothing / (float)a.V, g_exp(a.dtype));
  ep.planes = a.planes;
  if (a.dtype == TT_DTYPE_BF16)
    return grad ? pick<Bf16, true>(t.cfg, g, ep, s) : pick<Bf16, false>(t.cfg, g, ep, s);
  return grad ? pick<Fp16, true>(t.cfg, g, ep, s) : pick<Fp16, false>(t.cfg, g, ep, s);
}

}  // namespace ttb
