// tt_loss_grad.hip -- the two products of the backward, on the piece's G as it lies:
//   dh[i][d] = sum_v G_iv W_vd   x = d (columns of the weight), y = positions, k = v
//   dW[v][d] = sum_i G_iv h_id   x = d (columns of the packed positions), y = v, k = positions
// dh is summed in fp32 over the splits and pieces of the vocabulary (each tile owned by one
// workgroup, so the order is fixed); dW is complete in one piece and rounded once.
//
// Bound by the matrix cores: 8192 x 4096 x 16384 bf16 (one piece), dh 0.84 ms and dW 0.83 ms,
// 1.31 and 1.33 PFLOP/s; 2048 x 2048 x 32000 fp16, dh 218 us and dW 247 us.  With few
// positions dW is its own bytes: 2 x 49768 x 1152 bf16, 35 us = 3.3 TB/s.
#include "tt_loss.h"

#include <algorithm>

namespace ttb {

template <class E, class T, int PL, bool MEND, bool WHOLE>
__device__ __forceinline__ void dhidden_tiles(GemmArgs &a, float *out, int64_t ld,
                                              const DhPlan &plan, int add, char *lds) {
  const int n = a.ycount ? *a.ycount : a.yn;
  const int64_t split = dh_split_stride(n, T::Y, ld);
  a.splits = dh_splits(plan, n, threadIdx.x & 63);
  gemm_tiles<E, T, PL, true, false, MEND, WHOLE>(a, lds, [&](const TileAt &t, f4 (&acc)[T::MI][T::NI], char *) {
    const int tid = own_thread(), lane = tid & 63, wv = tid >> 6, g = lane >> 4, c = lane & 15;
    const int x = t.ix * T::X + (wv % T::NWX) * T::wx + 4 * g;
    const int y = t.iy * T::Y + (wv / T::NWX) * T::wy + c;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      if (y + 16 * j >= n) continue;
      float *o = out + t.is * split + (y + 16 * j) * ld + x;
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        if (x + 16 * i >= ld) continue;  // ld is a multiple of 64: whole groups of four
        f4 v = acc[i][j];
        if (add) v += *(const f4 *)(o + 16 * i);
        *(f4 *)(o + 16 * i) = v;
      }
    }
  });
}

template <class E, class T, int PL, bool MEND>
__global__ __launch_bounds__(T::NT) void k_dhidden(GemmArgs a, float *out, int64_t ld,
                                                   DhPlan plan, int add, const LossScalars *sc) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if constexpr (PL > 1)
    if (sc->whole) return dhidden_tiles<E, T, PL, MEND, true>(a, out, ld, plan, add, lds);
  dhidden_tiles<E, T, PL, MEND, false>(a, out, ld, plan, add, lds);
}

template <class O>
struct DwOut {
  O *out;             // dW of the piece's first row
  int64_t ld, nv;     // = D, rows of the piece
  GradScale scale;
};

template <class E, class T, class O, bool WHOLE>
__device__ __forceinline__ void dweight_tiles(const GemmArgs &a, const DwOut<O> &ep, char *lds) {
  const float s = ep.scale.get(ep.scale.sc->eh);
  typedef O o4 __attribute__((ext_vector_type(4)));
  gemm_tiles<E, T, sizeof(O) / 2, true, true, false, WHOLE>(a, lds, [&](const TileAt &t, f4 (&acc)[T::MI][T::NI], char *) {
    const int tid = own_thread(), lane = tid & 63, wv = tid >> 6, g = lane >> 4, c = lane & 15;
      const int x = t.ix * T::X + (wv % T::NWX) * T::wx;
      const int64_t y = (int64_t)t.iy * T::Y + (wv / T::NWX) * T::wy + c;
#pragma unroll
      for (int j = 0; j < T::NI; ++j) {
        O *o = ep.out + (y + 16 * j) * ep.ld + x;
        const bool in = y + 16 * j < ep.nv;
#pragma unroll
        for (int i = 0; i < T::MI; i += 2) {
          o4 v[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[u][r] = (O)(acc[i + u][j][r] * s);
          const int64_t left = ep.ld - (x + 16 * i);  // columns from this pair on
          if constexpr (sizeof(O) == 2) {
            if (left >= 32) {  // a whole pair: 16 bytes a lane (the same for every lane)
              store_pair_if(in, (char *)(o + 16 * i), v[0], v[1], g);
              continue;
            }
          }
          if (!in) continue;
          struct __attribute__((packed, aligned(2))) any { o4 v; };
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int e = 16 * u + 4 * g;
            if (left >= e + 4) {
              const any w = {v[u]};
              *(any *)(o + 16 * i + e) = w;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (e + r < left) o[16 * i + e + r] = v[u][r];
            }
          }
        }
      }
  });
}

template <class E, class T, class O>
__global__ __launch_bounds__(T::NT) void k_dweight(GemmArgs a, DwOut<O> ep) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if constexpr (sizeof(O) > 2)
    if (ep.scale.sc->whole) return dweight_tiles<E, T, O, true>(a, ep, lds);
  dweight_tiles<E, T, O, false>(a, ep, lds);
}

template <class E, class T, int PL, bool MEND>
static hipError_t go_dh(const GemmArgs &g, const LossArgs &a, int add, hipStream_t s) {
  const hipError_t e = lds_limit<T>(&k_dhidden<E, T, PL, MEND>);
  if (e != hipSuccess) return e;
  tt_launch(K_LOSS_DH, k_dhidden<E, T, PL, MEND>, dim3(gemm_grid<T>(a, std::max(g.tx * g.ty, DH_TILES))), dim3(T::NT), T::LDS,
            s, g, a.dhp, a.Dp, dh_plan(a), add, a.sv.sc);
  return hipGetLastError();
}

template <class E, class T, class O>
static hipError_t go_dw(const GemmArgs &g, const LossArgs &a, int64_t v0, int64_t nv,
                        hipStream_t s) {
  const hipError_t e = lds_limit<T>(&k_dweight<E, T, O>);
  if (e != hipSuccess) return e;
  DwOut<O> ep;
  ep.out = (O *)a.dw + v0 * a.D;
  ep.ld = a.D; ep.nv = nv; ep.scale = grad_scale(a);
  tt_launch(K_LOSS_DW, k_dweight<E, T, O>, dim3(gemm_grid<T>(a, (int64_t)g.tx * g.ty)), dim3(T::NT), T::LDS, s, g, ep);
  return hipGetLastError();
}

template <class E, int PL, bool MEND>
static hipError_t pick_dh(int cfg, const GemmArgs &g, const LossArgs &a, int add, hipStream_t s) {
  if (cfg == 0) return go_dh<E, TileL, PL, MEND>(g, a, add, s);
  if (cfg == 1) return go_dh<E, TileM, PL, MEND>(g, a, add, s);
  if (cfg == 3) return go_dh<E, TileN, PL, MEND>(g, a, add, s);
  return go_dh<E, TileS, PL, MEND>(g, a, add, s);
}

hipError_t launch_dhidden(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s) {
  GemmArgs g = {};
  g.P = weight_operand(a, v0, nv);
  g.Q = g_operand(a, nv);
  g.K = (nv + GK - 1) / GK * GK;
  g.xn = (int)a.D;
  g.yn = (int)dh_rows(a);
  g.ycount = a.twin ? nullptr : &a.sv.sc->count;
  const GemmShape t = dh_shape(a);
  g.tx = (int)((a.D + t.bx - 1) / t.bx);
  g.ty = (int)((dh_rows(a) + t.by - 1) / t.by);
  const int add = v0 > 0;
  if (a.planes > 1) return pick_dh<Fp16, 2, false>(t.cfg, g, a, add, s);
  const bool mend = !a.pack_w && a.D % 2;
  if (a.dtype == TT_DTYPE_BF16)
    return mend ? pick_dh<Bf16, 1, true>(t.cfg, g, a, add, s) : pick_dh<Bf16, 1, false>(t.cfg, g, a, add, s);
  return mend ? pick_dh<Fp16, 1, true>(t.cfg, g, a, add, s) : pick_dh<Fp16, 1, false>(t.cfg, g, a, add, s);
}

template <class E, class O>
static hipError_t pick_dw(int cfg, const GemmArgs &g, const LossArgs &a, int64_t v0, int64_t nv,
                          hipStream_t s) {
  if (cfg == 0) return go_dw<E, TileL, O>(g, a, v0, nv, s);
  if (cfg == 1) return go_dw<E, TileM, O>(g, a, v0, nv, s);
  if (cfg == 3) return go_dw<E, TileN, O>(g, a, v0, nv, s);
  if (cfg == 4) return go_dw<E, TileT, O>(g, a, v0, nv, s);
  if (cfg == 5) return go_dw<E, TileM1, O>(g, a, v0, nv, s);
  return go_dw<E, TileS, O>(g, a, v0, nv, s);
}

hipError_t launch_dweight(const LossArgs &a, int64_t v0, int64_t nv, hipStream_t s) {
  int64_t large = 0;
  // with few positions the launch is one of stores: two workgroups on a CU, one of them storing
  if (a.D > 128 && nv > 128 && a.N > 128)
    large = std::min(nv, large_tiles((nv + 255) / 256, (a.D + 255) / 256, a.cus) * 256);
  hipError_t e = hipSuccess;
  // rows [r0, r0 + n) of the piece in tiles of t
  auto part = [&](int64_t r0, int64_t n, GemmShape t) {
    if (n <= 0 || e != hipSuccess) return;
    GemmArgs g = {};
    g.P = hidden_operand(a);
    g.Q = g_operand(a, nv);
    g.Q.p += r0 * 2;
    g.Q.cols -= r0;
    g.K = a.Npad;
    g.xn = (int)a.D;
    g.yn = (int)n;
    g.kcount = a.twin ? nullptr : &a.sv.sc->count;
      g.tx = (int)((a.D + t.bx - 1) / t.bx);
    g.ty = (int)((n + t.by - 1) / t.by);
    g.splits = 1;
    if (a.dtype == TT_DTYPE_BF16) e = pick_dw<Bf16, __bf16>(t.cfg, g, a, v0 + r0, n, s);
    else if (a.dtype == TT_DTYPE_F16) e = pick_dw<Fp16, _Float16>(t.cfg, g, a, v0 + r0, n, s);
    else e = pick_dw<Fp16, float>(t.cfg, g, a, v0 + r0, n, s);
  };
  part(0, large, {0, 256, 256});
  part(large, nv - large, gemm_shape(a.D, nv - large, a.cus));
  return e;
}

}  // namespace ttb
