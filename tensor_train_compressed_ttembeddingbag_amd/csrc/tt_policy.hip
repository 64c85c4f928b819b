// tt_policy.hip -- losses that are functions of the targets' log-probabilities under a vocabulary
// head, l_i = log softmax(<hidden_i, weight> / T) at the target: preference losses over pairs of
// sequences and the clipped policy loss.
//
// Both are cross entropy without a reduction (tt_loss.hip), some arithmetic per position between its
// forward and its backward, and dL/dl_i as the gradient that the backward is given.  The arithmetic is
// fp64: log-probabilities of some -10 are rounded to 2^-21, and what comes here are their sums over
// sequences, differences and ratios next to a bound, of which fp32 would lose more than that.  It is
// 12 to 40 bytes a position beside a product of the whole vocabulary (4096 positions: 9 us and 5 us for their sum).
// No result depends on the order of atomics: sums go in a fixed order.
#include "tt_loss.h"

#include <algorithm>

namespace ttb {

// positions whose sum one workgroup takes in the launch that works them out
constexpr int64_t ONE_BLOCK = 2048;
constexpr int SUM_BLOCK = 1024;  // positions per partial sum past that

// pairs whose rows the last workgroup adds up (tickets go through one address at some 13 ns each)
constexpr int64_t TICKETS = 256;

struct PreferArgs {
  int64_t N, V, P, ignore;
  int kind, average, reduction;
  double beta, smoothing, margin;
  const int64_t *tgt, *off;
  const float *nll, *ref;   // ref may be null
  float *loss, *ratios;     // [P] or [1]; [2 P] or null
  double *rows;             // [P] (workspace)
  int32_t *status;
  int *ticket;              // the last workgroup adds the rows up, or null
  // saved, or null
  int *seq;                 // [N] a position's sequence
  float *coef;              // [2 P] dL/dl of its positions, for a gradient of 1 of its pair's loss
};

struct PolicyArgs {
  int64_t N, V, ignore;
  int reduction;
  double low, high, kl;
  const int64_t *tgt;
  const float *nll, *adv, *old, *ref;  // old and ref may be null
  float *loss, *logps;                 // [N] or [1]; [N] or null
  double *part;                        // [blocks][2] (workspace)
  float *coef;                         // [N] dloss/dl, or null
};

__device__ __forceinline__ bool in_vocabulary(int64_t t, int64_t ignore, int64_t V) {
  return t != ignore && t >= 0 && t < V;
}

// sums of two values over a block's threads, in a fixed order; every thread gets them
template <int NT>
__device__ __forceinline__ void block_sums(double &x, double &y, double (*s)[2]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    x += __shfl_xor(x, o);
    y += __shfl_xor(y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6][0] = x, s[threadIdx.x >> 6][1] = y;
  __syncthreads();
  x = y = 0.0;
  for (int w = 0; w < NT / 64; ++w) x += s[w][0], y += s[w][1];
}

// the loss and the slopes of pair p from its sequences' sums and counts, four of each
__device__ __forceinline__ void prefer_pair(const PreferArgs &a, int64_t p, const double (*s_sum)[2]) {
  double h[2], share[2];
  for (int k = 0; k < 2; ++k) {
    double s = 0.0, c = 0.0;
    for (int w = 0; w < 4; ++w) s += s_sum[4 * k + w][0], c += s_sum[4 * k + w][1];
    share[k] = a.average ? 1.0 / fmax(c, 1.0) : 1.0;
    h[k] = s * share[k];
    if (a.ratios) a.ratios[p + k * a.P] = (float)h[k];
  }
  const double x = h[0] - h[1];
  double row, slope;  // the pair's loss, and its derivative by x
  if (a.kind == TT_PREFER_SQUARE) {
    const double gap = x - 0.5 / a.beta;
    row = gap * gap;
    slope = 2.0 * gap;
  } else {
    const double y = a.beta * x - a.margin;
    if (a.kind == TT_PREFER_HINGE) {
      const bool short_of = !(y >= 1.0);
      row = short_of ? 1.0 - y : 0.0;
      slope = short_of ? -a.beta : 0.0;
    } else {
      // -log S(y) = log(1 + exp -|y|) + max(0, -y); a weight of 0 takes nothing from an infinity
      const double e = a.smoothing, far = exp(-fabs(y));
      row = log1p(far);
      if (!(y >= 0.0) && e < 1.0) row += (1.0 - e) * -y;
      if (!(y <= 0.0) && e > 0.0) row += e * y;
      // S(y) - (1 - e) by the smaller of S(y) and S(-y)
      const double small = far / (1.0 + far);
      slope = a.beta * (y >= 0.0 ? e - small : small - (1.0 - e));
    }
  }
  __hip_atomic_store(&a.rows[p], row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (a.reduction == TT_REDUCE_NONE) a.loss[p] = (float)row;
  if (a.coef) {
    a.coef[p] = (float)(slope * share[0]);
    a.coef[p + a.P] = (float)(-slope * share[1]);
  }
}

// the rows' sum in a fixed order
template <int NT>
__device__ __forceinline__ void add_rows(const PreferArgs &a) {
  __shared__ double s_add[NT / 64][2];
  double x = 0.0, none = 0.0;
  for (int64_t i = threadIdx.x; i < a.P; i += NT)
    x += __hip_atomic_load(&a.rows[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  block_sums<NT>(x, none, s_add);
  if (threadIdx.x == 0)
    a.loss[0] = (float)(a.reduction == TT_REDUCE_MEAN ? x / (double)max(a.P, (int64_t)1) : x);
}

// A pair per workgroup: half of it adds the preferred sequence up, half the other one.
__global__ __launch_bounds__(512) void k_prefer(PreferArgs a) {
  __shared__ double s_sum[8][2];
  const int tid = threadIdx.x, half = tid >> 8, t = tid & 255;
  const int64_t p = blockIdx.x, q = p + half * a.P;
  int64_t i0 = a.off[q], i1 = a.off[q + 1];
  if (i0 < 0 || i1 < i0 || i1 > a.N || (q == 0 && i0 != 0)) {
    if (t == 0) set_status(a.status, TT_DEV_BAD_OFFSETS);
    i0 = i1 = 0;
  }
  double sum = 0.0, n = 0.0;
#pragma unroll 4
  for (int64_t i = i0 + t; i < i1; i += 256) {
    const float l = -a.nll[i], r = a.ref ? a.ref[i] : 0.f;
    if (in_vocabulary(a.tgt[i], a.ignore, a.V)) {
      sum += (double)l - (double)r;
      n += 1.0;
    }
    if (a.seq) a.seq[i] = (int)q;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    sum += __shfl_xor(sum, o);
    n += __shfl_xor(n, o);
  }
  if ((tid & 63) == 0) s_sum[tid >> 6][0] = sum, s_sum[tid >> 6][1] = n;
  __syncthreads();
  __shared__ int s_last;
  if (tid == 0) prefer_pair(a, p, s_sum);
  if (!a.ticket) return;
  // A row is written through to memory by its own scope, and the ticket waits for it alone.
  if (tid == 0) {
    vmem_drain();
    s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) add_rows<512>(a);
}

__global__ __launch_bounds__(256) void k_prefer_sum(PreferArgs a) { add_rows<256>(a); }

struct PolicyRow {
  double loss, coef;
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs &a, int64_t i, double l) {
  const double A = (double)a.adv[i];
  const double r = a.old ? exp(l - (double)a.old[i]) : 1.0;
  const double lo = 1.0 - a.low, hi = 1.0 + a.high;
  const double held = (r < lo ? lo : r > hi ? hi : r) * A, free = r * A;
  const bool clipped = free > held;  // (not if either is no number: that goes on into the loss)
  PolicyRow o = {clipped ? -held : -free, clipped ? 0.0 : -free};
  if (a.kl != 0.0) {
    const double d = (double)a.ref[i] - l, m = expm1(d);
    o.loss += a.kl * (m == INFINITY ? m : m - d);
    o.coef -= a.kl * m;
  }
  return o;
}

// NT positions at a time per workgroup; with a reduction each workgroup takes `per` positions and
// leaves their sum and how many count, or the loss where it is the only one.
template <int NT>
__global__ __launch_bounds__(NT) void k_policy(PolicyArgs a, int64_t per) {
  __shared__ double s_sum[NT / 64][2];
  const int64_t i0 = (int64_t)blockIdx.x * per, i1 = min(i0 + per, a.N);
  double sum = 0.0, n = 0.0;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += NT) {
    const bool on = in_vocabulary(a.tgt[i], a.ignore, a.V);
    const float l = -a.nll[i];
    PolicyRow r = {0.0, 0.0};
    if (on) r = policy_row(a, i, (double)l);
    if (a.logps) a.logps[i] = on ? l : 0.f;
    if (a.coef) a.coef[i] = (float)r.coef;
    if (a.reduction == TT_REDUCE_NONE) a.loss[i] = (float)r.loss;
    sum += r.loss;
    n += on;
  }
  if (a.reduction == TT_REDUCE_NONE) return;
  block_sums<NT>(sum, n, s_sum);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) {
    a.loss[0] = (float)(a.reduction == TT_REDUCE_MEAN ? sum / fmax(n, 1.0) : sum);
  } else {
    a.part[2 * blockIdx.x] = sum;
    a.part[2 * blockIdx.x + 1] = n;
  }
}
__global__ __launch_bounds__(256) void k_policy_sum(PolicyArgs a, int64_t blocks) {
  __shared__ double s_sum[4][2];
  double sum = 0.0, n = 0.0;
  for (int64_t b = threadIdx.x; b < blocks; b += 256) sum += a.part[2 * b], n += a.part[2 * b + 1];
  block_sums<256>(sum, n, s_sum);
  if (threadIdx.x == 0) a.loss[0] = (float)(a.reduction == TT_REDUCE_MEAN ? sum / fmax(n, 1.0) : sum);
}

// ---------------------------------------------------------------- host
static int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
static int64_t elem_size(int dtype) { return dtype == TT_DTYPE_F32 ? 4 : 2; }

struct Part {  // of a buffer, behind what the cross entropy has in it
  char *base;
  int64_t off;
  template <class T>
  void take(T *&p, int64_t n) {
    p = (T *)(base + off);
    off = round_up(off + n * (int64_t)sizeof(T), 256);
  }
};

template <class Desc>
static int cross_entropy(const Desc *d, const void *weight, float temperature, LossArgs &a) {
  if (!d) return TT_EINVAL;
  const tt_loss_desc l = {d->n, d->v, d->d, d->hidden_stride, d->weight_stride, d->ignore_index,
                          d->dtype, TT_DTYPE_F32, TT_REDUCE_NONE, 0, 0.f, 1.f};
  if (d->reduction < TT_REDUCE_NONE || d->reduction > TT_REDUCE_SUM) return TT_EINVAL;
  if (!(temperature > 0.f && temperature < INFINITY)) return TT_EINVAL;
  const int rc = loss_args(&l, weight, a);
  a.temp = temperature;
  a.few32 = 1;
  return rc;
}

// Products of positions, rows and columns from which on the backward of a loss whose slope is exactly 0 for
// some positions (clipped, or without an advantage; hinge: pairs that are far enough apart) leaves these
// out: a copy of the others costs some 10 us at 2^36, of which three products are 320 us.
constexpr double KEEP_FROM = (double)(1ll << 36);
static bool keeps(const LossArgs &a, bool zero_slopes) {
  return zero_slopes && !a.twin && (double)a.N * (double)a.V * (double)a.D >= KEEP_FROM;
}

static bool finite(double x) { return x > -INFINITY && x < INFINITY; }

static int prefer_args(const tt_prefer_desc *d, const void *weight, LossArgs &a, PreferArgs &p) {
  const int rc = cross_entropy(d, weight, 1.f, a);
  if (rc != TT_OK) return rc;
  if (d->pairs < 0 || d->kind < TT_PREFER_SIGMOID || d->kind > TT_PREFER_SQUARE) return TT_EINVAL;
  if (!(d->beta > 0.0) || !finite(d->beta) || !finite(d->margin)) return TT_EINVAL;
  if (!(d->label_smoothing >= 0.0 && d->label_smoothing <= 1.0)) return TT_EINVAL;
  if (d->label_smoothing != 0.0 && d->kind != TT_PREFER_SIGMOID) return TT_EINVAL;
  if (d->margin != 0.0 && d->kind == TT_PREFER_SQUARE) return TT_EINVAL;
  if (d->pairs >= (1 << 23)) return TT_ESHAPE;  // a launch has less than 2^32 threads, 512 of them a pair
  p = {};
  p.N = d->n; p.V = d->v; p.P = d->pairs; p.ignore = d->ignore_index;
  p.kind = d->kind; p.average = d->average != 0; p.reduction = d->reduction;
  p.beta = d->beta; p.smoothing = d->label_smoothing; p.margin = d->margin;
  return TT_OK;
}
static int64_t prefer_saved(LossArgs &a, PreferArgs &p, void *saved) {
  Part b = {(char *)saved, saved_layout(a, saved)};
  b.take(p.seq, p.N);
  b.take(p.coef, 2 * p.P);
  return b.off;
}
static bool zero_slopes(const PreferArgs &p) { return p.kind == TT_PREFER_HINGE; }
static bool zero_slopes(const PolicyArgs &p) { return p.kl == 0.0; }
// what a backward has beside the cross entropy's: the rows that are kept
template <class Args>
static void backward_part(const LossArgs &a, const Args &p, Part &b, Kept &kept) {
  if (keeps(a, zero_slopes(p))) b.off += kept_layout(a, b.base + b.off, kept);
}
template <class Args>
static hipError_t backward_from(LossArgs &a, const Args &p, const Kept &kept, hipStream_t s) {
  if (p.N && keeps(a, zero_slopes(p))) {
    const hipError_t e = keep_rows(a, kept, s);
    if (e != hipSuccess) return e;
  }
  return loss_backward(a, s);
}

static int64_t prefer_ws(LossArgs &a, PreferArgs &p, void *ws, int mode, Kept &kept) {
  Part b = {(char *)ws, ws_layout(a, ws, mode)};
  if (mode == TT_LOSS_BACKWARD) {
    backward_part(a, p, b, kept);
  } else {
    b.take(a.loss, p.N);
    b.take(p.rows, p.P);
    p.nll = a.loss;
  }
  return std::max<int64_t>(b.off, 256);
}

static int policy_args(const tt_policy_desc *d, const void *weight, LossArgs &a, PolicyArgs &p) {
  const int rc = cross_entropy(d, weight, d ? d->temperature : 1.f, a);
  if (rc != TT_OK) return rc;
  if (!(d->clip_low >= 0.0) || !(d->clip_high >= 0.0)) return TT_EINVAL;
  if (!(d->kl_coef >= 0.0) || !finite(d->kl_coef)) return TT_EINVAL;
  p = {};
  p.N = d->n; p.V = d->v; p.ignore = d->ignore_index; p.reduction = d->reduction;
  p.low = d->clip_low; p.high = d->clip_high; p.kl = d->kl_coef;
  return TT_OK;
}
static int64_t policy_saved(LossArgs &a, PolicyArgs &p, void *saved) {
  Part b = {(char *)saved, saved_layout(a, saved)};
  b.take(p.coef, p.N);
  return b.off;
}
static int64_t policy_ws(LossArgs &a, PolicyArgs &p, void *ws, int mode, Kept &kept) {
  Part b = {(char *)ws, ws_layout(a, ws, mode)};
  if (mode == TT_LOSS_BACKWARD) {
    backward_part(a, p, b, kept);
  } else {
    b.take(a.loss, p.N);
    b.take(p.part, 2 * ((p.N + SUM_BLOCK - 1) / SUM_BLOCK));
    p.nll = a.loss;
  }
  return std::max<int64_t>(b.off, 256);
}

static bool misaligned(const void *p, int64_t size) { return (uintptr_t)p % size != 0; }

}  // namespace ttb

using namespace ttb;

extern "C" {

size_t tt_prefer_saved_size(const tt_prefer_desc *desc) {
  LossArgs a;
  PreferArgs p;
  return prefer_args(desc, nullptr, a, p) == TT_OK ? (size_t)prefer_saved(a, p, nullptr) : 0;
}

size_t tt_prefer_workspace_size(const tt_prefer_desc *desc, int mode) {
  LossArgs a;
  PreferArgs p;
  Kept kept;
  if (mode < TT_LOSS_FORWARD || mode > TT_LOSS_ONLY) return 0;
  return prefer_args(desc, nullptr, a, p) == TT_OK ? (size_t)prefer_ws(a, p, nullptr, mode, kept) : 0;
}

int tt_prefer_forward(const tt_prefer_desc *desc, const void *hidden, const void *weight,
                      const int64_t *targets, const int64_t *offsets, const float *reference_logps,
                      float *loss, float *ratios, void *saved, size_t saved_bytes, void *ws,
                      size_t ws_bytes, int32_t *dev_status, void *stream) {
  LossArgs a;
  PreferArgs p;
  Kept kept;
  const int rc = prefer_args(desc, weight, a, p);
  if (rc != TT_OK) return rc;
  if (!weight || !ws || !offsets) return TT_EINVAL;
  if (!loss && (p.P || p.reduction != TT_REDUCE_NONE)) return TT_EINVAL;
  if (p.N && (!hidden || !targets)) return TT_EINVAL;
  if (misaligned(weight, elem_size(a.dtype)) || misaligned(hidden, elem_size(a.dtype))) return TT_EINVAL;
  if (misaligned(saved, 256) || misaligned(ws, 256)) return TT_EWORKSPACE;
  if (saved && (size_t)prefer_saved(a, p, saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)prefer_ws(a, p, ws, saved ? TT_LOSS_FORWARD : TT_LOSS_ONLY, kept) > ws_bytes) return TT_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  a.hidden = hidden; a.tgt = targets; a.limit = offsets + 2 * p.P; a.status = dev_status;
  p.tgt = targets; p.off = offsets; p.ref = reference_logps; p.loss = loss; p.ratios = ratios;
  p.status = dev_status;
  if (p.N && loss_forward(a, s) != hipSuccess) return TT_EHIP;
  // (k_pack has cleared the ticket, which a loss without a reduction does not use)
  if (p.reduction != TT_REDUCE_NONE && p.N && !a.direct && p.P && p.P <= TICKETS) p.ticket = &a.sv.sc->ticket;
  if (p.P) tt_launch(K_ALIGN, k_prefer, dim3((unsigned)p.P), dim3(512), 0, s, p);
  if (p.reduction != TT_REDUCE_NONE && !p.ticket)
    tt_launch(K_ALIGN, k_prefer_sum, dim3(1), dim3(256), 0, s, p);
  return hipGetLastError() == hipSuccess ? TT_OK : TT_EHIP;
}

int tt_prefer_backward(const tt_prefer_desc *desc, const void *weight, const void *saved,
                       size_t saved_bytes, const float *grad_loss, void *grad_hidden, void *grad_weight,
                       void *ws, size_t ws_bytes, void *stream) {
  LossArgs a;
  PreferArgs p;
  Kept kept;
  const int rc = prefer_args(desc, weight, a, p);
  if (rc != TT_OK) return rc;
  if (!weight || !saved || !ws) return TT_EINVAL;
  if (!grad_loss && (p.P || p.reduction != TT_REDUCE_NONE)) return TT_EINVAL;
  if (misaligned(weight, elem_size(a.dtype)) || misaligned(grad_hidden, elem_size(a.dtype)) ||
      misaligned(grad_weight, elem_size(a.dtype)))
    return TT_EINVAL;
  if (misaligned(saved, 256) || misaligned(ws, 256)) return TT_EWORKSPACE;
  if ((size_t)prefer_saved(a, p, (void *)saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)prefer_ws(a, p, ws, TT_LOSS_BACKWARD, kept) > ws_bytes) return TT_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  a.coef = p.coef; a.seq = p.seq; a.pairs = p.P; a.of = p.reduction;
  a.up = grad_loss; a.dh = grad_hidden; a.dw = grad_weight;
  return backward_from(a, p, kept, s) == hipSuccess ? TT_OK : TT_EHIP;
}

size_t tt_policy_saved_size(const tt_policy_desc *desc) {
  LossArgs a;
  PolicyArgs p;
  return policy_args(desc, nullptr, a, p) == TT_OK ? (size_t)policy_saved(a, p, nullptr) : 0;
}

size_t tt_policy_workspace_size(const tt_policy_desc *desc, int mode) {
  LossArgs a;
  PolicyArgs p;
  Kept kept;
  if (mode < TT_LOSS_FORWARD || mode > TT_LOSS_ONLY) return 0;
  return policy_args(desc, nullptr, a, p) == TT_OK ? (size_t)policy_ws(a, p, nullptr, mode, kept) : 0;
}

int tt_policy_forward(const tt_policy_desc *desc, const void *hidden, const void *weight,
                      const int64_t *actions, const float *advantages, const float *old_logps,
                      const float *reference_logps, float *loss, float *logps, void *saved,
                      size_t saved_bytes, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
  LossArgs a;
  PolicyArgs p;
  Kept kept;
  const int rc = policy_args(desc, weight, a, p);
  if (rc != TT_OK) return rc;
  if (!weight || !ws || (p.N && (!hidden || !actions || !advantages))) return TT_EINVAL;
  if (p.N && p.kl != 0.0 && !reference_logps) return TT_EINVAL;
  if (!loss && (p.N || p.reduction != TT_REDUCE_NONE)) return TT_EINVAL;
  if (misaligned(weight, elem_size(a.dtype)) || misaligned(hidden, elem_size(a.dtype))) return TT_EINVAL;
  if (misaligned(saved, 256) || misaligned(ws, 256)) return TT_EWORKSPACE;
  if (saved && (size_t)policy_saved(a, p, saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)policy_ws(a, p, ws, saved ? TT_LOSS_FORWARD : TT_LOSS_ONLY, kept) > ws_bytes) return TT_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  a.hidden = hidden; a.tgt = actions; a.status = dev_status;
  p.tgt = actions; p.adv = advantages; p.old = old_logps; p.ref = reference_logps;
  p.loss = loss; p.logps = logps;
  if (p.N && loss_forward(a, s) != hipSuccess) return TT_EHIP;
  const bool none = p.reduction == TT_REDUCE_NONE;
  if (none || p.N > ONE_BLOCK) {
    const int64_t per = none ? 256 : SUM_BLOCK, blocks = (p.N + per - 1) / per;
    if (blocks) tt_launch(K_ALIGN, k_policy<256>, dim3((unsigned)blocks), dim3(256), 0, s, p, per);
    if (!none) tt_launch(K_ALIGN, k_policy_sum, dim3(1), dim3(256), 0, s, p, blocks);
  } else {
    tt_launch(K_ALIGN, k_policy<1024>, dim3(1), dim3(1024), 0, s, p, p.N);
  }
  return hipGetLastError() == hipSuccess ? TT_OK : TT_EHIP;
}

int tt_policy_backward(const tt_policy_desc *desc, const void *weight, const void *saved,
                       size_t saved_bytes, const float *grad_loss, void *grad_hidden, void *grad_weight,
                       void *ws, size_t ws_bytes, void *stream) {
  LossArgs a;
  PolicyArgs p;
  Kept kept;
  const int rc = policy_args(desc, weight, a, p);
  if (rc != TT_OK) return rc;
  if (!weight || !saved || !ws) return TT_EINVAL;
  if (!grad_loss && (p.N || p.reduction != TT_REDUCE_NONE)) return TT_EINVAL;
  if (misaligned(weight, elem_size(a.dtype)) || misaligned(grad_hidden, elem_size(a.dtype)) ||
      misaligned(grad_weight, elem_size(a.dtype)))
    return TT_EINVAL;
  if (misaligned(saved, 256) || misaligned(ws, 256)) return TT_EWORKSPACE;
  if ((size_t)policy_saved(a, p, (void *)saved) > saved_bytes) return TT_EWORKSPACE;
  if ((size_t)policy_ws(a, p, ws, TT_LOSS_BACKWARD, kept) > ws_bytes) return TT_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  a.coef = p.coef; a.of = p.reduction; a.all = a.sv.sc;
  a.up = grad_loss; a.dh = grad_hidden; a.dw = grad_weight;
  return backward_from(a, p, kept, s) == hipSuccess ? TT_OK : TT_EHIP;
}

}  // extern "C"
