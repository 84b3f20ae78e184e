// Losses over rows of logits, on gfx950: the token log-probability, the
// clipped policy loss with a KL term, and the preference loss of paired
// sequences, each with the gradient of the logits.
//
//   lse_r  = log sum_j exp(x_rj)            (shifted by the row's maximum)
//   logp_r = x_r,target - lse_r
//   d loss / d x_rj = dlogp_r ([j = target] - exp(x_rj - lse_r))
//
// where dlogp_r is the loss's derivative by the row's log-probability.  A row
// whose target is outside the vocabulary has none: it is not read, its
// log-probability and its gradient are 0.  Row sums are fp32 a thread (at
// most a few hundred terms) joined in a fixed tree; everything a row has one
// of is computed in fp64.  No float atomics: results are bitwise the same
// from run to run.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "devops.hpp"
#include "train_ops.hpp"

namespace muon {

using namespace dev;

namespace {

// Running maximum and sum of exp(x - max) of one thread's elements.
struct Online {
  float m = kLowest, s = 0.f;
  template <int N>
  __device__ __forceinline__ void add(const float *v) {
    float t = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k) t = fmaxf(t, v[k]);
    const float n = fmaxf(m, t);
    s *= exp_term(m, n);
    m = n;
#pragma unroll
    for (int k = 0; k < N; ++k) s += exp_term(v[k], m);
  }
  __device__ __forceinline__ void join(float m2, float s2) {
    const float n = fmaxf(m, m2);
    s = s * exp_term(m, n) + s2 * exp_term(m2, n);
    m = n;
  }
};

template <int WAVES>
__device__ __forceinline__ Online block_join(Online o, float *red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const float m = __shfl_xor(o.m, d), s = __shfl_xor(o.s, d);
    o.join(m, s);
  }
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    red[2 * w] = o.m;
    red[2 * w + 1] = o.s;
  }
  __syncthreads();
  Online t;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) t.join(red[2 * i], red[2 * i + 1]);
  return t;
}

}  // namespace

// One workgroup a row: maximum, sum and the target's log-probability.  HBM-
// bound.  grad (may be NULL) starts as that of a row without a gradient.
template <bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void kl_rows(LogitArgs a, RowStat *stat, RowGrad *grad, float *logp,
                                                   float *lse) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ float red[2 * THREADS / 64];
  const int64_t r = blockIdx.x;
  const int64_t target = index_at(a.targets, r);
  if (grad && threadIdx.x == 0) grad[r] = RowGrad{0.f, 0.f, 0.f, 0};
  if (target < 0 || target >= a.vocab) {
    if (threadIdx.x == 0) {
      if (stat) stat[r] = RowStat{0.f, 0.f, 0.0, 0.0};
      if (logp) logp[r] = 0.f;
      if (lse) lse[r] = 0.f;
    }
    return;
  }
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  const Row<BF16> row(x, a.vocab);
  constexpr int UNROLL = 4;
  Online o;
  int i = threadIdx.x;
  for (; i + (UNROLL - 1) * THREADS < row.vecs; i += UNROLL * THREADS) {
    uint4 w[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) w[k] = load16(x + row.col(i + k * THREADS));
#pragma unroll
    for (int k = 0; k < UNROLL; k += 2) {
      float v[2 * E::N];
      E::unpack(w[k], v);
      E::unpack(w[k + 1], v + E::N);
      o.add<2 * E::N>(v);
    }
  }
  for (; i < row.vecs; i += THREADS) {
    float v[E::N];
    E::unpack(load16(x + row.col(i)), v);
    o.add<E::N>(v);
  }
  if ((int)threadIdx.x < row.singles()) {
    const float v = E::get(x[row.single(threadIdx.x)]);
    o.add<1>(&v);
  }
  o = block_join<THREADS / 64>(o, red);
  if (threadIdx.x == 0) {
    const double log_total = log((double)o.s);
    const double lp = (double)E::get(x[target]) - (double)o.m - log_total;
    if (stat) stat[r] = RowStat{o.m, o.s, lp, expm1(lp)};
    if (logp) logp[r] = (float)lp;
    if (lse) lse[r] = (float)((double)o.m + log_total);
  }
}

namespace {

// Vectors of a row that a thread of the policy kernel keeps: the first ones in
// LDS (64 KB a workgroup of 1024, two of them on a CU), the others in registers.
constexpr int KEEP_LDS = 4, KEEP_REGS = 2, KEEP = KEEP_LDS + KEEP_REGS;
// Loads of the rest under way at a time.
constexpr int AHEAD = 2;

}  // namespace

// The policy loss and its gradient, one workgroup a row:
//   ratio = exp(logp - old), J = min(ratio a, clip(ratio) a)
//   KL estimate exp(d) - 1 - d, d = ref - logp
// The derivative by logp is -a ratio while the unclipped branch is the
// smaller, plus kl_coef (1 - exp(d)).
//
// HBM-bound, one read and one write of a row.  The first KEEP vectors of each
// thread stay on the CU between the row's sum and its gradient, in LDS and
// registers; the rest is read again, from the caches: with two workgroups of
// 1024 threads on a CU, 512 rows of the chip are under way (128 MB at 131072
// bf16 columns), which the memory-side cache holds, the more so as the
// gradient is streamed past it.  Measured over 1.2 GB of logits, in TB/s of
// one read and one write (a large copy: 5.15):
//                                     bf16 131072  50257  32000  fp32 50257
//   this                                     5.0    5.9    5.6         5.3
//   4 vectors in registers, none in LDS      4.9    5.4    5.5         4.9
//   whole rows in registers, half the waves  4.2    4.2    4.2         4.2
//   nothing kept                             4.5    4.7    4.8         4.6
//   nothing kept, ordinary stores            3.6    4.5    4.7         3.6
// The row's own arithmetic, in fp64, is two function calls deep in one wave:
// lanes 0 to 2 share a call of expm1.
template <bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void kl_policy(LogitArgs a, PolicyArgs p, void *dlogits, int64_t dld,
                                                        double *terms) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ float red[2 * THREADS / 64];
  __shared__ float coef[2];
  __shared__ uint4 held[KEEP_LDS][THREADS];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t target = index_at(a.targets, r);
  const float w = p.weights[r];
  T *d = static_cast<T *>(dlogits) + r * dld;
  if (target < 0 || target >= a.vocab || w == 0.f) {
    const Row<BF16> out(d, a.vocab);
    for (int i = tid; i < out.vecs; i += THREADS) stream16(d + out.col(i), make_uint4(0, 0, 0, 0));
    if (tid < out.singles()) d[out.single(tid)] = T(0);
    if (tid < 4) terms[4 * r + tid] = 0.0;
    if (tid == 0) p.logp[r] = 0.f;
    return;
  }
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  const Row<BF16> row(x, a.vocab);
  uint4 keep[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = tid + k * THREADS;
    keep[k] = i < row.vecs ? load16(x + row.col(i)) : E::none();
  }
  const bool lone = tid < row.singles();
  const float single = lone ? E::get(x[row.single(tid)]) : -INFINITY;
  const float at_target = E::get(x[target]);
  Online o;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    if (k * THREADS < row.vecs) {
      float v[E::N];
      E::unpack(keep[k], v);
      o.add<E::N>(v);
      if (k < KEEP_LDS) held[k][tid] = keep[k];  // read back by this thread alone
    }
  }
  int far = tid + KEEP * THREADS;
  for (; far + (AHEAD - 1) * THREADS < row.vecs; far += AHEAD * THREADS) {
    uint4 in[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) in[k] = load16(x + row.col(far + k * THREADS));
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      float v[E::N];
      E::unpack(in[k], v);
      o.add<E::N>(v);
    }
  }
  for (; far < row.vecs; far += THREADS) {
    float v[E::N];
    E::unpack(load16(x + row.col(far)), v);
    o.add<E::N>(v);
  }
  o.add<1>(&single);
  o = block_join<THREADS / 64>(o, red);
  if (tid < 64) {
    const double logp = (double)at_target - (double)o.m - log((double)o.s);
    // lane 0: the ratio, lane 1: the KL term, lane 2: the target's own share
    double arg = 0.0;
    if (tid == 0 && p.old_logp) arg = logp - (double)p.old_logp[r];
    if (tid == 1 && p.ref_logp) arg = (double)p.ref_logp[r] - logp;
    if (tid == 2) arg = logp;
    const double em1 = expm1(arg);
    const double ratio = 1.0 + shfl_f64(em1, 0), ed = shfl_f64(em1, 1), share = shfl_f64(em1, 2);
    const double kl = ed - shfl_f64(arg, 1);
    const double adv = p.advantages[r];
    const double clipped = fmin(fmax(ratio, 1.0 - p.clip_low), 1.0 + p.clip_high);
    const bool active = !(ratio * adv > clipped * adv);  // a NaN stays one
    const double pg = active ? -ratio * adv : -clipped * adv;
    const double dlogp = (double)w * ((active ? -adv * ratio : 0.0) - p.kl_coef * ed);
    if (tid == 0) {
      coef[0] = (float)(-dlogp / (double)o.s);
      coef[1] = (float)(-dlogp * share);
      p.logp[r] = (float)logp;
      terms[4 * r] = (double)w * (pg + p.kl_coef * kl);
      terms[4 * r + 1] = (double)w * pg;
      terms[4 * r + 2] = (double)w * kl;
      terms[4 * r + 3] = active ? 0.0 : (double)w;
    }
  }
  __syncthreads();
  // the vectors are unpacked a second time: kept unpacked over the sum, bf16
  // ones would take twice the registers
#pragma unroll
  for (int k = KEEP_LDS; k < KEEP; ++k)
    asm volatile("" : "+v"(keep[k].x), "+v"(keep[k].y), "+v"(keep[k].z), "+v"(keep[k].w));
  const float c = coef[0], dt = coef[1], m = o.m;
  auto grad = [&](uint4 in, int i) {
    float v[E::N];
    E::unpack(in, v);
#pragma unroll
    for (int j = 0; j < E::N; ++j) v[j] = c * exp_shift(v[j], m);
    stream16(d + row.col(i), E::pack(v));
  };
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = tid + k * THREADS;
    if (i < row.vecs) grad(k < KEEP_LDS ? held[k][tid] : keep[k], i);
  }
  far = tid + KEEP * THREADS;
  for (; far + (AHEAD - 1) * THREADS < row.vecs; far += AHEAD * THREADS) {
    uint4 in[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) in[k] = load16(x + row.col(far + k * THREADS));
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) grad(in[k], far + k * THREADS);
  }
  for (; far < row.vecs; far += THREADS) grad(load16(x + row.col(far)), far);
  if (lone) d[row.single(tid)] = E::put(c * exp_shift(single, m));
  // the target's own element, by the thread that wrote over it
  const int at = (int)target - row.head;
  const bool in_vec = at >= 0 && at / E::N < row.vecs;
  if (in_vec ? at / E::N % THREADS == tid : lone && row.single(tid) == (uint32_t)target) d[target] = E::put(dt);
}

// The four sums over the rows, in a fixed order.
__global__ __launch_bounds__(1024) void kl_policy_sum(const double *terms, int64_t rows, float *stats) {
  __shared__ double red[16];
  double sum[4] = {};
  for (int64_t r = threadIdx.x; r < rows; r += 1024) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] += terms[4 * r + k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double t = block_sum<16>(sum[k], red);
    if (threadIdx.x == 0) stats[k] = (float)t;
  }
}

namespace {

// Sequence bounds as the kernels use them: whatever the offsets hold, rows
// outside [0, rows) are never touched.
__device__ __forceinline__ void sequence(const IndexVec &off, int64_t s, int64_t rows, int64_t *lo, int64_t *hi) {
  *lo = min(max(index_at(off, s), (int64_t)0), rows);
  *hi = min(max(index_at(off, s + 1), *lo), rows);
}

}  // namespace

// Sum of the log-probabilities of each sequence, and from them the pair's
// loss and its rows' gradient coefficients; one workgroup a pair, half of it
// a sequence:
//   gain = sum logp - ref, m = beta (gain_chosen - gain_rejected)
//   loss = -(1 - s) log sigmoid(m) - s log sigmoid(-m)
//   d loss / d logp = +- beta (sigmoid(m) - (1 - s)) / pairs
// Bound by the latency of its few dependent loads.
__global__ __launch_bounds__(1024) void kl_pairs(LogitArgs a, PreferenceArgs p, const RowStat *stat, RowGrad *grad,
                                                 double *losses) {
  __shared__ double red[16];
  const int64_t i = blockIdx.x;
  const int side = threadIdx.x >> 9, tid = threadIdx.x & 511;
  const int64_t s = i + side * p.pairs;
  int64_t lo, hi;
  sequence(p.offsets, s, a.rows, &lo, &hi);
  const double ref[2] = {(double)p.ref_logp[i], (double)p.ref_logp[i + p.pairs]};
  double t = 0.0;
  for (int64_t r = lo + tid; r < hi; r += 512) t += stat[r].logp;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) t += shfl_xor_f64(t, k);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = t;
  __syncthreads();
  double gain[2] = {};
#pragma unroll
  for (int w = 0; w < 16; ++w) gain[w >> 3] += red[w];
  gain[0] -= ref[0];
  gain[1] -= ref[1];
  const double m = p.beta * (gain[0] - gain[1]);
  const double q = exp(-fabs(m));
  const double sig = (m >= 0.0 ? 1.0 : q) / (1.0 + q);
  const double chosen = p.beta * (sig - (1.0 - p.smoothing)) / (double)p.pairs;
  const double d = side ? -chosen : chosen;
  for (int64_t r = lo + tid; r < hi; r += 512) {
    const int64_t target = index_at(a.targets, r);
    if (target < 0 || target >= a.vocab) continue;
    const RowStat st = stat[r];
    grad[r] = RowGrad{st.max, (float)(-d / (double)st.total), (float)(-d * st.share), d != 0.0};
  }
  if (tid == 0) p.rewards[s] = (float)(p.beta * (side ? gain[1] : gain[0]));
  if (threadIdx.x == 0) {
    // softplus(-m) and softplus(m) without overflow
    const double l = log1p(q);
    losses[i] = (1.0 - p.smoothing) * (fmax(-m, 0.0) + l) + p.smoothing * (fmax(m, 0.0) + l);
  }
}

// The mean of the pairs' losses, by one workgroup of the gradient kernel.
__device__ __forceinline__ void mean_loss(const double *losses, int64_t pairs, float *loss) {
  __shared__ double red[4];
  double t = 0.0;
  for (int64_t i = threadIdx.x; i < pairs; i += 256) t += losses[i];
  t = block_sum<4>(t, red);
  if (threadIdx.x == 0) *loss = (float)(t / (double)pairs);
}

// The gradient of the logits, element by element; a row without one gets
// zeros and is not read.  The rows are taken from the last to the first: the
// last ones that the row sums read are still in the memory-side cache.
template <bool BF16>
__global__ __launch_bounds__(256) void kl_grad(LogitArgs a, const RowGrad *grad, void *dlogits, int64_t dld,
                                               int pieces, const double *losses, int64_t pairs, float *loss) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  if (blockIdx.x == 0) mean_loss(losses, pairs, loss);
  if (a.rows == 0) return;
  const int64_t r = a.rows - 1 - blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces;
  const RowGrad g = grad[r];
  const int64_t target = index_at(a.targets, r);
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  T *d = static_cast<T *>(dlogits) + r * dld;
  const Row<BF16> row(g.live ? x : d, a.vocab);
  const int v0 = (int)((int64_t)row.vecs * piece / pieces), v1 = (int)((int64_t)row.vecs * (piece + 1) / pieces);
  if (!g.live) {
    for (int i = v0 + threadIdx.x; i < v1; i += 256) stream16(d + row.col(i), make_uint4(0, 0, 0, 0));
    if (piece == 0 && (int)threadIdx.x < row.singles()) d[row.single(threadIdx.x)] = T(0);
    return;
  }
#pragma unroll 4
  for (int i = v0 + threadIdx.x; i < v1; i += 256) {
    float v[E::N];
    E::unpack(load16(x + row.col(i)), v);
#pragma unroll
    for (int k = 0; k < E::N; ++k) v[k] = g.c * exp_shift(v[k], g.max);
    const int at = (int)target - (int)row.col(i);
    if (at >= 0 && at < E::N) {
#pragma unroll
      for (int k = 0; k < E::N; ++k) v[k] = k == at ? g.dt : v[k];
    }
    stream16(d + row.col(i), E::pack(v));
  }
  if (piece == 0 && (int)threadIdx.x < row.singles()) {
    const int j = row.single(threadIdx.x);
    d[j] = E::put(j == target ? g.dt : g.c * exp_shift(E::get(x[j]), g.max));
  }
}

// ------------------------------------------------------------- launchers

namespace {

hipError_t rows_launch(const LogitArgs &a, bool bf16, RowStat *stat, RowGrad *grad, float *logp, float *lse,
                       hipStream_t s) {
  const dim3 g((unsigned)a.rows);
  // 256 threads where 512 would have fewer than two rounds of loads: 20000 x
  // 4096 bf16 take 35 us instead of 56, 4000 x 1000 7 instead of 11; from
  // there on 512 are as fast or faster (100 x 50257 fp32 6.7 against 8.3)
  const bool small = a.vocab <= 4096 * (bf16 ? 2 : 1);
  if (bf16 && small) hipLaunchKernelGGL((kl_rows<true, 256>), g, dim3(256), 0, s, a, stat, grad, logp, lse);
  else if (bf16) hipLaunchKernelGGL((kl_rows<true, 512>), g, dim3(512), 0, s, a, stat, grad, logp, lse);
  else if (small) hipLaunchKernelGGL((kl_rows<false, 256>), g, dim3(256), 0, s, a, stat, grad, logp, lse);
  else hipLaunchKernelGGL((kl_rows<false, 512>), g, dim3(512), 0, s, a, stat, grad, logp, lse);
  return hipGetLastError();
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

hipError_t launch_token_logprob(const LogitArgs &a, bool bf16, float *logp, float *lse, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return rows_launch(a, bf16, nullptr, nullptr, logp, lse, s);
}

PolicyLayout policy_layout(int64_t rows) {
  PolicyLayout l{};
  l.terms = 0;
  l.total = up256(4 * sizeof(double) * (size_t)std::max<int64_t>(rows, 1));
  return l;
}

namespace {

template <bool BF16>
void policy_launch(const LogitArgs &a, const PolicyArgs &p, void *dlogits, int64_t dld, double *terms, hipStream_t s) {
  const dim3 g((unsigned)a.rows);
  const int64_t vecs = a.vocab / Elem<BF16>::N;
  if (vecs <= 256 * KEEP) hipLaunchKernelGGL((kl_policy<BF16, 256>), g, dim3(256), 0, s, a, p, dlogits, dld, terms);
  else hipLaunchKernelGGL((kl_policy<BF16, 1024>), g, dim3(1024), 0, s, a, p, dlogits, dld, terms);
}

}  // namespace

hipError_t launch_policy(const LogitArgs &a, const PolicyArgs &p, bool bf16, void *dlogits, int64_t dld, char *ws,
                         hipStream_t s) {
  const PolicyLayout l = policy_layout(a.rows);
  double *terms = reinterpret_cast<double *>(ws + l.terms);
  if (a.rows > 0) {
    if (bf16) policy_launch<true>(a, p, dlogits, dld, terms, s);
    else policy_launch<false>(a, p, dlogits, dld, terms, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kl_policy_sum, dim3(1), dim3(1024), 0, s, terms, a.rows, p.stats);
  return hipGetLastError();
}

PreferenceLayout preference_layout(int64_t rows, int64_t pairs) {
  PreferenceLayout l{};
  l.stat = 0;
  l.grad = up256(sizeof(RowStat) * (size_t)rows);
  l.losses = l.grad + up256(sizeof(RowGrad) * (size_t)rows);
  l.total = l.losses + up256(sizeof(double) * (size_t)pairs);
  return l;
}

hipError_t launch_preference(const LogitArgs &a, const PreferenceArgs &p, bool bf16, void *dlogits, int64_t dld,
                             char *ws, hipStream_t s) {
  const PreferenceLayout l = preference_layout(a.rows, p.pairs);
  RowStat *stat = reinterpret_cast<RowStat *>(ws + l.stat);
  RowGrad *grad = reinterpret_cast<RowGrad *>(ws + l.grad);
  double *losses = reinterpret_cast<double *>(ws + l.losses);
  hipError_t e = hipSuccess;
  if (a.rows > 0) e = rows_launch(a, bf16, stat, grad, nullptr, nullptr, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kl_pairs, dim3((unsigned)p.pairs), dim3(1024), 0, s, a, p, stat, grad, losses);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // pieces of a row: 8192 elements or more, and a grid that stays in range
  int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(a.vocab / 8192, 64));
  if (a.rows > 0) pieces = std::max<int64_t>(1, std::min(pieces, (((int64_t)1 << 31) - 1) / a.rows));
  const dim3 g((unsigned)std::max<int64_t>(1, a.rows * pieces));
  if (bf16) hipLaunchKernelGGL(kl_grad<true>, g, dim3(256), 0, s, a, grad, dlogits, dld, (int)pieces, losses, p.pairs, p.loss);
  else hipLaunchKernelGGL(kl_grad<false>, g, dim3(256), 0, s, a, grad, dlogits, dld, (int)pieces, losses, p.pairs, p.loss);
  return hipGetLastError();
}

}  // namespace muon
