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
    s *= exp_shift(m, n);
    m = n;
#pragma unroll
    for (int k = 0; k < N; ++k) s += exp_shift(v[k], m);
  }
  __device__ __forceinline__ void join(float m2, float s2) {
    const float n = fmaxf(m, m2);
    s = s * exp_shift(m, n) + s2 * exp_shift(m2, n);
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

// One workgroup a row: maximum, sum and the target's log-probability.
template <bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS) void kl_rows(LogitArgs a, const float *weights, RowStat *stat, float *logp,
                                                   float *lse) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ float red[2 * THREADS / 64];
  const int64_t r = blockIdx.x;
  const int64_t target = index_at(a.targets, r);
  if (target < 0 || target >= a.vocab || (weights && weights[r] == 0.f)) {
    if (threadIdx.x == 0) {
      if (stat) stat[r] = RowStat{0.f, 0.f, 0.0};
      if (logp) logp[r] = 0.f;
      if (lse) lse[r] = 0.f;
    }
    return;
  }
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  Online o;
  const int64_t vecs = a.vocab / E::N;
  int64_t i = threadIdx.x;
  for (; i + 3 * THREADS < vecs; i += 4 * THREADS) {
    uint4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = load16(x + (i + k * THREADS) * E::N);
    float v[4 * E::N];
#pragma unroll
    for (int k = 0; k < 4; ++k) E::unpack(w[k], v + k * E::N);
    o.add<4 * E::N>(v);
  }
  for (; i < vecs; i += THREADS) {
    float v[E::N];
    E::unpack(load16(x + i * E::N), v);
    o.add<E::N>(v);
  }
  i = vecs * E::N + threadIdx.x;
  if (i < a.vocab) {
    const float v = E::get(x[i]);
    o.add<1>(&v);
  }
  o = block_join<THREADS / 64>(o, red);
  if (threadIdx.x == 0) {
    const double log_total = log((double)o.s);
    const double lp = (double)E::get(x[target]) - (double)o.m - log_total;
    if (stat) stat[r] = RowStat{o.m, o.s, lp};
    if (logp) logp[r] = (float)lp;
    if (lse) lse[r] = (float)((double)o.m + log_total);
  }
}

// The policy loss of every row and its four sums, in one workgroup.
//   ratio = exp(logp - old), J = min(ratio a, clip(ratio) a)
//   KL estimate exp(d) - 1 - d, d = ref - logp
// The derivative by logp is -a ratio while the unclipped branch is the
// smaller, plus kl_coef (1 - exp(d)).
__global__ __launch_bounds__(1024) void kl_policy(LogitArgs a, PolicyArgs p, const RowStat *stat, RowGrad *grad) {
  __shared__ double red[16];
  double sum[4] = {};
  const double lo = 1.0 - p.clip_low, hi = 1.0 + p.clip_high;
  for (int64_t r = threadIdx.x; r < a.rows; r += 1024) {
    const int64_t target = index_at(a.targets, r);
    const float w = p.weights[r];
    if (target < 0 || target >= a.vocab || w == 0.f) {
      p.logp[r] = 0.f;
      grad[r] = RowGrad{0.f, 0.f, 0.f, 0};
      continue;
    }
    const RowStat st = stat[r];
    const double adv = p.advantages[r];
    const double ratio = p.old_logp ? exp(st.logp - (double)p.old_logp[r]) : 1.0;
    const double clipped = fmin(fmax(ratio, lo), hi);
    const bool active = ratio * adv <= clipped * adv;
    double kl = 0.0, dkl = 0.0;
    if (p.ref_logp) {
      const double d = (double)p.ref_logp[r] - st.logp;
      dkl = -expm1(d);
      kl = -dkl - d;
    }
    const double pg = active ? -ratio * adv : -clipped * adv;
    const double dlogp = (double)w * ((active ? -adv * ratio : 0.0) + p.kl_coef * dkl);
    sum[0] += (double)w * (pg + p.kl_coef * kl);
    sum[1] += (double)w * pg;
    sum[2] += (double)w * kl;
    sum[3] += active ? 0.0 : (double)w;
    p.logp[r] = (float)st.logp;
    grad[r] = RowGrad{st.max, (float)(-dlogp / (double)st.total), (float)(-dlogp * expm1(st.logp)), dlogp != 0.0};
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double t = block_sum<16>(sum[k], red);
    if (threadIdx.x == 0) p.stats[k] = (float)t;
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

// Sum of the log-probabilities of each sequence, one workgroup a pair, and
// the pair's loss and coefficient:
//   gain = sum logp - ref, m = beta (gain_chosen - gain_rejected)
//   loss = -(1 - s) log sigmoid(m) - s log sigmoid(-m)
//   d loss / d logp = +- beta (sigmoid(m) - (1 - s)) / pairs
__global__ __launch_bounds__(256) void kl_pairs(LogitArgs a, PreferenceArgs p, const RowStat *stat, double *coef) {
  __shared__ double red[4];
  const int64_t i = blockIdx.x;
  double gain[2];
  for (int side = 0; side < 2; ++side) {
    const int64_t s = i + side * p.pairs;
    int64_t lo, hi;
    sequence(p.offsets, s, a.rows, &lo, &hi);
    double t = 0.0;
    for (int64_t r = lo + threadIdx.x; r < hi; r += 256) t += stat[r].logp;
    gain[side] = block_sum<4>(t, red) - (double)p.ref_logp[s];
    if (threadIdx.x == 0) p.rewards[s] = (float)(p.beta * gain[side]);
  }
  if (threadIdx.x == 0) {
    const double m = p.beta * (gain[0] - gain[1]);
    const double q = exp(-fabs(m)), l = log1p(q);
    // softplus(-m) and softplus(m), and sigmoid(m), without overflow
    const double up = fmax(-m, 0.0) + l, down = fmax(m, 0.0) + l;
    const double sig = (m >= 0.0 ? 1.0 : q) / (1.0 + q);
    coef[2 * i] = (1.0 - p.smoothing) * up + p.smoothing * down;
    coef[2 * i + 1] = p.beta * (sig - (1.0 - p.smoothing)) / (double)p.pairs;
  }
}

// The mean loss (first workgroup) and every row's gradient coefficients.
__global__ __launch_bounds__(256) void kl_pair_rows(LogitArgs a, PreferenceArgs p, const RowStat *stat,
                                                    const double *coef, RowGrad *grad) {
  __shared__ double red[4];
  if (blockIdx.x == 0) {
    double t = 0.0;
    for (int64_t i = threadIdx.x; i < p.pairs; i += 256) t += coef[2 * i];
    t = block_sum<4>(t, red);
    if (threadIdx.x == 0) p.loss[0] = (float)(t / (double)p.pairs);
  }
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= a.rows) return;
  // the last sequence that starts at or before the row
  int64_t lo = 0, hi = 2 * p.pairs - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (index_at(p.offsets, mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  int64_t s0, s1;
  sequence(p.offsets, lo, a.rows, &s0, &s1);
  const int64_t target = index_at(a.targets, r);
  RowGrad g{0.f, 0.f, 0.f, 0};
  if (r >= s0 && r < s1 && target >= 0 && target < a.vocab) {
    const RowStat st = stat[r];
    const double d = lo < p.pairs ? coef[2 * lo + 1] : -coef[2 * (lo - p.pairs) + 1];
    g = RowGrad{st.max, (float)(-d / (double)st.total), (float)(-d * expm1(st.logp)), d != 0.0};
  }
  grad[r] = g;
}

// The gradient of the logits, element by element; a row without one gets
// zeros and is not read.
template <bool BF16>
__global__ __launch_bounds__(256) void kl_grad(LogitArgs a, const RowGrad *grad, void *dlogits, int64_t dld,
                                               int pieces) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  const int64_t r = blockIdx.x;
  const int piece = blockIdx.y;
  const RowGrad g = grad[r];
  const int64_t target = index_at(a.targets, r);
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  T *d = static_cast<T *>(dlogits) + r * dld;
  const int64_t vecs = (a.vocab + E::N - 1) / E::N;
  const int64_t v0 = vecs * piece / pieces, v1 = vecs * (piece + 1) / pieces;
  for (int64_t i = v0 + threadIdx.x; i < v1; i += 256) {
    const int64_t j = i * E::N;
    if (j + E::N <= a.vocab) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (g.live) {
        float v[E::N];
        E::unpack(load16(x + j), v);
#pragma unroll
        for (int k = 0; k < E::N; ++k) v[k] = j + k == target ? g.dt : g.c * exp_shift(v[k], g.max);
        w = E::pack(v);
      }
      store16(d + j, w);
    } else {
      for (int64_t k = j; k < a.vocab; ++k)
        d[k] = !g.live ? T(0) : E::put(k == target ? g.dt : g.c * exp_shift(E::get(x[k]), g.max));
    }
  }
}

// ------------------------------------------------------------- launchers

namespace {

hipError_t rows_launch(const LogitArgs &a, bool bf16, const float *weights, RowStat *stat, float *logp, float *lse,
                       hipStream_t s) {
  const dim3 g((unsigned)a.rows);
  if (bf16) hipLaunchKernelGGL((kl_rows<true, 512>), g, dim3(512), 0, s, a, weights, stat, logp, lse);
  else hipLaunchKernelGGL((kl_rows<false, 512>), g, dim3(512), 0, s, a, weights, stat, logp, lse);
  return hipGetLastError();
}

hipError_t grad_launch(const LogitArgs &a, bool bf16, const RowGrad *grad, void *dlogits, int64_t dld,
                       hipStream_t s) {
  const int pieces = (int)std::max<int64_t>(1, std::min<int64_t>(a.vocab / 8192, 64));
  const dim3 g((unsigned)a.rows, (unsigned)pieces);
  if (bf16) hipLaunchKernelGGL(kl_grad<true>, g, dim3(256), 0, s, a, grad, dlogits, dld, pieces);
  else hipLaunchKernelGGL(kl_grad<false>, g, dim3(256), 0, s, a, grad, dlogits, dld, pieces);
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
  l.stat = 0;
  l.grad = up256(sizeof(RowStat) * (size_t)rows);
  l.total = l.grad + up256(sizeof(RowGrad) * (size_t)std::max<int64_t>(rows, 1));
  return l;
}

hipError_t launch_policy(const LogitArgs &a, const PolicyArgs &p, bool bf16, void *dlogits, int64_t dld, char *ws,
                         hipStream_t s) {
  const PolicyLayout l = policy_layout(a.rows);
  RowStat *stat = reinterpret_cast<RowStat *>(ws + l.stat);
  RowGrad *grad = reinterpret_cast<RowGrad *>(ws + l.grad);
  hipError_t e = hipSuccess;
  if (a.rows > 0) e = rows_launch(a, bf16, p.weights, stat, nullptr, nullptr, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kl_policy, dim3(1), dim3(1024), 0, s, a, p, stat, grad);
  e = hipGetLastError();
  if (e != hipSuccess || a.rows == 0) return e;
  return grad_launch(a, bf16, grad, dlogits, dld, s);
}

PreferenceLayout preference_layout(int64_t rows, int64_t pairs) {
  PreferenceLayout l{};
  l.stat = 0;
  l.grad = up256(sizeof(RowStat) * (size_t)rows);
  l.coef = l.grad + up256(sizeof(RowGrad) * (size_t)rows);
  l.total = l.coef + up256(2 * sizeof(double) * (size_t)pairs);
  return l;
}

hipError_t launch_preference(const LogitArgs &a, const PreferenceArgs &p, bool bf16, void *dlogits, int64_t dld,
                             char *ws, hipStream_t s) {
  const PreferenceLayout l = preference_layout(a.rows, p.pairs);
  RowStat *stat = reinterpret_cast<RowStat *>(ws + l.stat);
  RowGrad *grad = reinterpret_cast<RowGrad *>(ws + l.grad);
  double *coef = reinterpret_cast<double *>(ws + l.coef);
  hipError_t e = hipSuccess;
  if (a.rows > 0) e = rows_launch(a, bf16, nullptr, stat, nullptr, nullptr, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kl_pairs, dim3((unsigned)p.pairs), dim3(256), 0, s, a, p, stat, coef);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned blocks = (unsigned)std::max<int64_t>(1, (a.rows + 255) / 256);
  hipLaunchKernelGGL(kl_pair_rows, dim3(blocks), dim3(256), 0, s, a, p, stat, coef, grad);
  if ((e = hipGetLastError()) != hipSuccess || a.rows == 0) return e;
  return grad_launch(a, bf16, grad, dlogits, dld, s);
}

}  // namespace muon
