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
// log-probability and its gradient are 0.  Row sums are fp32 a thread, joined
// in a fixed tree.  A thread has up to 64 terms in short rows and vocab / 512
// or fewer in long ones, and each addition rounds by at most 2^-24: 131072
// columns are off by at most 2^-16 (the largest vocabulary, 2^29, by 2^-4 if
// all its roundings had one sign).  Everything a row has one of is computed in
// fp64.  No float atomics: results are bitwise the same from run to run.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "devops.hpp"
#include "train_ops.hpp"

namespace muon {

using namespace dev;

namespace {

// Running maximum and sum of exp(x - max) of one thread's elements.  (Which
// products are fused is spelled out, so that the same order gives the same
// bits in every kernel.)
struct Online {
  float m = kLowest, s = 0.f;
  template <int N>
  __device__ __forceinline__ void add(const float *v) {
    float t = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k) t = fmaxf(t, v[k]);
    const float n = fmaxf(m, t);
    s = fmaf(s, exp_term(m, n), exp_term(v[0], n));
    m = n;
#pragma unroll
    for (int k = 1; k < N; ++k) s += exp_term(v[k], m);
  }
  // symmetric in its halves: lanes that join the same two get the same bits
  __device__ __forceinline__ void join(float m2, float s2) {
#pragma clang fp contract(off)
    const float n = fmaxf(m, m2);
    const float mine = s * exp_term(m, n), other = s2 * exp_term(m2, n);
    s = mine + other;
    m = n;
  }
};

__device__ __forceinline__ Online wave_join(Online o) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const float m = __shfl_xor(o.m, d), s = __shfl_xor(o.s, d);
    o.join(m, s);
  }
  return o;
}

template <int WAVES>
__device__ __forceinline__ Online block_join(Online o, float *red) {
  o = wave_join(o);
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

// c v, where a factor of 0 leaves nothing of an infinite value (a target of
// probability 0); NaN stays NaN.
__device__ __forceinline__ double times(double c, double v) { return c == 0.0 && fabs(v) == INFINITY ? 0.0 : c * v; }

// Maximum and sum of a row's vectors [v0, v1), and of its single elements if
// asked for, by a workgroup; every thread gets them.
template <bool BF16, int THREADS, int UNROLL = 4>
__device__ __forceinline__ Online row_online(const typename Elem<BF16>::type *x, const Row<BF16> &row, int v0, int v1,
                                             bool singles, float *red) {
  typedef Elem<BF16> E;
  Online o;
  int i = v0 + threadIdx.x;
  for (; i + (UNROLL - 1) * THREADS < v1; i += UNROLL * THREADS) {
    uint4 w[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) w[k] = load16(x + row.col(i + k * THREADS));
#pragma unroll
    for (int k = 0; k < UNROLL; k += 2) {
      float v[2 * E::N];
      E::unpack(w[k], v);
      E::unpack(w[k + 1], v + E::N);
      o.template add<2 * E::N>(v);
    }
  }
  for (; i < v1; i += THREADS) {
    float v[E::N];
    E::unpack(load16(x + row.col(i)), v);
    o.template add<E::N>(v);
  }
  if (singles && (int)threadIdx.x < row.singles()) {
    const float v = E::get(x[row.single(threadIdx.x)]);
    o.template add<1>(&v);
  }
  return block_join<THREADS / 64>(o, red);
}
template <bool BF16, int THREADS, int UNROLL = 4>
__device__ __forceinline__ Online row_online(const typename Elem<BF16>::type *x, int64_t vocab, float *red) {
  const Row<BF16> row(x, vocab);
  return row_online<BF16, THREADS, UNROLL>(x, row, 0, row.vecs, true, red);
}

}  // namespace

// One workgroup a row: maximum, sum and the target's log-probability.  HBM-
// bound (4093 x 50257 fp32: 112 us, 5.9 TB/s), unless rows are few: an element
// costs a wave about 44 cycles, so a row of 131072 on one CU takes 9 us (32
// rows: 9.2 us), and there is no workspace through which CUs could share it.
// grad (may be NULL) starts as that of a row without a gradient.
template <bool BF16, int THREADS, int UNROLL>
__global__ __launch_bounds__(THREADS, UNROLL > 4 ? 4 : 8) void kl_rows(LogitArgs a, RowStat *stat, RowGrad *grad,
                                                                       float *logp, float *lse) {
  typedef Elem<BF16> E;
  __shared__ float red[2 * THREADS / 64];
  const int64_t r = a.row0 + blockIdx.x;
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
  const typename E::type *x = static_cast<const typename E::type *>(a.logits) + r * a.ld;
  const float at_target = E::get(x[target]);
  const Online o = row_online<BF16, THREADS, UNROLL>(x, a.vocab, red);
  if (threadIdx.x == 0) {
    const double log_total = log((double)o.s);
    const double lp = (double)at_target - (double)o.m - log_total;
    if (stat) stat[r] = RowStat{o.m, o.s, lp, expm1(lp)};
    if (logp) logp[r] = (float)lp;
    if (lse) lse[r] = (float)((double)o.m + log_total);
  }
}

namespace {

// A short row in the registers of one wave: VECS 16-byte vectors a lane, and
// up to two of the single elements (fewer than 80) at the row's ends.
template <bool BF16, int VECS>
struct ShortRow {
  typedef Elem<BF16> E;
  uint4 in[VECS];
  float lone[2];
  __device__ __forceinline__ ShortRow(const typename E::type *x, const Row<BF16> &row) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < VECS; ++k) in[k] = lane + 64 * k < row.vecs ? load16(x + row.col(lane + 64 * k)) : E::none();
#pragma unroll
    for (int k = 0; k < 2; ++k) lone[k] = lane + 64 * k < row.singles() ? E::get(x[row.single(lane + 64 * k)]) : -INFINITY;
  }
  __device__ __forceinline__ Online sum() const {
    Online o;
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      float v[E::N];
      E::unpack(in[k], v);
      o.template add<E::N>(v);
    }
    o.template add<2>(lone);
    return wave_join(o);
  }
};

}  // namespace

// Short rows, a wave each: no barrier, and the row's own arithmetic of one wave
// runs beside the others' loads.  Bound by the latency of target, row and join
// (8192 x 1000 bf16: 7.7 us, the policy loss's 13); two to four rows a wave,
// whose fp64 functions are then called once, take as long.
template <bool BF16, int VECS>
__global__ __launch_bounds__(256) void kl_rows_short(LogitArgs a, RowStat *stat, RowGrad *grad, float *logp, float *lse) {
  typedef Elem<BF16> E;
  const int lane = threadIdx.x & 63;
  const int64_t r = a.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  const int64_t target = index_at(a.targets, r);
  if (grad && lane == 0) grad[r] = RowGrad{0.f, 0.f, 0.f, 0};
  if (target < 0 || target >= a.vocab) {
    if (lane == 0) {
      if (stat) stat[r] = RowStat{0.f, 0.f, 0.0, 0.0};
      if (logp) logp[r] = 0.f;
      if (lse) lse[r] = 0.f;
    }
    return;
  }
  const typename E::type *x = static_cast<const typename E::type *>(a.logits) + r * a.ld;
  const float at_target = E::get(x[target]);
  const Row<BF16> row(x, a.vocab);
  const Online o = ShortRow<BF16, VECS>(x, row).sum();
  if (lane == 0) {
    const double log_total = log((double)o.s);
    const double lp = (double)at_target - (double)o.m - log_total;
    if (stat) stat[r] = RowStat{o.m, o.s, lp, expm1(lp)};
    if (logp) logp[r] = (float)lp;
    if (lse) lse[r] = (float)((double)o.m + log_total);
  }
}

namespace {

// Vectors of a row that a thread of the policy kernel keeps: the first ones in
// LDS (64 KB a workgroup of 1024, two of them on a CU), the others in registers.
constexpr int KEEP_LDS = 4, KEEP_REGS = 2, KEEP = KEEP_LDS + KEEP_REGS;
// The policy loss of up to FEW_ROWS rows of at least FEW_ROW 16-byte vectors is
// computed in pieces: at most FEW_GROUPS workgroups, FEW_VECS vectors or more
// each.  Kernel time in us, in pieces and one workgroup a row: 8 x 50257 fp32
// (12564 vectors) 9.3 14.2; 4000 vectors (32000 bf16) either way, 61 rows 10.8
// 11.5, 127 rows 13.3 12.5; 20 x 8192 bf16 (1024) 9.4 7.5.  Call time, 131072
// bf16 columns: 8 rows 15.6 21.4, 64 15.8 22.8, 128 22.7 23.7, 250 38 33.
constexpr int FEW_ROWS = 128, FEW_ROW = 8192, FEW_GROUPS = 1024, FEW_VECS = 512;
// Workgroups that add up the rows' terms, at most; one for every SUM_ROWS rows.
constexpr int SUM_GROUPS = 256, SUM_ROWS = 1024;
// Loads of the rest under way at a time.
constexpr int AHEAD = 2;

}  // namespace

namespace {

// What a policy row has besides its logits: lane 0 holds the old log-
// probability, lane 1 the reference's.
struct PolicyRow {
  float weight, at_target, other, advantage;
};
struct PolicyCoef {
  float c, dt;  // d x_j = c exp(x_j - max) away from the target, dt at the target
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs &p, int64_t r, float weight, float at_target) {
  const int lane = threadIdx.x & 63;
  PolicyRow q{weight, at_target, 0.f, p.advantages[r]};
  if (lane == 0 && p.old_logp) q.other = p.old_logp[r];
  if (lane == 1 && p.ref_logp) q.other = p.ref_logp[r];
  return q;
}

// A row's loss and derivative, by one wave in fp64: its lanes 0 to 2
// share a call of expm1.  Lane 0 writes logp and the four terms if asked to.
__device__ __forceinline__ PolicyCoef policy_coef(const PolicyArgs &p, const PolicyRow &q, Online o, int64_t r,
                                                  int64_t rows, bool write, double *terms) {
  const int lane = threadIdx.x & 63;
  const double logp = (double)q.at_target - (double)o.m - log((double)o.s);
  // lane 0: the ratio (1 without old_logp, if there is a logp at all), lane 1:
  // the KL term, lane 2: the target's own share
  double arg = 0.0;
  if (lane == 0) arg = p.old_logp ? logp - (double)q.other : logp != logp ? logp : 0.0;
  if (lane == 1 && p.ref_logp) arg = (double)q.other - logp;
  if (lane == 2) arg = logp;
  const double em1 = expm1(arg);
  const double ratio = 1.0 + shfl_f64(em1, 0), ed = shfl_f64(em1, 1), share = shfl_f64(em1, 2);
  const double d = shfl_f64(arg, 1), kl = ed == INFINITY ? ed : ed - d;  // (d may be +inf too)
  const double adv = q.advantage, w = q.weight;
  const double clipped = fmin(fmax(ratio, 1.0 - p.clip_low), 1.0 + p.clip_high);
  const double plain = times(adv, ratio);  // (the ratio may be infinite, and the advantage 0)
  const bool active = !(plain > clipped * adv);  // a NaN stays one
  const double pg = active ? -plain : -clipped * adv;
  const double dlogp = w * ((active ? -plain : 0.0) - times(p.kl_coef, ed));
  if (write && lane == 0) {
    p.logp[r] = (float)logp;
    put_shared(&terms[r], w * (pg + times(p.kl_coef, kl)));
    put_shared(&terms[rows + r], w * pg);
    put_shared(&terms[2 * rows + r], w * kl);
    put_shared(&terms[3 * rows + r], active ? 0.0 : w);
  }
  return {(float)(-dlogp / (double)o.s), (float)(-dlogp * share)};
}

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
template <bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void kl_policy(LogitArgs a, PolicyArgs p, void *dlogits, int64_t dld,
                                                        double *terms, int32_t *done) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ float red[2 * THREADS / 64];
  __shared__ float coef[2];
  __shared__ uint4 held[KEEP_LDS][THREADS];
  const int64_t r = a.row0 + blockIdx.x;
  const int tid = threadIdx.x;
  if (r == 0 && tid == 0) *done = 0;
  const int64_t target = index_at(a.targets, r);
  const float w = p.weights[r];
  T *d = static_cast<T *>(dlogits) + r * dld;
  if (target < 0 || target >= a.vocab || w == 0.f) {
    const Row<BF16> out(d, a.vocab);
    for (int i = tid; i < out.vecs; i += THREADS) stream16(d + out.col(i), make_uint4(0, 0, 0, 0));
    if (tid < out.singles()) d[out.single(tid)] = T(0);
    if (tid < 4) terms[tid * a.rows + r] = 0.0;
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
  const PolicyRow q = policy_row(p, r, w, at_target);
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
    const PolicyCoef g = policy_coef(p, q, o, r, a.rows, true, terms);
    if (tid == 0) {
      coef[0] = g.c;
      coef[1] = g.dt;
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
    for (int j = 0; j < E::N; ++j) v[j] = c * exp_grad<BF16>(v[j], m);
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
  if (lone) d[row.single(tid)] = E::put(c * exp_grad<BF16>(single, m));
  // the target's own element, by the thread that wrote over it
  const int at = (int)target - row.head;
  const bool in_vec = at >= 0 && at / E::N < row.vecs;
  if (in_vec ? at / E::N % THREADS == tid : lone && row.single(tid) == (uint32_t)target) d[target] = E::put(dt);
}

// The same for short rows, a wave each.
template <bool BF16, int VECS>
__global__ __launch_bounds__(256) void kl_policy_short(LogitArgs a, PolicyArgs p, void *dlogits, int64_t dld,
                                                       double *terms, int32_t *done) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  const int lane = threadIdx.x & 63;
  const int64_t r = a.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  if (r == 0 && lane == 0) *done = 0;
  const int64_t target = index_at(a.targets, r);
  const float w = p.weights[r];
  T *d = static_cast<T *>(dlogits) + r * dld;
  if (target < 0 || target >= a.vocab || w == 0.f) {
    const Row<BF16> out(d, a.vocab);
    for (int i = lane; i < out.vecs; i += 64) stream16(d + out.col(i), make_uint4(0, 0, 0, 0));
    for (int i = lane; i < out.singles(); i += 64) d[out.single(i)] = T(0);
    if (lane < 4) terms[lane * a.rows + r] = 0.0;
    if (lane == 0) p.logp[r] = 0.f;
    return;
  }
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  const PolicyRow q = policy_row(p, r, w, E::get(x[target]));
  const Row<BF16> row(x, a.vocab);
  const ShortRow<BF16, VECS> held(x, row);
  const Online o = held.sum();
  const PolicyCoef own = policy_coef(p, q, o, r, a.rows, true, terms);
  const float c = __shfl(own.c, 0), dt = __shfl(own.dt, 0);
  const int rel = (int)target - row.head;
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int i = lane + 64 * k;
    if (i >= row.vecs) continue;
    float v[E::N];
    E::unpack(held.in[k], v);
#pragma unroll
    for (int j = 0; j < E::N; ++j) v[j] = rel - i * E::N == j ? dt : c * exp_grad<BF16>(v[j], o.m);
    stream16(d + row.col(i), E::pack(v));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (lane + 64 * k >= row.singles()) continue;
    const int j = row.single(lane + 64 * k);
    d[j] = E::put(j == target ? dt : c * exp_grad<BF16>(held.lone[k], o.m));
  }
}

// The four sums over the rows, in a fixed order, four of a workgroup's waves a
// sum; the last workgroup to finish adds up the workgroups' sums.  done was
// cleared by the rows' kernel.
__global__ __launch_bounds__(1024) void kl_policy_sum(const double *terms, int64_t rows, double *part, int32_t *done,
                                                      float *stats) {
  __shared__ double red[16];
  __shared__ int last;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, kind = w & 3, groups = gridDim.x;
  const int64_t r0 = rows * blockIdx.x / groups, r1 = rows * (blockIdx.x + 1) / groups;
  auto four = [&](double sum) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += shfl_xor_f64(sum, d);
    if (lane == 0) red[w] = sum;
    __syncthreads();
    const int k = threadIdx.x & 3;
    sum = red[k] + red[k + 4] + red[k + 8] + red[k + 12];
    __syncthreads();
    return sum;  // thread k has sum k
  };
  double sum = 0.0;
#pragma unroll 8
  for (int64_t r = r0 + (w >> 2) * 64 + lane; r < r1; r += 256) sum += terms[kind * rows + r];
  sum = four(sum);
  if (groups > 1) {
    if (threadIdx.x < 4) put_shared(&part[threadIdx.x * groups + blockIdx.x], sum);
    if (threadIdx.x < 64) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // of all lanes
      if (threadIdx.x == 0) last = arrive(done) == groups - 1;
    }
    __syncthreads();
    if (!last) return;
    const int i = (w >> 2) * 64 + lane;
    sum = four(i < groups ? get_shared(&part[kind * groups + i]) : 0.0);
  }
  if (threadIdx.x < 4) stats[threadIdx.x] = (float)sum;
}

namespace {

// What a piece of a row leaves: its maximum and sum, and the row's target (the
// gradient of another piece may be written over it, in place, before it is
// read again).
struct PieceStat {
  float max, sum, at_target;
};

}  // namespace

// Few rows, in pieces, as a CU's arithmetic (44 cycles a wave and element of
// the sum) is what bounds a row on one CU.  First the pieces' maxima and sums;
// then every piece's gradient, each workgroup joining its row's pieces and
// doing the row's arithmetic for itself.  The last row's first piece to finish
// adds up the rows' terms.
template <bool BF16>
__global__ __launch_bounds__(256, 8) void kl_policy_pieces(LogitArgs a, const float *weights, int pieces,
                                                           PieceStat *part, int32_t *done) {
  __shared__ float red[8];
  const int64_t r = blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces;
  if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;
  const int64_t target = index_at(a.targets, r);
  if (target < 0 || target >= a.vocab || weights[r] == 0.f) return;
  typedef Elem<BF16> E;
  const typename E::type *x = static_cast<const typename E::type *>(a.logits) + r * a.ld;
  const Row<BF16> row(x, a.vocab);
  const int v0 = (int)((int64_t)row.vecs * piece / pieces), v1 = (int)((int64_t)row.vecs * (piece + 1) / pieces);
  const Online o = row_online<BF16, 256>(x, row, v0, v1, piece == 0, red);
  if (threadIdx.x == 0) part[blockIdx.x] = PieceStat{o.m, o.s, E::get(x[target])};
}

template <bool BF16>
__global__ __launch_bounds__(256, 8) void kl_policy_few(LogitArgs a, PolicyArgs p, int pieces, const PieceStat *part,
                                                        void *dlogits, int64_t dld, double *terms, int32_t *done) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int HELD = 4;
  __shared__ float coef[3];
  __shared__ int last;
  const int64_t r = blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces, tid = threadIdx.x;
  const int64_t target = index_at(a.targets, r);
  const float w = p.weights[r];
  const bool live = target >= 0 && target < a.vocab && w != 0.f;
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  T *d = static_cast<T *>(dlogits) + r * dld;
  const Row<BF16> row(live ? x : d, a.vocab);
  const int v0 = (int)((int64_t)row.vecs * piece / pieces) + tid, v1 = (int)((int64_t)row.vecs * (piece + 1) / pieces);
  const bool lone = piece == 0 && tid < row.singles();
  if (live) {
    uint4 in[HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k) in[k] = v0 + k * 256 < v1 ? load16(x + row.col(v0 + k * 256)) : E::none();
    const float single = lone ? E::get(x[row.single(tid)]) : 0.f;
    if (tid < 64) {
      const PolicyRow q = policy_row(p, r, w, part[r * pieces].at_target);
      Online o;
      if (tid < pieces) {
        o.m = part[r * pieces + tid].max;
        o.s = part[r * pieces + tid].sum;
      }
      o = wave_join(o);
      const PolicyCoef g = policy_coef(p, q, o, r, a.rows, piece == 0, terms);
      if (tid == 0) {
        coef[0] = g.c;
        coef[1] = g.dt;
        coef[2] = o.m;
      }
    }
    __syncthreads();
    const float c = coef[0], dt = coef[1], m = coef[2];
    const int rel = (int)target - row.head;
    auto grad = [&](uint4 v4, int i) {
      float v[E::N];
      E::unpack(v4, v);
#pragma unroll
      for (int j = 0; j < E::N; ++j) v[j] = c * exp_grad<BF16>(v[j], m);
      const int j0 = rel - i * E::N;
      if (j0 >= 0 && j0 < E::N) {
#pragma unroll
        for (int j = 0; j < E::N; ++j) v[j] = j == j0 ? dt : v[j];
      }
      store16(d + row.col(i), E::pack(v));
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (v0 + k * 256 < v1) grad(in[k], v0 + k * 256);
    for (int i = v0 + HELD * 256; i < v1; i += 256) grad(load16(x + row.col(i)), i);
    if (lone) d[row.single(tid)] = E::put((int)row.single(tid) == target ? dt : c * exp_grad<BF16>(single, m));
  } else {
    for (int i = v0; i < v1; i += 256) store16(d + row.col(i), make_uint4(0, 0, 0, 0));
    if (lone) d[row.single(tid)] = T(0);
    if (piece == 0 && tid == 0) {
      p.logp[r] = 0.f;
      for (int k = 0; k < 4; ++k) put_shared(&terms[k * a.rows + r], 0.0);
    }
  }
  if (piece != 0) return;
  if (tid == 0) last = arrive(done) == (int)a.rows - 1;
  __syncthreads();
  if (!last) return;
  // a wave a sum, in a fixed order
  double sum = 0.0;
  for (int64_t i = tid & 63; i < a.rows; i += 64) sum += get_shared(&terms[(tid >> 6) * a.rows + i]);
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) sum += shfl_xor_f64(sum, k);
  if ((tid & 63) == 0) p.stats[tid >> 6] = (float)sum;
}

// ------------------------------------------------------- preference loss
//
//   gain = sum logp - ref, m = beta (gain_chosen - gain_rejected)
//   loss = -(1 - s) log sigmoid(m) - s log sigmoid(-m)
//   d loss / d logp = +- beta (s sigmoid(m) - (1 - s) sigmoid(-m)) / pairs
//
// A row's gradient needs its whole pair's log-probabilities, so its logits
// are read twice.  Logits that the memory-side cache (256 MB) holds or nearly
// holds, and short rows, are walked by three launches: the rows' sums
// (kl_rows), the pairs (kl_pairs), the gradient (kl_grad).  Larger ones are
// walked pair by pair in one launch (kp_loss, after kp_plan), the gradient
// following the sums at a distance of the longest pair and some rows more, so
// that it finds them in that cache.

namespace {

// A pair's loss, rewards and the coefficient of its chosen rows.
__device__ __forceinline__ double pair_loss(const PreferenceArgs &p, int64_t i, double chosen, double rejected,
                                            bool write, double *loss) {
  const double gain[2] = {chosen - (double)p.ref_logp[i], rejected - (double)p.ref_logp[i + p.pairs]};
  const double reward[2] = {times(p.beta, gain[0]), times(p.beta, gain[1])};
  const double m = p.beta == 0.0 ? reward[0] - reward[1] : p.beta * (gain[0] - gain[1]);
  // sigmoid(m) and sigmoid(-m) each from exp(-|m|): as 1 minus the other, the
  // far one would be 0 from |m| = 37 on, and no longer accurate to fp32 from 20
  const double q = exp(-fabs(m));
  const double up = (m >= 0.0 ? 1.0 : q) / (1.0 + q), down = (m >= 0.0 ? q : 1.0) / (1.0 + q);
  if (write) {
    p.rewards[i] = (float)reward[0];
    p.rewards[i + p.pairs] = (float)reward[1];
    // softplus(-m) and softplus(m) without overflow
    const double l = log1p(q);
    put_shared(loss, times(1.0 - p.smoothing, fmax(-m, 0.0) + l) + times(p.smoothing, fmax(m, 0.0) + l));
  }
  return p.beta * (p.smoothing * up - (1.0 - p.smoothing) * down) / (double)p.pairs;
}

// The mean of the pairs' losses, in a fixed order.
template <int THREADS>
__device__ __forceinline__ void mean_loss(const PreferenceArgs &p, const double *losses, double *red) {
  double t = 0.0;
  for (int64_t i = threadIdx.x; i < p.pairs; i += THREADS) t += get_shared(&losses[i]);
  t = block_sum<THREADS / 64>(t, red);
  if (threadIdx.x == 0) put_shared(p.loss, (float)(t / (double)p.pairs));
}

// Sequence bounds as kl_pairs uses them: whatever the offsets hold, rows
// outside [0, rows) are never touched.
__device__ __forceinline__ void sequence(const IndexVec &off, int64_t s, int64_t rows, int64_t *lo, int64_t *hi) {
  *lo = min(max(index_at(off, s), (int64_t)0), rows);
  *hi = min(max(index_at(off, s + 1), *lo), rows);
}

}  // namespace

// Sum of the log-probabilities of each sequence, and from them the pair's
// loss and its rows' gradient coefficients; one workgroup a pair, half of it
// a sequence.  Bound by the latency of its few dependent loads.
__global__ __launch_bounds__(1024) void kl_pairs(LogitArgs a, PreferenceArgs p, const RowStat *stat, RowGrad *grad,
                                                 double *losses) {
  __shared__ double red[16];
  const int64_t i = blockIdx.x;
  const int side = threadIdx.x >> 9, tid = threadIdx.x & 511;
  int64_t lo, hi;
  sequence(p.offsets, i + side * p.pairs, a.rows, &lo, &hi);
  double t = 0.0;
  for (int64_t r = lo + tid; r < hi; r += 512) t += stat[r].logp;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) t += shfl_xor_f64(t, k);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = t;
  __syncthreads();
  double sum[2] = {};
#pragma unroll
  for (int w = 0; w < 16; ++w) sum[w >> 3] += red[w];
  const double chosen = pair_loss(p, i, sum[0], sum[1], threadIdx.x == 0, &losses[i]);
  const double d = side ? -chosen : chosen;
  for (int64_t r = lo + tid; r < hi; r += 512) {
    const int64_t target = index_at(a.targets, r);
    if (target < 0 || target >= a.vocab) continue;
    const RowStat st = stat[r];
    grad[r] = RowGrad{st.max, (float)(-d / (double)st.total), (float)(-d * st.share), d != 0.0};
  }
}

// The gradient of the logits, element by element; a row without one gets
// zeros and is not read.  The rows are taken from the last to the first: the
// last ones that the row sums read are still in the memory-side cache.
template <bool BF16>
__global__ __launch_bounds__(256) void kl_grad(LogitArgs a, const RowGrad *grad, void *dlogits, int64_t dld,
                                               int pieces, PreferenceArgs p, const double *losses) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ double red[4];
  if (blockIdx.x == 0) mean_loss<256>(p, losses, red);
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
    for (int k = 0; k < E::N; ++k) v[k] = g.c * exp_grad<BF16>(v[k], g.max);
    const int at = (int)target - (int)row.col(i);
    if (at >= 0 && at < E::N) {
#pragma unroll
      for (int k = 0; k < E::N; ++k) v[k] = k == at ? g.dt : v[k];
    }
    stream16(d + row.col(i), E::pack(v));
  }
  if (piece == 0 && (int)threadIdx.x < row.singles()) {
    const int j = row.single(threadIdx.x);
    d[j] = E::put(j == target ? g.dt : g.c * exp_grad<BF16>(E::get(x[j]), g.max));
  }
}

// The same for short rows, a wave each.
template <bool BF16, int VECS>
__global__ __launch_bounds__(256) void kl_grad_short(LogitArgs a, const RowGrad *grad, void *dlogits, int64_t dld,
                                                     PreferenceArgs p, const double *losses) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ double red[4];
  if (blockIdx.x == 0) mean_loss<256>(p, losses, red);
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  const RowGrad g = grad[r];
  T *d = static_cast<T *>(dlogits) + r * dld;
  if (!g.live) {
    const Row<BF16> out(d, a.vocab);
    for (int i = lane; i < out.vecs; i += 64) stream16(d + out.col(i), make_uint4(0, 0, 0, 0));
    for (int i = lane; i < out.singles(); i += 64) d[out.single(i)] = T(0);
    return;
  }
  const int64_t target = index_at(a.targets, r);
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  const Row<BF16> row(x, a.vocab);
  const ShortRow<BF16, VECS> held(x, row);
  const int rel = (int)target - row.head;
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int i = lane + 64 * k;
    if (i >= row.vecs) continue;
    float v[E::N];
    E::unpack(held.in[k], v);
#pragma unroll
    for (int j = 0; j < E::N; ++j) v[j] = rel - i * E::N == j ? g.dt : g.c * exp_grad<BF16>(v[j], g.max);
    stream16(d + row.col(i), E::pack(v));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (lane + 64 * k >= row.singles()) continue;
    const int j = row.single(lane + 64 * k);
    d[j] = E::put(j == target ? g.dt : g.c * exp_grad<BF16>(held.lone[k], g.max));
  }
}

// One workgroup: the sequences' bounds and the pairs' places in the order of
// the walk, the counters, and whatever belongs to pairs without a row.
__global__ __launch_bounds__(1024) void kp_plan(LogitArgs a, PreferenceArgs p, PreferenceWork w, int slack) {
  __shared__ int wtop[16];
  __shared__ double red[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // bounds: clamped into the rows and, whatever the offsets hold, never
  // decreasing, so that every row belongs to one sequence at most
  int carry = 0;
  for (int64_t j0 = 0; j0 <= 2 * p.pairs; j0 += 1024) {
    const int64_t j = j0 + tid;
    int v = j <= 2 * p.pairs ? (int)min(max(index_at(p.offsets, j), (int64_t)0), a.rows) : 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int u = __shfl_up(v, d);
      if (lane >= d) v = max(v, u);
    }
    if (lane == 63) wtop[wave] = v;
    __syncthreads();
    int all = carry;
    for (int i = 0; i < 16; ++i) {
      if (i == wave) v = max(v, all);
      all = max(all, wtop[i]);
    }
    if (j <= 2 * p.pairs) w.bounds[j] = v;
    carry = all;
    __syncthreads();
  }
  int sum = 0, most = 0, none = 0;
  for (int64_t i0 = 0; i0 < p.pairs; i0 += 1024) {
    const int64_t i = i0 + tid;
    int n = 0;
    if (i < p.pairs) {
      n = w.bounds[i + 1] - w.bounds[i] + w.bounds[i + p.pairs + 1] - w.bounds[i + p.pairs];
      w.done[i] = w.ready[i] = 0;
      if (n == 0) {
        pair_loss(p, i, 0.0, 0.0, true, &w.losses[i]);
        ++none;
      }
      most = max(most, n);
    }
    int x = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int u = __shfl_up(x, d);
      if (lane >= d) x += u;
    }
    if (lane == 63) wtop[wave] = x;
    __syncthreads();
    int base = sum;
    for (int k = 0; k < 16; ++k) {
      if (k == wave) x += base;
      base += wtop[k];
    }
    if (i < p.pairs) w.starts[i] = x - n;
    sum = base;
    __syncthreads();
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) most = max(most, __shfl_xor(most, d));
  if (lane == 0) wtop[wave] = most;
  const int empty = (int)block_sum<16>((double)none, red);
  if (tid == 0) {
    for (int i = 0; i < 16; ++i) most = max(most, wtop[i]);
    w.starts[p.pairs] = sum;
    w.walk->ticket = 0;
    w.walk->pairs_done = empty;
    w.walk->rows = sum;
    w.walk->lag = (int)min((int64_t)sum, (int64_t)most + slack);
    w.walk->late = 0;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (empty == p.pairs) mean_loss<1024>(p, w.losses, red);
}

namespace {

struct Place {
  int64_t row, pair;  // pair -1: a row of no sequence
};

// The at-th row of the walk: the pairs' rows, then those of no sequence.
__device__ __forceinline__ Place place(const PreferenceArgs &p, const PreferenceWork &w, int64_t rows, int64_t n,
                                       int64_t at) {
  auto inside = [&](int64_t row) { return min(max(uniform(row), (int64_t)0), rows - 1); };
  if (at >= n) {
    const int64_t lead = w.bounds[0];
    return {inside(at - n < lead ? at - n : w.bounds[2 * p.pairs] + (at - n - lead)), -1};
  }
  // the last pair that starts at or before this place, 64 probes at a time
  int64_t lo = 0, hi = p.pairs;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, probe = lo + (threadIdx.x & 63) * step;
    const int c = max(__popcll(__ballot(probe < hi && w.starts[min(probe, p.pairs)] <= at)), 1);
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
  }
  const int64_t pair = uniform(lo);
  const int64_t off = at - w.starts[pair], len = w.bounds[pair + 1] - w.bounds[pair];
  return {inside(off < len ? w.bounds[pair] + off : w.bounds[pair + p.pairs] + (off - len)), pair};
}

}  // namespace

// A workgroup takes a ticket t and does the sum of the walk's t-th row, then
// the gradient of the row `lag` places before it.  What a gradient waits for
// are sums of earlier tickets, and a sum waits for nothing, so every wait
// ends.  The grid has 2 rows' workgroups, as the host does not know the lag;
// those too many, spread over the grid, end at once.
//
// Should a wait not end all the same (another call running on the same
// workspace), it is given up after max_polls looks, and so are those that
// would follow: their rows' gradients and the loss become NaN, and tickets and
// rows beyond the walk are not taken.
//
// 12500 rows of 50257 bf16 in 16 pairs: 457 us, 4.6 TB/s; the second reads that
// the cache still holds are what it gains over three launches (545).  The
// tickets come from one address, 18 ns apart (230 us in all, beside the rows'
// own time); with a gradient as a unit of its own they took the time of both.
// Rows between a pair's last sum and its first gradient: 64 (256: 470 us, 512:
// 492, 1024: 521; the shorter the way, the more the cache still holds).
template <bool BF16>
__global__ __launch_bounds__(PREF_THREADS, 8) void kp_loss(LogitArgs a, PreferenceArgs p, PreferenceWork w,
                                                           void *dlogits, int64_t dld) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int THREADS = PREF_THREADS, AHEAD = 4;
  __shared__ float red[2 * THREADS / 64];
  __shared__ double red64[THREADS / 64];
  __shared__ uint64_t unit;
  __shared__ int last;
  __shared__ struct {
    float max, c, dt;
    int live;
  } grad;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t n = uniform(w.walk->rows), lag = uniform(w.walk->lag);
  const uint64_t units = (uint64_t)(a.rows + lag), groups = 2 * (uint64_t)a.rows, group = (uint64_t)a.row0 + blockIdx.x;
  if (group * units / groups == (group + 1) * units / groups) return;
  if (tid == 0) unit = atomicAdd((unsigned long long *)&w.walk->ticket, 1ull);
  __syncthreads();
  const int64_t t = uniform((int64_t)unit);
  if ((uint64_t)t >= units) return;
  if (t < n) {
    const Place at = place(p, w, a.rows, n, t);
    const int64_t r = at.row, pair = at.pair;
    const int64_t target = uniform(index_at(a.targets, r));
    double logp = 0.0, share = 0.0;
    Online o;
    if (target >= 0 && target < a.vocab) {
      const T *x = static_cast<const T *>(a.logits) + r * a.ld;
      const float at_target = E::get(x[target]);
      o = row_online<BF16, THREADS>(x, a.vocab, red);
      if (tid == 0) {
        logp = (double)at_target - (double)o.m - log((double)o.s);
        share = expm1(logp);
      }
    }
    if (tid == 0) {
      RowStat *st = w.stat + r;
      put_shared(&st->max, o.m);
      put_shared(&st->total, o.s);
      put_shared(&st->logp, logp);
      put_shared(&st->share, share);
      last = arrive(&w.done[pair]) == (int)(w.starts[pair + 1] - w.starts[pair]) - 1;
    }
    __syncthreads();
    if (last) {
      // the pair's sums, half of the workgroup a sequence
      const int64_t s = pair + tid / (THREADS / 2) * p.pairs;
      double sum = 0.0;
      for (int64_t i = w.bounds[s] + tid % (THREADS / 2); i < w.bounds[s + 1]; i += THREADS / 2)
        sum += get_shared(&w.stat[i].logp);
#pragma unroll
      for (int k = 32; k > 0; k >>= 1) sum += shfl_xor_f64(sum, k);
      if (lane == 0) red64[tid >> 6] = sum;
      __syncthreads();
      if (tid == 0) {
        double of[2] = {};
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) of[i / (THREADS / 128)] += red64[i];
        put_shared(&w.coef[pair], pair_loss(p, pair, of[0], of[1], true, &w.losses[pair]));
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        put_shared(&w.ready[pair], 1);
        last = arrive(&w.walk->pairs_done) == (int)p.pairs - 1;
      }
      __syncthreads();
      if (last) {
        mean_loss<THREADS>(p, w.losses, red64);
        if (tid == 0) {  // the loss is NaN if a gradient gives up, whichever comes last
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          if (get_shared(&w.walk->late)) put_shared(p.loss, __builtin_nanf(""));
        }
      }
    }
  }
  if (t < lag) return;
  const Place at = place(p, w, a.rows, n, t - lag);
  const int64_t r = at.row, pair = at.pair;
  const int64_t target = uniform(index_at(a.targets, r));
  const bool live = pair >= 0 && target >= 0 && target < a.vocab;
  const T *x = static_cast<const T *>(a.logits) + r * a.ld;
  T *d = static_cast<T *>(dlogits) + r * dld;
  const Row<BF16> row(live ? x : d, a.vocab);
  uint4 in[AHEAD];
  if (live) {  // the first loads are under way while thread 0 waits for the pair
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      in[k] = E::none();
      if (tid + k * THREADS < row.vecs) in[k] = load16(x + row.col(tid + k * THREADS));
    }
    if (tid == 0) {
      bool late = false;
      for (int left = w.max_polls; !(left >= 0 && get_shared(&w.ready[pair])); --left) {
        late = left <= 0 || get_shared(&w.walk->late);
        if (late) break;
        __builtin_amdgcn_s_sleep(2);
      }
      asm volatile("" ::: "memory");
      const RowStat *st = w.stat + r;
      const double coef = get_shared(&w.coef[pair]), total = (double)get_shared(&st->total), share = get_shared(&st->share);
      const double dl = r >= w.bounds[pair] && r < w.bounds[pair + 1] ? coef : -coef;
      grad.max = get_shared(&st->max);
      grad.c = (float)(-dl / total);
      grad.dt = (float)(-dl * share);
      grad.live = dl != 0.0;
      if (late) {
        grad.c = grad.dt = __builtin_nanf("");
        grad.live = 1;
        put_shared(&w.walk->late, 1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        put_shared(p.loss, __builtin_nanf(""));
      }
    }
  }
  __syncthreads();
  if (!live || !grad.live) {
    for (int i = tid; i < row.vecs; i += THREADS) stream16(d + row.col(i), make_uint4(0, 0, 0, 0));
    if (tid < row.singles()) d[row.single(tid)] = T(0);
    return;
  }
  const float c = grad.c, dt = grad.dt, m = grad.max;
  const int rel = (int)target - row.head;  // the target's place among the vectors
  auto put = [&](uint4 v4, int i) {
    float v[E::N];
    E::unpack(v4, v);
#pragma unroll
    for (int k = 0; k < E::N; ++k) v[k] = c * exp_grad<BF16>(v[k], m);
    const int k0 = rel - i * E::N;
    if (k0 >= 0 && k0 < E::N) {
#pragma unroll
      for (int k = 0; k < E::N; ++k) v[k] = k == k0 ? dt : v[k];
    }
    stream16(d + row.col(i), E::pack(v));
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (tid + k * THREADS < row.vecs) put(in[k], tid + k * THREADS);
  int i = tid + AHEAD * THREADS;
  for (; i + (AHEAD - 1) * THREADS < row.vecs; i += AHEAD * THREADS) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) in[k] = load16(x + row.col(i + k * THREADS));
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) put(in[k], i + k * THREADS);
  }
  for (; i < row.vecs; i += THREADS) put(load16(x + row.col(i)), i);
  if (tid < row.singles()) {
    const int j = row.single(tid);
    d[j] = E::put(j == target ? dt : c * exp_grad<BF16>(E::get(x[j]), m));
  }
}

// ------------------------------------------------------------- launchers

// Looks, about a microsecond apart, that a gradient takes at its pair before it
// gives up: four seconds and more.  Not in the header; a test sets it to -1 to
// see every wait given up.
extern "C" {
int muon_preference_max_polls = 1 << 22;
}

namespace {

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

namespace {

// A grid holds fewer than 2^32 threads: more rows take several launches.
constexpr int64_t ROWS_A_LAUNCH = (int64_t)1 << 21;
template <class F>
hipError_t by_rows(LogitArgs a, int64_t rows, F launch) {
  for (a.row0 = 0; a.row0 < rows; a.row0 += ROWS_A_LAUNCH) {
    launch(a, dim3((unsigned)std::min(ROWS_A_LAUNCH, rows - a.row0)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Vectors a lane of a row that one wave holds; 0: the row is too long for that.
// 8192 rows, in us, a wave and a workgroup of 256 a row: log-probability, 1000
// bf16 columns 8.3 12.4, 4096 15.7 17.3, 2000 fp32 13.2 15.9; policy loss
// 18.8 28.3, 29.5 32.7, 27.9 29.6; preference loss 20.4 30.4, 42.8 43.0, 39.4
// 41.5; 300 rows the same either way.
template <bool BF16>
int short_vecs(int64_t vocab) {
  for (int vecs = 2; vecs <= 8; vecs *= 2)
    if (vocab <= 64 * vecs * Elem<BF16>::N) return vecs;
  return 0;
}

// 256 threads where 512 would have fewer than two rounds of loads (20000 x
// 4096 bf16: 35 us instead of 56); from there on 512 are as fast or faster
// (100 x 50257 fp32 6.7 against 8.3).  Where every row can have a CU to itself,
// 1024 and eight loads under way (32 x 131072: 10.3 us instead of 11.0).
template <bool BF16>
hipError_t rows_launch(const LogitArgs &a, RowStat *stat, RowGrad *grad, float *logp, float *lse, hipStream_t s) {
  const int vecs = short_vecs<BF16>(a.vocab);
  return by_rows(a, a.rows, [&](const LogitArgs &a, dim3 g) {
    const dim3 g4((g.x + 3) / 4);
    if (vecs == 2) hipLaunchKernelGGL((kl_rows_short<BF16, 2>), g4, dim3(256), 0, s, a, stat, grad, logp, lse);
    else if (vecs == 4) hipLaunchKernelGGL((kl_rows_short<BF16, 4>), g4, dim3(256), 0, s, a, stat, grad, logp, lse);
    else if (vecs == 8) hipLaunchKernelGGL((kl_rows_short<BF16, 8>), g4, dim3(256), 0, s, a, stat, grad, logp, lse);
    else if (a.vocab <= 1024 * Elem<BF16>::N) hipLaunchKernelGGL((kl_rows<BF16, 256, 4>), g, dim3(256), 0, s, a, stat, grad, logp, lse);
    else if (a.rows <= 256 && a.vocab >= 8192 * Elem<BF16>::N) hipLaunchKernelGGL((kl_rows<BF16, 1024, 8>), g, dim3(1024), 0, s, a, stat, grad, logp, lse);
    else hipLaunchKernelGGL((kl_rows<BF16, 512, 4>), g, dim3(512), 0, s, a, stat, grad, logp, lse);
  });
}

}  // namespace

hipError_t launch_token_logprob(const LogitArgs &a, bool bf16, float *logp, float *lse, hipStream_t s) {
  return bf16 ? rows_launch<true>(a, nullptr, nullptr, logp, lse, s) : rows_launch<false>(a, nullptr, nullptr, logp, lse, s);
}

PolicyLayout policy_layout(int64_t rows) {
  PolicyLayout l{};
  l.done = 0;
  l.part = 256;  // the few rows' pieces, or the workgroups' sums
  l.terms = l.part + up256(std::max(sizeof(PieceStat) * FEW_GROUPS, 4 * sizeof(double) * SUM_GROUPS));
  l.total = l.terms + up256(4 * sizeof(double) * (size_t)std::max<int64_t>(rows, 1));
  return l;
}

namespace {

template <bool BF16>
hipError_t policy_launch(const LogitArgs &a, const PolicyArgs &p, void *dlogits, int64_t dld, char *ws, hipStream_t s) {
  const PolicyLayout l = policy_layout(a.rows);
  double *terms = reinterpret_cast<double *>(ws + l.terms);
  int32_t *done = reinterpret_cast<int32_t *>(ws + l.done);
  const int64_t vecs = a.vocab / Elem<BF16>::N;
  if (a.rows > 0 && a.rows <= FEW_ROWS && vecs >= FEW_ROW) {
    static_assert(FEW_GROUPS / FEW_ROWS >= 2 && FEW_ROW / FEW_VECS >= 2, "two pieces at least");
    const int64_t pieces = std::min<int64_t>({FEW_GROUPS / a.rows, vecs / FEW_VECS, 64});  // a lane a piece joins them
    PieceStat *part = reinterpret_cast<PieceStat *>(ws + l.part);
    const dim3 g((unsigned)(a.rows * pieces));
    hipLaunchKernelGGL(kl_policy_pieces<BF16>, g, dim3(256), 0, s, a, p.weights, (int)pieces, part, done);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kl_policy_few<BF16>, g, dim3(256), 0, s, a, p, (int)pieces, part, dlogits, dld, terms, done);
    return hipGetLastError();
  }
  const int held = short_vecs<BF16>(a.vocab);
  hipError_t e = by_rows(a, a.rows, [&](const LogitArgs &a, dim3 g) {
    const dim3 g4((g.x + 3) / 4);
    if (held == 2) hipLaunchKernelGGL((kl_policy_short<BF16, 2>), g4, dim3(256), 0, s, a, p, dlogits, dld, terms, done);
    else if (held == 4) hipLaunchKernelGGL((kl_policy_short<BF16, 4>), g4, dim3(256), 0, s, a, p, dlogits, dld, terms, done);
    else if (held == 8) hipLaunchKernelGGL((kl_policy_short<BF16, 8>), g4, dim3(256), 0, s, a, p, dlogits, dld, terms, done);
    else if (vecs <= 256 * KEEP) hipLaunchKernelGGL((kl_policy<BF16, 256>), g, dim3(256), 0, s, a, p, dlogits, dld, terms, done);
    else hipLaunchKernelGGL((kl_policy<BF16, 1024>), g, dim3(1024), 0, s, a, p, dlogits, dld, terms, done);
  });
  if (e != hipSuccess) return e;
  const int64_t groups = std::min<int64_t>(SUM_GROUPS, std::max<int64_t>(1, a.rows / SUM_ROWS));
  hipLaunchKernelGGL(kl_policy_sum, dim3((unsigned)groups), dim3(1024), 0, s, terms, a.rows, reinterpret_cast<double *>(ws + l.part), done,
                     p.stats);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_policy(const LogitArgs &a, const PolicyArgs &p, bool bf16, void *dlogits, int64_t dld, char *ws,
                         hipStream_t s) {
  return bf16 ? policy_launch<true>(a, p, dlogits, dld, ws, s) : policy_launch<false>(a, p, dlogits, dld, ws, s);
}

PreferenceLayout preference_layout(int64_t rows, int64_t pairs) {
  PreferenceLayout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += up256(bytes);
    return p;
  };
  l.walk = take(sizeof(PreferenceWalk));
  l.stat = take(sizeof(RowStat) * (size_t)rows);
  l.grad = take(sizeof(RowGrad) * (size_t)rows);
  l.losses = take(sizeof(double) * (size_t)pairs);
  l.coef = take(sizeof(double) * (size_t)pairs);
  l.bounds = take(sizeof(int32_t) * (2 * (size_t)pairs + 1));
  l.starts = take(sizeof(int32_t) * ((size_t)pairs + 1));
  l.done = take(sizeof(int32_t) * (size_t)pairs);
  l.ready = take(sizeof(int32_t) * (size_t)pairs);
  l.total = at;
  return l;
}

namespace {

template <bool BF16>
hipError_t preference_launch(const LogitArgs &a, const PreferenceArgs &p, void *dlogits, int64_t dld, char *ws,
                             hipStream_t s) {
  const PreferenceLayout l = preference_layout(a.rows, p.pairs);
  PreferenceWork w{};
  w.max_polls = muon_preference_max_polls;
  w.walk = reinterpret_cast<PreferenceWalk *>(ws + l.walk);
  w.stat = reinterpret_cast<RowStat *>(ws + l.stat);
  w.losses = reinterpret_cast<double *>(ws + l.losses);
  w.coef = reinterpret_cast<double *>(ws + l.coef);
  w.bounds = reinterpret_cast<int32_t *>(ws + l.bounds);
  w.starts = reinterpret_cast<int32_t *>(ws + l.starts);
  w.done = reinterpret_cast<int32_t *>(ws + l.done);
  w.ready = reinterpret_cast<int32_t *>(ws + l.ready);
  RowGrad *grad = reinterpret_cast<RowGrad *>(ws + l.grad);
  hipError_t e;
  // One walk where the memory-side cache does not hold the logits but does hold
  // what lies between a sum and its gradient (a pair, here the average one, and
  // the 1024 rows under way), and where a row takes longer than its tickets.
  // In us, walk and three launches:
  //   total, pairs of 768 rows of 50257 bf16: 294 MB 168 161, 368 MB 206 206,
  //     441 MB 236 249, 588 MB 306 338, 1325 MB 652 791
  //   row, at about 600 MB and 1200 MB: 8 KB (4096 bf16) 1101 338; 16 KB 584 310;
  //     32 KB 479 383, 772 764; 44 KB 340 340, 643 672 (but 48 KB at 457 MB 288
  //     251); 64 KB 358 349, 649 770 (468 MB: 257 264); 80 KB 297 322, 606 727;
  //     128 KB (fp32, pairs of 300) 292 339, 560 726
  //   what lies between, at about 600 MB: 212 MB (80 rows of 200 KB a pair) 316
  //     343, 215 MB (700 of 128 KB) 336 326, 223 MB (1300 of 100 KB) 348 360, 306
  //     MB (200 of 256 KB) 353 329
  const int64_t row = a.vocab * (int64_t)sizeof(typename Elem<BF16>::type);
  const bool walk = row >= (56 << 10) && a.rows * row > (400 << 20) && (a.rows / p.pairs + 1024) * row <= (224 << 20);
  if (walk || a.rows > ROWS_A_LAUNCH || p.pairs > ROWS_A_LAUNCH) {
    hipLaunchKernelGGL(kp_plan, dim3(1), dim3(1024), 0, s, a, p, w, PREF_SLACK);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return by_rows(a, 2 * a.rows, [&](const LogitArgs &a, dim3 g) {
      hipLaunchKernelGGL(kp_loss<BF16>, g, dim3(PREF_THREADS), 0, s, a, p, w, dlogits, dld);
    });
  }
  if ((e = rows_launch<BF16>(a, w.stat, grad, nullptr, nullptr, s)) != hipSuccess) return e;
  hipLaunchKernelGGL(kl_pairs, dim3((unsigned)p.pairs), dim3(1024), 0, s, a, p, w.stat, grad, w.losses);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (const int held = short_vecs<BF16>(a.vocab)) {
    const dim3 g((unsigned)std::max<int64_t>(1, (a.rows + 3) / 4));
    if (held == 2) hipLaunchKernelGGL((kl_grad_short<BF16, 2>), g, dim3(256), 0, s, a, grad, dlogits, dld, p, w.losses);
    else if (held == 4) hipLaunchKernelGGL((kl_grad_short<BF16, 4>), g, dim3(256), 0, s, a, grad, dlogits, dld, p, w.losses);
    else hipLaunchKernelGGL((kl_grad_short<BF16, 8>), g, dim3(256), 0, s, a, grad, dlogits, dld, p, w.losses);
    return hipGetLastError();
  }
  // pieces of a row: 8192 elements or more, and a grid that stays in range
  const int64_t most = 4 * ROWS_A_LAUNCH / std::max<int64_t>(a.rows, 1);
  const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>({a.vocab / 8192, 64, most}));
  hipLaunchKernelGGL(kl_grad<BF16>, dim3((unsigned)std::max<int64_t>(1, a.rows * pieces)), dim3(256), 0, s, a, grad, dlogits, dld,
                     (int)pieces, p, w.losses);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_preference(const LogitArgs &a, const PreferenceArgs &p, bool bf16, void *dlogits, int64_t dld,
                             char *ws, hipStream_t s) {
  return bf16 ? preference_launch<true>(a, p, dlogits, dld, ws, s) : preference_launch<false>(a, p, dlogits, dld, ws, s);
}

}  // namespace muon
