// The balance loss of a mixture-of-experts router with its gradient, and the
// tokens each expert gets, on gfx950.
//
//   p_t = softmax(x_t), lse_t = log sum exp x_t, over the T counted tokens
//   f_e = counts_e / (T k),  balance = E sum_e f_e mean_t p_te
//   z   = mean_t lse_t^2,    loss = coef balance + z_coef z
//   d loss / d x_te = p_te (coef E / T (f_e - sum_j p_tj f_j) + 2 z_coef / T lse_t)
//
// (the counts are whole numbers and carry no gradient).  With f known, a
// token's share of the balance is E / T sum_j p_tj f_j, which its gradient
// needs anyway, so the logits are read once and no per-expert mean of p is
// kept.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "devops.hpp"
#include "train_ops.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int BH_GROUPS = 64;      // workgroups that count choices
constexpr int BM_GROUPS = 1024;    // workgroups of the main pass, at most

}  // namespace

// Choices per expert of one part of the tokens: hist[part][e], and the part's
// counted tokens at hist[part][E].
__global__ __launch_bounds__(1024) void kb_count(BalanceArgs a, int32_t *hist) {
  __shared__ int h[BAL_MAX_EXPERTS + 1];
  const int parts = gridDim.x;
  for (int e = threadIdx.x; e <= a.n_experts; e += 1024) h[e] = 0;
  __syncthreads();
  const int64_t t0 = a.tokens * blockIdx.x / parts, t1 = a.tokens * (blockIdx.x + 1) / parts;
  int live = 0;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += 1024) live += !a.valid || a.valid[t];
  if (live) atomicAdd(&h[a.n_experts], live);
  for (int64_t i = t0 * a.k + threadIdx.x; i < t1 * a.k; i += 1024) {
    const int64_t e = index_at(a.experts, i);
    if (e >= 0 && e < a.n_experts && (!a.valid || a.valid[i / a.k])) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.n_experts; e += 1024) hist[(int64_t)blockIdx.x * (a.n_experts + 1) + e] = h[e];
}

// One wave a token, ITEMS logits a lane (lane, lane + 64, ...).
template <bool BF16, int ITEMS>
__global__ __launch_bounds__(256) void kb_main(BalanceArgs a, const int32_t *hist, int parts, double *sums) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  __shared__ float f_of[BAL_MAX_EXPERTS];
  __shared__ int total;
  __shared__ double red[4];
  const int n = a.n_experts, lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e <= n; e += 256) {
    int c = 0;
    for (int i = 0; i < parts; ++i) c += hist[(int64_t)i * (n + 1) + e];
    if (e == n) total = c;
    else {
      f_of[e] = (float)c;
      if (blockIdx.x == 0) a.counts[e] = c;
    }
  }
  __syncthreads();
  const float tokens = (float)max(total, 1);
  float f[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) f[i] = lane + 64 * i < n ? f_of[lane + 64 * i] / (tokens * (float)a.k) : 0.f;
  const float cb = (float)(a.coef * (double)n / (double)tokens), cz = (float)(2.0 * a.z_coef / (double)tokens);
  double bal = 0.0, zz = 0.0;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
    T *d = static_cast<T *>(a.dlogits) + t * a.dld;
    if (a.valid && !a.valid[t]) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (lane + 64 * i < n) d[lane + 64 * i] = T(0);
      continue;
    }
    const T *x = static_cast<const T *>(a.logits) + t * a.ld;
    float v[ITEMS], m = kLowest, s = 0.f, pf = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      v[i] = lane + 64 * i < n ? E::get(x[lane + 64 * i]) : -INFINITY;
      m = fmaxf(m, v[i]);
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      v[i] = exp_shift(v[i], m);
      s += v[i];
      pf += v[i] * f[i];
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) {
      s += __shfl_xor(s, k);
      pf += __shfl_xor(pf, k);
    }
    const float inv = 1.f / s, mean_f = pf * inv, lse = m + logf(s);
    bal += (double)mean_f;
    zz += (double)lse * (double)lse;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (lane + 64 * i < n) d[lane + 64 * i] = E::put(v[i] * inv * (cb * (f[i] - mean_f) + cz * lse));
  }
  // every lane of a wave holds the wave's sums
  const double tb = block_sum<4>(lane == 0 ? bal : 0.0, red), tz = block_sum<4>(lane == 0 ? zz : 0.0, red);
  if (threadIdx.x == 0) {
    sums[3 * blockIdx.x] = tb;
    sums[3 * blockIdx.x + 1] = tz;
    sums[3 * blockIdx.x + 2] = (double)total;
  }
}

__global__ __launch_bounds__(256) void kb_final(BalanceArgs a, const double *sums, int groups) {
  __shared__ double red[4];
  double b = 0.0, z = 0.0;
  for (int i = threadIdx.x; i < groups; i += 256) {
    b += sums[3 * i];
    z += sums[3 * i + 1];
  }
  b = block_sum<4>(b, red);
  z = block_sum<4>(z, red);
  if (threadIdx.x == 0) {
    const double t = fmax(sums[2], 1.0);
    b *= (double)a.n_experts / t;
    z /= t;
    a.stats[0] = (float)(a.coef * b + a.z_coef * z);
    a.stats[1] = (float)b;
    a.stats[2] = (float)z;
  }
}

BalanceLayout balance_layout(int64_t tokens, int32_t n_experts) {
  (void)tokens;
  BalanceLayout l{};
  l.hist = 0;
  l.sums = ((size_t)BH_GROUPS * ((size_t)n_experts + 1) * 4 + 255) / 256 * 256;
  l.total = l.sums + 3 * sizeof(double) * BM_GROUPS;
  return l;
}

namespace {

template <bool BF16>
void main_launch(const BalanceArgs &a, const int32_t *hist, int parts, double *sums, int groups, hipStream_t s) {
  const dim3 g(groups), b(256);
  if (a.n_experts <= 64) hipLaunchKernelGGL((kb_main<BF16, 1>), g, b, 0, s, a, hist, parts, sums);
  else if (a.n_experts <= 256) hipLaunchKernelGGL((kb_main<BF16, 4>), g, b, 0, s, a, hist, parts, sums);
  else hipLaunchKernelGGL((kb_main<BF16, BAL_MAX_EXPERTS / 64>), g, b, 0, s, a, hist, parts, sums);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs &a, bool bf16, char *ws, hipStream_t s) {
  const BalanceLayout l = balance_layout(a.tokens, a.n_experts);
  int32_t *hist = reinterpret_cast<int32_t *>(ws + l.hist);
  double *sums = reinterpret_cast<double *>(ws + l.sums);
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(BH_GROUPS, a.tokens / 512));
  hipLaunchKernelGGL(kb_count, dim3(parts), dim3(1024), 0, s, a, hist);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(BM_GROUPS, (a.tokens + 3) / 4));
  if (bf16) main_launch<true>(a, hist, parts, sums, groups, s);
  else main_launch<false>(a, hist, parts, sums, groups, s);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(kb_final, dim3(1), dim3(256), 0, s, a, sums, groups);
  return hipGetLastError();
}

}  // namespace muon
