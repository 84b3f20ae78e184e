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

// Workgroups that count choices, at most: 131072 tokens of 256 experts, 8
// choices, take 68.7 us with 64, 66.3 with 128, 70.8 with 256 (every workgroup
// of the main pass adds up all their counts).
constexpr int BH_GROUPS = 128;
constexpr int BM_GROUPS = 512;  // workgroups of the main pass, at most: two on a CU
constexpr int BM_THREADS = 1024;
// Up to this many logits (and choices) one workgroup does the whole call.  In
// us, so and in two launches: 509 x 8 11.2 14.9, 256 x 64 11.6 14.8, but 1000 x
// 60 24.0 16.2, 4000 x 8 30 16.5.
constexpr int64_t BALANCE_SOLO = 16384;

// Adds the choices of tokens [t0, t1) to h; returns this thread's counted tokens.
__device__ __forceinline__ int count_choices(const BalanceArgs &a, int64_t t0, int64_t t1, int *h) {
  int live = 0;
  if (a.valid) {
#pragma unroll 4
    for (int64_t t = t0 + threadIdx.x; t < t1; t += 1024) live += a.valid[t] != 0;
  } else if (threadIdx.x == 0) {
    live = (int)(t1 - t0);
  }
  // tokens * k stays below 2^31; the loads of a round are under way together
  constexpr int ROUND = 4;
  const uint32_t k = (uint32_t)a.k, end = (uint32_t)t1 * k;
  for (uint32_t i = (uint32_t)t0 * k + threadIdx.x; i < end; i += ROUND * 1024) {
    int64_t e[ROUND];
    uint8_t ok[ROUND];
#pragma unroll
    for (int q = 0; q < ROUND; ++q) {
      const uint32_t j = i + q * 1024;
      e[q] = j < end ? index_at(a.experts, j) : -1;
      ok[q] = j < end && a.valid ? a.valid[j / k] : 1;
    }
#pragma unroll
    for (int q = 0; q < ROUND; ++q)
      if (e[q] >= 0 && e[q] < a.n_experts && ok[q]) atomicAdd(&h[e[q]], 1);
  }
  return live;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int x = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false));
}

// Reductions over LANES consecutive lanes (4, 16 or 64); every lane gets the
// same bits, since each step joins two lanes that hold the same two halves.
constexpr int QUAD_XOR1 = 0xb1, QUAD_XOR2 = 0x4e, ROW_ROR8 = 0x128, ROW_ROR4 = 0x124;
template <int LANES, class F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  v = f(v, dpp<QUAD_XOR1>(v));
  v = f(v, dpp<QUAD_XOR2>(v));
  if constexpr (LANES >= 16) {
    v = f(v, dpp<ROW_ROR8>(v));
    v = f(v, dpp<ROW_ROR4>(v));
  }
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}

}  // namespace

// Choices per expert of one part of the tokens: hist[part][e], and the part's
// counted tokens at hist[part][E].  Clears the main pass's arrival count.
__global__ __launch_bounds__(1024) void kb_count(BalanceArgs a, int32_t *hist, int32_t *arrive) {
  __shared__ int h[BAL_MAX_EXPERTS + 1];
  const int parts = gridDim.x;
  for (int e = threadIdx.x; e <= a.n_experts; e += 1024) h[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *arrive = 0;
  __syncthreads();
  const int live = count_choices(a, a.tokens * blockIdx.x / parts, a.tokens * (blockIdx.x + 1) / parts, h);
  if (live) atomicAdd(&h[a.n_experts], live);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.n_experts; e += 1024) hist[(int64_t)blockIdx.x * (a.n_experts + 1) + e] = h[e];
}

// A group of LANES lanes takes a token, VECS 16-byte vectors a lane, so that
// a wave reduces 64 / LANES tokens at a time and most steps stay inside a row
// of 16 lanes.  HBM-bound: one read and one write of the logits; 131072 x 256
// fp32 take 47 us, 5.3 TB/s (a wave a token, four loads of four bytes a lane
// and shuffles through LDS: 73 to 82); with ordinary stores a call takes 71 us
// instead of 69, in bf16 54 instead of 46.  The last workgroup to finish adds
// up the workgroups' sums, in their order.  With
// parts = 0 the only workgroup counts the choices itself.
template <bool BF16, int LANES, int VECS>
__global__ __launch_bounds__(BM_THREADS, 8) void kb_main(BalanceArgs a, const int32_t *hist, int parts, double *sums,
                                                         int32_t *arrive) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N, PER = BM_THREADS / LANES;
  __shared__ int count[BAL_MAX_EXPERTS + 1];
  __shared__ __attribute__((aligned(16))) float f_of[LANES * VECS * N];
  __shared__ double red[BM_THREADS / 64];
  __shared__ int last;
  const int n = a.n_experts, tid = threadIdx.x, l = tid & (LANES - 1);
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t t = (int64_t)blockIdx.x * PER + tid / LANES;
  float v[VECS][N];
  bool ok, next = t < a.tokens && (!a.valid || a.valid[t]);
  // the token's logits, and whether the next one counts
  auto fetch = [&](int64_t t) {
    ok = next;
    next = t + step < a.tokens && (!a.valid || a.valid[t + step]);
    if (!ok) return;
    const T *x = static_cast<const T *>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = (l + LANES * i) * N;
      if (c + N <= n) {
        E::unpack(load16(x + c), v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = c + j < n ? E::get(x[c + j]) : -INFINITY;
      }
    }
  };
  fetch(t);
  for (int e = tid; e <= n; e += BM_THREADS) count[e] = 0;
  __syncthreads();
  if (parts == 0) {
    const int live = count_choices(a, 0, a.tokens, count);
    if (live) atomicAdd(&count[n], live);
  } else {
    constexpr int ROUND = 8;
    const int all = parts * (n + 1);
    for (int i = tid; i < all; i += ROUND * BM_THREADS) {
      int c[ROUND];
#pragma unroll
      for (int q = 0; q < ROUND; ++q) c[q] = i + q * BM_THREADS < all ? hist[i + q * BM_THREADS] : 0;
#pragma unroll
      for (int q = 0; q < ROUND; ++q)
        if (c[q]) atomicAdd(&count[(i + q * BM_THREADS) % (n + 1)], c[q]);
    }
  }
  __syncthreads();
  const int total = count[n];
  const float tokens = (float)max(total, 1);
  for (int e = tid; e < LANES * VECS * N; e += BM_THREADS) {
    f_of[e] = e < n ? (float)count[e] / (tokens * (float)a.k) : 0.f;
    if (blockIdx.x == 0 && e < n) a.counts[e] = count[e];
  }
  __syncthreads();
  const float cb = (float)(a.coef * (double)n / (double)tokens), cz = (float)(2.0 * a.z_coef / (double)tokens);
  double bal = 0.0, zz = 0.0;
  for (; t < a.tokens; t += step) {
    T *d = static_cast<T *>(a.dlogits) + t * a.dld;
    if (ok) {
      float m = kLowest;
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, v[i][j]);
      m = group_reduce<LANES>(m, [](float p, float q) { return fmaxf(p, q); });
      float s = 0.f, pf = 0.f;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const float *f = f_of + (l + LANES * i) * N;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          v[i][j] = exp_shift(v[i][j], m);
          s += v[i][j];
          pf += v[i][j] * f[j];
        }
      }
      s = group_reduce<LANES>(s, [](float p, float q) { return p + q; });
      pf = group_reduce<LANES>(pf, [](float p, float q) { return p + q; });
      const float inv = 1.f / s, mean_f = pf * inv, lse = m + logf(s);
      if (l == 0) {
        bal += (double)mean_f;
        zz += (double)lse * (double)lse;
      }
      const float base = cz * lse;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const float *f = f_of + (l + LANES * i) * N;
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = v[i][j] * inv * (cb * (f[j] - mean_f) + base);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = (l + LANES * i) * N;
      if (c + N <= n) {
        stream16(d + c, E::pack(v[i]));
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c + j < n) d[c + j] = E::put(v[i][j]);
      }
    }
    fetch(t + step);
  }
  double tb = block_sum<BM_THREADS / 64>(bal, red), tz = block_sum<BM_THREADS / 64>(zz, red);
  if (parts != 0) {
    const int groups = gridDim.x;
    if (tid == 0) {
      put_shared(&sums[2 * blockIdx.x], tb);
      put_shared(&sums[2 * blockIdx.x + 1], tz);
      last = dev::arrive(arrive) == groups - 1;
    }
    __syncthreads();
    if (!last) return;
    const bool in = tid < groups;
    tb = block_sum<BM_THREADS / 64>(in ? get_shared(&sums[2 * tid]) : 0.0, red);
    tz = block_sum<BM_THREADS / 64>(in ? get_shared(&sums[2 * tid + 1]) : 0.0, red);
  }
  if (tid == 0) {
    const double den = (double)max(total, 1);
    tb *= (double)n / den;
    tz /= den;
    a.stats[0] = (float)(a.coef * tb + a.z_coef * tz);
    a.stats[1] = (float)tb;
    a.stats[2] = (float)tz;
  }
}

BalanceLayout balance_layout(int64_t tokens, int32_t n_experts) {
  (void)tokens;
  BalanceLayout l{};
  l.hist = 0;
  l.sums = ((size_t)BH_GROUPS * ((size_t)n_experts + 1) * 4 + 255) / 256 * 256;
  l.arrive = l.sums + 2 * sizeof(double) * BM_GROUPS;
  l.total = l.arrive + 256;
  return l;
}

namespace {

struct MainLaunch {
  const BalanceArgs &a;
  const int32_t *hist;
  int parts;
  double *sums;
  int32_t *arrive;
  hipStream_t s;
  template <bool BF16, int LANES, int VECS>
  void go() const {
    static_assert(BM_GROUPS <= BM_THREADS, "a thread a workgroup in the last sums");
    const int64_t per = BM_THREADS / LANES;
    const int64_t g = parts ? std::max<int64_t>(1, std::min<int64_t>(BM_GROUPS, (a.tokens + per - 1) / per)) : 1;
    hipLaunchKernelGGL((kb_main<BF16, LANES, VECS>), dim3((unsigned)g), dim3(BM_THREADS), 0, s, a, hist, parts, sums, arrive);
  }
  // the fewest lanes and vectors that hold a token (four bf16 vectors a lane
  // would not fit the 64 registers of a full CU)
  template <bool BF16>
  void choose() const {
    constexpr int N = Elem<BF16>::N;
    const int n = a.n_experts;
    if (n <= 4 * N) go<BF16, 4, 1>();
    else if (n <= 16 * N) go<BF16, 16, 1>();
    else if (n <= 32 * N) go<BF16, 16, 2>();
    else if (n <= 64 * N) go<BF16, BF16 ? 64 : 16, BF16 ? 1 : 4>();
    else go<BF16, 64, BAL_MAX_EXPERTS / (64 * N)>();
  }
};

}  // namespace

hipError_t launch_balance(const BalanceArgs &a, bool bf16, char *ws, hipStream_t s) {
  const BalanceLayout l = balance_layout(a.tokens, a.n_experts);
  int32_t *hist = reinterpret_cast<int32_t *>(ws + l.hist), *arrive = reinterpret_cast<int32_t *>(ws + l.arrive);
  int parts = 0;
  if (a.tokens * std::max(a.n_experts, a.k) > BALANCE_SOLO) {
    parts = (int)std::max<int64_t>(1, std::min<int64_t>(BH_GROUPS, a.tokens * a.k / 2048));
    hipLaunchKernelGGL(kb_count, dim3(parts), dim3(1024), 0, s, a, hist, arrive);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const MainLaunch m{a, hist, parts, reinterpret_cast<double *>(ws + l.sums), arrive, s};
  if (bf16) m.choose<true>();
  else m.choose<false>();
  return hipGetLastError();
}

}  // namespace muon
