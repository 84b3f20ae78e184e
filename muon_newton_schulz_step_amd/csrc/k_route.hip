// A router's choice of experts and its gradient, on gfx950.
//
//   s = softmax(x) or sigmoid(x),  rank = s + bias
//   a group's value = the sum of its `top` best ranks; the `keep` best groups
//   stay, and of their experts the k of best rank are chosen (equal ranks: the
//   lower index first)
//   w_j = scale s_j / (sum of the chosen s + 1e-20), or scale s_j
//
//   d s_j = scale (dw_j - sum_i dw_i s_i / S) / S, or scale dw_j
//   softmax: d x_e = [e chosen] s_e ds_e - s_e sum_j s_j ds_j
//   sigmoid: d x_e = [e chosen] s_e (1 - s_e) ds_e, with 1 - s(x) = s(-x): from
//   an s near 1 the difference keeps few digits, and none from x = 17 on
//
// Ranks are computed in fp32; a token in which two ranks that decide about the
// choice or its order are closer than fp32 tells apart is decided again in
// fp64 (route_exact), so that the choice is that of the definition; so is one
// with a NaN, for which fp32 has no place below its lowest number.  Without a
// bias the logits themselves order the experts, and only fp32 ones that differ
// in the last bits at the border, or in none, are decided again.
//
// Scores and weights are fp32, a weight off by the errors of its scores (as
// tol() below counts them): what takes the weights has no more bits.
//
// Few lanes a token, so that what a choice exchanges stays within a row of
// lanes.  131072 x 256 fp32, 8 of 256 in 4 of 8 groups: the choice 90 to 105 us,
// bound by its comparisons (the bytes take 26), the gradient 42.  A token that
// is decided again takes its whole wave: where all are, as with equal logits,
// the choice takes 730 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "devops.hpp"
#include "layer_ops.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int RT = 256;  // threads of a workgroup
constexpr float NORM_EPS = 1e-20f;
constexpr int QUAD_XOR1 = 0xb1, QUAD_XOR2 = 0x4e, ROW_ROR8 = 0x128, ROW_ROR4 = 0x124;

template <int CTRL>
__device__ __forceinline__ int dpp_i(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ float as_f(int x) { return __int_as_float(x); }

// Reduction over LANES consecutive lanes (4, 16 or 64); every lane gets it.
template <int LANES, class F>
__device__ __forceinline__ float reduce_f(float v, F f) {
  v = f(v, as_f(dpp_i<QUAD_XOR1>(__float_as_int(v))));
  v = f(v, as_f(dpp_i<QUAD_XOR2>(__float_as_int(v))));
  if constexpr (LANES >= 16) {
    v = f(v, as_f(dpp_i<ROW_ROR8>(__float_as_int(v))));
    v = f(v, as_f(dpp_i<ROW_ROR4>(__float_as_int(v))));
  }
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ int reduce_min(int v) {
  v = min(v, dpp_i<QUAD_XOR1>(v));
  v = min(v, dpp_i<QUAD_XOR2>(v));
  if constexpr (LANES >= 16) {
    v = min(v, dpp_i<ROW_ROR8>(v));
    v = min(v, dpp_i<ROW_ROR4>(v));
  }
  if constexpr (LANES == 64) {
    v = min(v, __shfl_xor(v, 16));
    v = min(v, __shfl_xor(v, 32));
  }
  return v;
}
// Sum over LANES consecutive lanes; every lane gets it.
template <int LANES>
__device__ __forceinline__ double add_up(double v) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) v += shfl_xor_f64(v, d);
  return v;
}
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// of a row's sum; a row of -inf has none
__device__ __forceinline__ float inverse(float s) { return s == 0.f ? 0.f : 1.f / s; }
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + exp_term(0.f, x)); }  // exp(0 - x)
// for ranks: two steps of fp32 off at most
__device__ __forceinline__ float sigmoid_fast(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e)); }

// Ranks as whole numbers of the same order, and back.
__device__ __forceinline__ uint32_t sortable(float r) {
  const uint32_t b = __float_as_uint(r);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unsorted(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
template <int LANES>
__device__ __forceinline__ uint32_t reduce_max_u(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<QUAD_XOR1>((int)v));
  v = max(v, (uint32_t)dpp_i<QUAD_XOR2>((int)v));
  if constexpr (LANES >= 16) {
    v = max(v, (uint32_t)dpp_i<ROW_ROR8>((int)v));
    v = max(v, (uint32_t)dpp_i<ROW_ROR4>((int)v));
  }
  if constexpr (LANES == 64) {
    v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    v = max(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}

// Descending order, by Batcher's merges of odd and even places.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = max(a, b);
            v[i + j + k] = min(a, b);
          }
}

template <bool BF16>
__device__ __forceinline__ float logit(const RouteArgs &a, int64_t t, int e) {
  typedef typename Elem<BF16>::type T;
  return Elem<BF16>::get(static_cast<const T *>(a.logits)[t * a.ld + e]);
}

// rank as it is compared: -inf is never chosen, and a zero has no sign (tokens with a NaN are decided in fp64)
__device__ __forceinline__ float orderly(float r) { return r != r ? kLowest : r + 0.f; }
// In fp64 there is room below every fp32 rank, and below the sum of two.
constexpr double kNanRank = -1e39;

// Whether the logits order the experts: without a bias, as far as no ranks are added up.
__device__ __forceinline__ bool ranked_by_logit(const RouteArgs &a) { return !a.bias && (a.groups == 1 || a.top == 1); }

// A token's choice in fp64, by a whole wave: expert e belongs to lane e % 64,
// its rank to rank[e] in LDS.  Writes k experts (-1 where there are no more)
// to chosen.
template <bool BF16>
__device__ __forceinline__ void route_exact(const RouteArgs &a, int64_t t, double *rank, int32_t *chosen) {
  const int lane = threadIdx.x & 63;
  const double ninf = -INFINITY;
  auto wave_max = [](double v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = fmax(v, shfl_xor_f64(v, m));
    return v;
  };
  double top = ninf, total = 0.0;
  for (int e = lane; e < a.experts; e += 64) {
    rank[e] = (double)logit<BF16>(a, t, e);
    top = fmax(top, rank[e]);
  }
  top = wave_max(top);
  const bool by_logit = ranked_by_logit(a);
  // exp(x - max) for the softmax, exp(-x) for the sigmoid
  for (int e = lane; e < a.experts; e += 64) {
    if (by_logit) {
      if (rank[e] != rank[e]) rank[e] = kNanRank;
      continue;
    }
    const double x = rank[e];
    if (x == ninf) continue;
    const double y = exp(a.softmax ? x - top : -x);
    total += y;
    rank[e] = a.softmax ? y : 1.0 / (1.0 + y);
  }
  if (a.softmax) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) total += shfl_xor_f64(total, m);
  } else {
    total = 1.0;
  }
  for (int e = lane; e < a.experts; e += 64) {
    if (rank[e] == ninf || by_logit) continue;
    const double b = a.bias ? (double)a.bias[e] : 0.0, r = rank[e] / total + b;
    rank[e] = b == ninf ? ninf : r != r ? kNanRank : r;
  }
  // the best rank in [lo, hi) but for expert `but`, and the expert (or INT_MAX)
  auto best = [&](int lo, int hi, int but, double &v) {
    double m = ninf;
    int at = INT32_MAX;
    for (int e = lane; e < hi; e += 64)
      if (e >= lo && e != but && rank[e] > m) {
        m = rank[e];
        at = e;
      }
    v = wave_max(m);
    at = m == v ? at : INT32_MAX;
#pragma unroll
    for (int q = 32; q > 0; q >>= 1) at = min(at, __shfl_xor(at, q));
    return at;
  };
  if (a.groups > 1) {
    const int size = a.experts / a.groups;
    double value = ninf;  // of group `lane`
    for (int g = 0; g < a.groups; ++g) {
      double v1, v2;
      const int e = best(g * size, (g + 1) * size, -1, v1);
      if (a.top > 1 && best(g * size, (g + 1) * size, e, v2) != INT32_MAX) v1 += v2;
      if (lane == g) value = v1;
    }
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double v = shfl_f64(value, g);
      before += v > value || (v == value && g < lane);
    }
    const uint64_t open = __ballot(lane < a.groups && before < a.keep);
    for (int e = lane; e < a.experts; e += 64)
      if (!(open >> (e / size) & 1)) rank[e] = ninf;
  }
  for (int j = 0; j < a.k; ++j) {
    double v;
    const int e = best(0, a.experts, -1, v);
    if (lane == 0) chosen[j] = e == INT32_MAX ? -1 : e;
    if (e != INT32_MAX && (e & 63) == lane) rank[e] = ninf;
  }
}

// LANES lanes take a token, V consecutive experts a lane.
template <bool BF16, int LANES, int V>
__global__ __launch_bounds__(RT) void kr_route(RouteArgs a) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int PER = RT / LANES, N = E::N < V ? E::N : V;
  __shared__ int32_t chosen[PER][ROUTE_MAX_CHOICES + 1];
  __shared__ double exact[RT / 64][LANES * V];
  const int l = threadIdx.x & (LANES - 1), slot = threadIdx.x / LANES;
  const int64_t t = (int64_t)blockIdx.x * PER + slot;
  const bool in = t < a.tokens;
  const bool ok = in && (!a.valid || a.valid[t]);
  const int e0 = l * V;
  const bool by_logit = ranked_by_logit(a);
  float r[V];
  {
    const T *x = static_cast<const T *>(a.logits) + (ok ? t : 0) * a.ld + e0;
#pragma unroll
    for (int i = 0; i < V; i += N) {
      if (ok && N == E::N && e0 + i + N <= a.experts) {
        E::unpack(load16(x + i), r + i);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) r[i + j] = ok && e0 + i + j < a.experts ? E::get(x[i + j]) : -INFINITY;
      }
    }
  }
  float m = 0.f, inv = 0.f;  // softmax: the row's maximum, 1 / sum
  if (a.softmax) {
    m = kLowest;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, r[i]);
    m = reduce_f<LANES>(m, Max());
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += exp_term(r[i], m);
    inv = inverse(reduce_f<LANES>(s, Sum()));
  }
  if (!by_logit) {
    float b[V];
    if (a.bias && e0 + V <= a.experts) {
#pragma unroll
      for (int i = 0; i < V; i += 4) Elem<false>::unpack(load16(a.bias + e0 + i), b + i);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = a.bias && e0 + i < a.experts ? a.bias[e0 + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = a.softmax ? exp_term(r[i], m) * inv : sigmoid_fast(r[i]);
      r[i] = r[i] == -INFINITY ? r[i] : s + b[i];
    }
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    nan |= r[i] != r[i];
    r[i] = orderly(r[i]);
  }
  // of lane 0: whether the token is decided again in fp64
  bool close = __ballot(nan) >> (threadIdx.x & 63 & ~(LANES - 1)) & (LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1);
  // What a score may be off by, in units of 2^-24: an exponential of d carries |d| + 4 of itself, which moves a
  // sigmoid by at most 5 in all; a softmax's sum carries sum p (|d| + 2) <= 7 + 2 for 1024 experts, at most 22 for
  // its additions and 4 for the quotient and the product, its term s (|d| + 2) < 3.  The bias adds a rounding of
  // the rank.  Twice that for the difference of two ranks, twice again for values that are sums of two.
  auto tol = [&](float rank) { return by_logit ? 0.f : (40.f + fabsf(rank)) * (4.f * 5.9604645e-8f); };
  if (a.groups > 1) {
    const int size = a.experts / a.groups, span = size / V;  // lanes of a group
    if (LANES >= 16 && size % V == 0 && (span & (span - 1)) == 0) {
      // a lane's experts are of one group: its two best, joined over the group's lanes
      float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v2 = fmaxf(v2, fminf(v1, r[i]));
        v1 = fmaxf(v1, r[i]);
      }
      for (int d = 1; d < span; d <<= 1) {
        const float o1 = __shfl_xor(v1, d), o2 = __shfl_xor(v2, d);
        v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
        v1 = fmaxf(v1, o1);
      }
      const float value = a.top > 1 && v2 != -INFINITY ? fmaxf(v1 + v2, kLowest) : v1;
      // groups before this lane's
      const int g = l / span, first = (int)(threadIdx.x & 63) - l;
      int before = 0;
      for (int q = 1; q < a.groups; ++q) {
        const int h = g + q < a.groups ? g + q : g + q - a.groups;
        const float o = __shfl(value, first + (h & (LANES - 1)) * span);
        before += o > value || (o == value && h < g);
      }
      const bool kept = g < a.groups && before < a.keep;
      if (!by_logit) {
        const float in_ = -reduce_f<LANES>(kept && value != -INFINITY ? -value : -INFINITY, Max());
        const float out = reduce_f<LANES>(g < a.groups && !kept ? value : -INFINITY, Max());
        if (out != -INFINITY && in_ - out <= tol(in_)) close = true;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) r[i] = kept ? r[i] : -INFINITY;
    } else {
      // every lane goes through the groups' values, group by group
      uint32_t open = 0;
      float value[ROUTE_MAX_GROUPS / 4];  // of group l + LANES i, i < groups / LANES
#pragma unroll
      for (int i = 0; i < ROUTE_MAX_GROUPS / 4; ++i) value[i] = -INFINITY;
      for (int g = 0; g < a.groups; ++g) {
        const int lo = g * size - e0, hi = lo + size;
        float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = i >= lo && i < hi ? r[i] : -INFINITY;
          v2 = fmaxf(v2, fminf(v1, x));
          v1 = fmaxf(v1, x);
        }
        const float best = reduce_f<LANES>(v1, Max());
        if (a.top > 1) {
          // the second: of the lane that holds the best, its second; of the others, their first
          const int who = reduce_min<LANES>(v1 == best ? l : LANES);
          const float second = reduce_f<LANES>(l == who ? v2 : v1, Max());
          v1 = second == -INFINITY ? best : fmaxf(best + second, kLowest);
        } else {
          v1 = best;
        }
#pragma unroll
        for (int i = 0; i < ROUTE_MAX_GROUPS / 4; ++i)
          if (g == l + LANES * i) value[i] = v1;
      }
      // the `keep` best, one at a time; the first that stays outside tells how close it was
      float last = INFINITY;
      for (int q = 0; q <= a.keep && q < a.groups; ++q) {
        float v = -INFINITY;
#pragma unroll
        for (int i = 0; i < ROUTE_MAX_GROUPS / 4; ++i) v = fmaxf(v, value[i]);
        const float best = reduce_f<LANES>(v, Max());
        if (q == a.keep) {
          close |= !by_logit && last - best <= tol(last);
          break;
        }
        last = best;
        int at = INT32_MAX;
#pragma unroll
        for (int i = ROUTE_MAX_GROUPS / 4 - 1; i >= 0; --i)
          if (value[i] == best && best != -INFINITY) at = l + LANES * i;
        at = reduce_min<LANES>(at);
        if (at == INT32_MAX) break;
        open |= 1u << at;
#pragma unroll
        for (int i = 0; i < ROUTE_MAX_GROUPS / 4; ++i)
          if (l + LANES * i == at) value[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!(open >> min((e0 + i) / size, 31) & 1)) r[i] = -INFINITY;
    }
  }
  bool done = false;
  if constexpr (LANES >= 16) {
    if (a.k + 2 <= LANES) {
      // The k + 2 best by keys whose low bits are replaced by the expert: each
      // lane sorts its own, then the best of the lanes' first ones is taken,
      // time and again.  What the bits left out decide is settled among the
      // chosen by their full ranks.
      constexpr uint32_t LOW = LANES * V - 1;
      static_assert((LANES * V & LOW) == 0, "a power of two");
      uint32_t key[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t there = r[i] == -INFINITY ? 0u : ~0u;
        key[i] = ((sortable(r[i]) & ~LOW) | (LOW - (uint32_t)(e0 + i))) & there;
      }
      sort_down(key);
      uint32_t mine = 0, least = 0;  // the lane's one of them, and the last
      for (int j = 0; j < a.k + 2; ++j) {
        const uint32_t best = reduce_max_u<LANES>(key[0]);
        if (l == j) mine = best;
        least = best;
        // (a choice between neighbours would become an index, and that a chain of comparisons)
        const uint32_t won = key[0] == best ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = (key[i + 1] & won) | (key[i] & ~won);
        key[V - 1] &= ~won;
      }
      const int e = mine ? (int)(LOW - (mine & LOW)) : -1;
      float x = -INFINITY, bias = 0.f, rank = -INFINITY;
      if (e >= 0) {
        x = logit<BF16>(a, t, e);
        if (a.bias) bias = a.bias[e];
        rank = orderly(by_logit ? x : (a.softmax ? exp_term(x, m) * inv : sigmoid_fast(x)) + bias);
      }
      int place = 0;
      bool near = false;
      const int first = (int)(threadIdx.x & 63) - l;
      for (int j = 0; j < a.k + 2; ++j) {
        const float o = __shfl(rank, first + j);
        const int f = __shfl(e, first + j);
        const bool other = f >= 0 && f != e;
        place += other && (o > rank || (o == rank && f < e));
        if (!by_logit) {
          const bool same = __shfl(x, first + j) == x && __shfl(bias, first + j) == bias;  // equal by their inputs
          near |= other && !same && fabsf(o - rank) <= tol(rank);
        }
      }
      if (l < a.k) chosen[slot][l] = -1;
      __builtin_amdgcn_wave_barrier();
      if (e >= 0 && place < a.k) chosen[slot][place] = e;
      // close: a rank near that of another of them, or near what may lie outside
      const float kth = -reduce_f<LANES>(e >= 0 && place < a.k ? -rank : -INFINITY, Max());
      const bool exact_keys = by_logit && BF16;
      if (least != 0 && !exact_keys && !(kth - unsorted(least | LOW) > tol(kth))) close = true;
      if (reduce_f<LANES>(e >= 0 && near && place < a.k ? 1.f : 0.f, Max()) != 0.f) close = true;
      done = true;
    }
  }
  if (!done) {
    // the k best, one at a time, and the first that stays outside
    float last = INFINITY;
    for (int j = 0; j <= a.k; ++j) {
      if (j == a.k && by_logit) break;
      float v = r[0];
#pragma unroll
      for (int i = 1; i < V; ++i) v = fmaxf(v, r[i]);
      const float best = reduce_f<LANES>(v, Max());
      if (!by_logit && best != -INFINITY && last - best <= tol(best)) close = true;
      last = best;
      if (j == a.k) break;
      int at = INT32_MAX;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (r[i] == best && best != -INFINITY) at = e0 + i;
      at = reduce_min<LANES>(at);
      if (l == 0) chosen[slot][j] = at == INT32_MAX ? -1 : at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i == at) r[i] = -INFINITY;
    }
  }
  uint64_t redo = __ballot(close && ok && l == 0);
  while (redo) {
    const int lane = __ffsll((unsigned long long)redo) - 1;
    redo &= redo - 1;
    const int who = (threadIdx.x & ~63) / LANES + lane / LANES;
    route_exact<BF16>(a, (int64_t)blockIdx.x * PER + who, exact[threadIdx.x >> 6], chosen[who]);
  }
  __builtin_amdgcn_wave_barrier();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  if (!in) return;
  float sum = 0.f, s[(ROUTE_MAX_CHOICES + LANES - 1) / LANES];
  int e[(ROUTE_MAX_CHOICES + LANES - 1) / LANES];
#pragma unroll
  for (int q = 0; q < (ROUTE_MAX_CHOICES + LANES - 1) / LANES; ++q) {
    const int j = l + LANES * q;
    e[q] = ok && j < a.k ? chosen[slot][j] : -1;
    s[q] = 0.f;
    if (e[q] >= 0) {
      const float x = logit<BF16>(a, t, e[q]);
      s[q] = a.softmax ? exp_term(x, m) * inv : sigmoid(x);
    }
    sum += s[q];
  }
  sum = reduce_f<LANES>(sum, Sum());
  const float f = a.renormalize ? a.scale / (sum + NORM_EPS) : a.scale;
#pragma unroll
  for (int q = 0; q < (ROUTE_MAX_CHOICES + LANES - 1) / LANES; ++q) {
    const int j = l + LANES * q;
    if (j >= a.k) continue;
    const int64_t at = t * a.k + j;
    if (a.choices.is64) static_cast<int64_t *>(const_cast<void *>(a.choices.p))[at] = e[q];
    else static_cast<int32_t *>(const_cast<void *>(a.choices.p))[at] = e[q];
    a.weights[at] = e[q] >= 0 ? s[q] * f : 0.f;
  }
}

// LANES lanes take a token, VECS 16-byte vectors a lane, and the choices a lane
// each, in up to Q rounds.
//
// Where one score holds nearly all of a sum, what the gradient is made of
// cancels: dw_j against the mean of dw, ds_e against sum_j s_j ds_j.  Sums and
// differences of the chosen are in fp64, on scores whose own error is a factor
// (softmax: exponentials over their sum in fp64), so that only the factors'
// errors are left; in fp32 a score of 1 - 1e-6 left 6% of error.
template <bool BF16, int LANES, int VECS, int Q>
__global__ __launch_bounds__(RT) void kr_backward(RouteArgs a) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int PER = RT / LANES, N = E::N;
  const int l = threadIdx.x & (LANES - 1), lane0 = (int)(threadIdx.x & 63) - l;
  const int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / LANES;
  const bool in = t < a.tokens;
  const bool ok = in && (!a.valid || a.valid[t]);
  const int64_t row = ok ? t : 0;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  float v[VECS][N];
  float m = 0.f;
  double inv = 0.0;
  if (a.softmax) {
    m = kLowest;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = (l + LANES * i) * N;
      if (ok && c + N <= a.experts) {
        E::unpack(load16(x + c), v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = ok && c + j < a.experts ? E::get(x[c + j]) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, v[i][j]);
    }
    m = reduce_f<LANES>(m, Max());
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] = exp_term(v[i][j], m);
        s += (double)v[i][j];
      }
    s = add_up<LANES>(s);
    inv = s == 0.0 ? 0.0 : 1.0 / s;
  }
  // the chosen experts' scores, their sum S and sum_i dw_i s_i
  int e[Q];
  float dw[Q];
  double s[Q], total = 0.0, dot = 0.0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int j = l + LANES * q;
    e[q] = -1;
    dw[q] = 0.f;
    s[q] = 0.0;
    if (ok && j < a.k) {
      const int64_t c = index_at(a.choices, t * a.k + j);
      if (c >= 0 && c < a.experts) {
        e[q] = (int)c;
        const float z = E::get(x[e[q]]);
        s[q] = a.softmax ? (double)exp_term(z, m) * inv : (double)sigmoid(z);
        dw[q] = a.dweights[t * a.k + j];
        dot += (double)dw[q] * s[q];
      }
    }
    total += s[q];
  }
  total = add_up<LANES>(total);
  dot = add_up<LANES>(dot);
  const double over = a.renormalize ? 1.0 / (total + (double)NORM_EPS) : 1.0;  // 1 / S
  const double f = (double)a.scale * over;
  const double mean = a.renormalize ? dot * over : 0.0;
  // sum_j s_j ds_j; renormalised it is scale / S dot (1 - total / S), all but 0
  const double inner = !a.softmax ? 0.0 : a.renormalize ? f * dot * ((double)NORM_EPS * over) : f * dot;
  // what a choice gives its expert: the whole element, or where an earlier
  // choice is the same expert what it adds to that
  float whole[Q], more[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const double ds = f * ((double)dw[q] - mean);
    if (a.softmax) {
      whole[q] = (float)(s[q] * (ds - inner));
      more[q] = (float)(s[q] * ds);
    } else {
      whole[q] = more[q] = e[q] >= 0 ? (float)(s[q] * (double)sigmoid(-E::get(x[e[q]])) * ds) : 0.f;
    }
  }
  const float part = (float)(inv * inner);
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) v[i][j] = a.softmax ? -v[i][j] * part : 0.f;
  uint32_t again = 0;  // of this lane's choices, those whose expert has come before
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    for (int u = 0; u < LANES && u + LANES * q < a.k; ++u) {
      const bool second = again >> q & 1;
      const int c = __shfl(second ? -2 - e[q] : e[q], lane0 + u);  // -1: none; below: second
      const float add = __shfl(second ? more[q] : whole[q], lane0 + u);
      if (c != -1) {
        const int which = c < 0 ? -2 - c : c;
#pragma unroll
        for (int p = 0; p < Q; ++p)
          if (e[p] == which && (p > q || (p == q && l > u))) again |= 1u << p;
        const int at = which - l * N;
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (at == LANES * N * i + j) v[i][j] = c < 0 ? v[i][j] + add : add;
      }
    }
  }
  if (!in) return;
  T *d = static_cast<T *>(a.dlogits) + t * a.dld;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (l + LANES * i) * N;
    if (!ok) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = 0.f;
    }
    if (c + N <= a.experts) {
      if (!a.first) {
        if (!ok) continue;
        float w[N];
        E::unpack(load16(d + c), w);
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] += w[j];
        store16(d + c, E::pack(v[i]));
      } else {
        stream16(d + c, E::pack(v[i]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j < a.experts && (a.first || ok)) d[c + j] = E::put(a.first ? v[i][j] : E::get(d[c + j]) + v[i][j]);
    }
  }
}

// Calls launch(args, workgroups) for as many tokens at a time as a grid of
// below 2^32 threads takes, LANES a token.
template <bool BF16, int LANES, class F>
hipError_t in_grids(RouteArgs a, F launch) {
  constexpr int PER = RT / LANES;
  constexpr int64_t MOST = (((int64_t)1 << 32) / RT - 1) * PER;
  const int64_t e = sizeof(typename Elem<BF16>::type), ids = (a.choices.is64 ? 8 : 4) * (int64_t)a.k;
  auto on = [](auto &p, int64_t bytes) {
    if (p) p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(reinterpret_cast<uintptr_t>(p) + bytes);
  };
  for (int64_t left = a.tokens;; left -= MOST) {
    a.tokens = std::min(left, MOST);
    launch(a, (unsigned)((a.tokens + PER - 1) / PER));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || left <= MOST) return err;  // (behind the last one a row stride may be any)
    on(a.logits, MOST * a.ld * e);
    on(a.valid, MOST);
    on(a.choices.p, MOST * ids);
    on(a.weights, MOST * a.k * 4);
    on(a.dweights, MOST * a.k * 4);
    on(a.dlogits, MOST * a.dld * e);
  }
}

template <bool BF16>
hipError_t route(const RouteArgs &a, hipStream_t s) {
  auto go = [&](auto lanes, auto per) {
    constexpr int L = decltype(lanes)::value, V = decltype(per)::value;
    return in_grids<BF16, L>(a, [&](const RouteArgs &b, unsigned grid) {
      hipLaunchKernelGGL((kr_route<BF16, L, V>), dim3(grid), dim3(RT), 0, s, b);
    });
  };
  typedef std::integral_constant<int, 4> c4;
  typedef std::integral_constant<int, 8> c8;
  typedef std::integral_constant<int, 16> c16;
  typedef std::integral_constant<int, 64> c64;
  const int n = a.experts;
  if (n <= 16) return go(c4(), c4());
  if (n <= 32) return go(c4(), c8());
  if (n <= 64) return go(c16(), c4());
  if (n <= 128) return go(c16(), c8());
  if (n <= 256) return go(c16(), c16());
  if (n <= 512) return go(c64(), c8());
  return go(c64(), c16());
}

template <bool BF16>
hipError_t route_backward(const RouteArgs &a, hipStream_t s) {
  auto go = [&](auto lanes, auto per) {
    constexpr int L = decltype(lanes)::value, V = decltype(per)::value;
    // 131072 x 8 bf16 logits: 10 us with every round there may be, 7.5 with one
    constexpr int ALL = (ROUTE_MAX_CHOICES + L - 1) / L;
    return in_grids<BF16, L>(a, [&](const RouteArgs &b, unsigned grid) {
      if (ALL == 1 || a.k <= L) hipLaunchKernelGGL((kr_backward<BF16, L, V, 1>), dim3(grid), dim3(RT), 0, s, b);
      else hipLaunchKernelGGL((kr_backward<BF16, L, V, ALL>), dim3(grid), dim3(RT), 0, s, b);
    });
  };
  constexpr int N = Elem<BF16>::N;
  typedef std::integral_constant<int, 1> c1;
  typedef std::integral_constant<int, 2> c2;
  typedef std::integral_constant<int, 4> c4;
  typedef std::integral_constant<int, 16> c16;
  typedef std::integral_constant<int, 64> c64;
  const int n = a.experts;
  if (n <= 4 * N) return go(c4(), c1());
  if (n <= 16 * N) return go(c16(), c1());
  if (n <= 32 * N) return go(c16(), c2());
  if (n <= 64 * N) return go(c16(), c4());
  return go(c64(), std::integral_constant<int, ROUTE_MAX_EXPERTS / (64 * N)>());
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  return bf16 ? route<true>(a, s) : route<false>(a, s);
}

hipError_t launch_route_backward(const RouteArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  return bf16 ? route_backward<true>(a, s) : route_backward<false>(a, s);
}

}  // namespace muon
