// The order of a layer's tokens by expert, and the weighted sum of what the
// experts return with its gradients, on gfx950.
//
// Order: a stable counting sort of the tokens * k choices by expert.  The
// choices are cut into parts; each part is counted by one wave into LDS, the
// counts are summed over the parts expert by expert, and each part's wave then
// walks its choices 64 at a time: a choice's slot is its expert's next free one
// plus the number of lanes before it with the same expert, found by comparing
// the experts' bits across the wave (a ballot a bit).  Nothing depends on the
// order in which workgroups run.  Bound by latency: a few dependent passes over
// some hundred KB (131072 choices of 256 experts: 4.8 + 5.3 + 7.6 us).
//
// Sum: out[t] = residual[t] + sum_j w[t][j] y[place[t][j]], in fp32, j by j,
// rounded once.  Bound by HBM: every row of y is read once (16384 x 8 rows of
// 4096 bf16: 240 us, 5.0 TB/s; the gradients 449).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "devops.hpp"
#include "layer_ops.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int OW = 4;            // waves of a workgroup, a part each
constexpr int OP = 1024;         // parts, at most (a multiple of 64)
constexpr int SOLO_WAVES = 16;
// Up to so many choices one workgroup does the whole call: 8192 of 64 experts
// take 11.7 us, 16384 20.3; three launches 13 of either.
constexpr int64_t ORDER_SOLO = 8192;
constexpr int SOLO_EXPERTS = 512;      // and up to so many experts (its counts are 32 KB of LDS)

__device__ __forceinline__ int expert_at(const OrderArgs &a, int64_t i) {
  const int64_t e = index_at(a.choices, i);
  return e >= 0 && e < a.experts ? (int)e : -1;
}

// Lanes of the wave whose expert is this lane's (of lanes with e >= 0).
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t m = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot(e >> b & 1);
    m &= (e >> b & 1) ? set : ~set;
  }
  return m;
}

// Counts choices [i0, i1) into h, in LDS, by one wave.
__device__ __forceinline__ void count_part(const OrderArgs &a, int64_t i0, int64_t i1, int *h) {
  const int lane = threadIdx.x & 63;
#pragma unroll 4
  for (int64_t i = i0 + lane; i < i1; i += 64) {
    const int e = expert_at(a, i);
    if (e >= 0) atomicAdd(&h[e], 1);
  }
}

// Gives choices [i0, i1) their slots, by one wave; next[e], in LDS, is the
// expert's next free one.
__device__ __forceinline__ void place_part(const OrderArgs &a, int64_t i0, int64_t i1, int bits, int *next) {
  const int lane = threadIdx.x & 63;
  int e = i0 + lane < i1 ? expert_at(a, i0 + lane) : -1;
  for (int64_t i = i0 + lane; i - lane < i1; i += 64) {
    const int ahead = i + 64 < i1 ? expert_at(a, i + 64) : -1;
    const uint64_t same = same_expert(e, bits);
    const int before = __popcll(same & ((1ull << lane) - 1));
    int slot = -1;
    if (e >= 0) {
      slot = next[e] + before;
      a.tokens[slot] = (int32_t)(i / a.k);
    }
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && before == 0) next[e] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < i1) a.place[i] = slot;
    e = ahead;
  }
}

// Exclusive sum over the workgroup's threads, THREADS of them; red holds a
// number a wave.  total: the sum of all.
template <int THREADS>
__device__ __forceinline__ int scan_threads(int v, int *red, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) red[wave] = x;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) base += red[w];
    all += red[w];
  }
  *total = all;
  __syncthreads();
  return base + x - v;
}

}  // namespace

// The whole call by one workgroup of SOLO_WAVES waves, a part a wave.
__global__ __launch_bounds__(SOLO_WAVES * 64) void ko_solo(OrderArgs a, int bits) {
  extern __shared__ int h[];  // [SOLO_WAVES][experts]
  __shared__ int red[SOLO_WAVES];
  const int wave = threadIdx.x >> 6, x = a.experts;
  for (int i = threadIdx.x; i < SOLO_WAVES * x; i += SOLO_WAVES * 64) h[i] = 0;
  __syncthreads();
  const int64_t i0 = a.n * wave / SOLO_WAVES, i1 = a.n * (wave + 1) / SOLO_WAVES;
  count_part(a, i0, i1, h + wave * x);
  __syncthreads();
  const int e = threadIdx.x;
  int sum = 0, all;
  if (e < x)
    for (int w = 0; w < SOLO_WAVES; ++w) sum += h[w * x + e];
  int at = scan_threads<SOLO_WAVES * 64>(sum, red, &all);
  if (e < x) {
    a.offsets[e] = at;
    if (e == 0) a.offsets[x] = all;
    for (int w = 0; w < SOLO_WAVES; ++w) {
      const int c = h[w * x + e];
      h[w * x + e] = at;
      at += c;
    }
  }
  __syncthreads();
  place_part(a, i0, i1, bits, h + wave * x);
  for (int64_t i = all + (int64_t)threadIdx.x; i < a.n; i += SOLO_WAVES * 64) a.tokens[i] = -1;
}

// hist[part][e]
__global__ __launch_bounds__(OW * 64) void ko_count(OrderArgs a, int32_t *hist, int parts) {
  extern __shared__ int h[];  // [OW][experts]
  const int wave = threadIdx.x >> 6, x = a.experts, part = blockIdx.x * OW + wave;
  for (int i = threadIdx.x; i < OW * x; i += OW * 64) h[i] = 0;
  __syncthreads();
  count_part(a, a.n * part / parts, a.n * (part + 1) / parts, h + wave * x);
  __syncthreads();
  for (int i = threadIdx.x; i < OW * x; i += OW * 64) hist[(int64_t)blockIdx.x * OW * x + i] = h[i];
}

// A workgroup takes 16 experts: 64 threads an expert, parts / 64 parts a
// thread.  hist becomes the sum over the parts before, totals[e] over all.
__global__ __launch_bounds__(1024) void ko_scan(int32_t *hist, int32_t *totals, int parts, int experts) {
  __shared__ int red[16][65];
  const int ei = threadIdx.x & 15, seg = threadIdx.x >> 4, e = blockIdx.x * 16 + ei, per = parts / 64;
  int c[OP / 64], sum = 0;
#pragma unroll
  for (int q = 0; q < OP / 64; ++q) {
    c[q] = q < per && e < experts ? hist[(int64_t)(seg * per + q) * experts + e] : 0;
    sum += c[q];
  }
  red[ei][seg] = sum;
  __syncthreads();
  int base = 0;
  for (int s = 0; s < seg; ++s) base += red[ei][s];
  if (e >= experts) return;
  if (seg == 63) totals[e] = base + sum;
#pragma unroll
  for (int q = 0; q < OP / 64; ++q)
    if (q < per) {
      hist[(int64_t)(seg * per + q) * experts + e] = base;
      base += c[q];
    }
}

__global__ __launch_bounds__(OW * 64) void ko_place(OrderArgs a, const int32_t *hist, const int32_t *totals, int parts,
                                                    int bits) {
  extern __shared__ int h[];  // [OW][experts]
  __shared__ int red[OW];
  const int wave = threadIdx.x >> 6, x = a.experts;
  constexpr int PER = ROUTE_MAX_EXPERTS / (OW * 64);
  // the experts' first slots
  int t[PER], sum = 0, all;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = (int)threadIdx.x * PER + q;
    t[q] = e < x ? totals[e] : 0;
    sum += t[q];
  }
  int at = scan_threads<OW * 64>(sum, red, &all);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = (int)threadIdx.x * PER + q;
    if (e < x) {
#pragma unroll
      for (int w = 0; w < OW; ++w) h[w * x + e] = at + hist[((int64_t)blockIdx.x * OW + w) * x + e];
      if (blockIdx.x == 0) a.offsets[e] = at;
    }
    at += t[q];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[x] = all;
  __syncthreads();
  const int64_t part = (int64_t)blockIdx.x * OW + wave;
  place_part(a, a.n * part / parts, a.n * (part + 1) / parts, bits, h + wave * x);
  for (int64_t i = all + (int64_t)blockIdx.x * (OW * 64) + threadIdx.x; i < a.n; i += (int64_t)gridDim.x * (OW * 64))
    a.tokens[i] = -1;
}

OrderLayout order_layout(int64_t n, int32_t experts) {
  (void)n;
  OrderLayout l{};
  l.hist = 0;
  l.totals = ((size_t)OP * (size_t)experts * 4 + 255) / 256 * 256;
  l.total = l.totals + ROUTE_MAX_EXPERTS * 4;
  return l;
}

hipError_t launch_order(const OrderArgs &a, char *ws, hipStream_t s) {
  const OrderLayout l = order_layout(a.n, a.experts);
  int32_t *hist = reinterpret_cast<int32_t *>(ws + l.hist), *totals = reinterpret_cast<int32_t *>(ws + l.totals);
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  if (a.n <= ORDER_SOLO && a.experts <= SOLO_EXPERTS) {
    hipLaunchKernelGGL(ko_solo, dim3(1), dim3(SOLO_WAVES * 64), SOLO_WAVES * a.experts * 4, s, a, bits);
    return hipGetLastError();
  }
  // parts of 256 choices and more, a multiple of 64
  const int parts = (int)std::min<int64_t>(OP, std::max<int64_t>(1, a.n / 256 / 64) * 64);
  const int groups = parts / OW, lds = OW * a.experts * 4;
  hipLaunchKernelGGL(ko_count, dim3(groups), dim3(OW * 64), lds, s, a, hist, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(ko_scan, dim3((a.experts + 15) / 16), dim3(1024), 0, s, hist, totals, parts, a.experts);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(ko_place, dim3(groups), dim3(OW * 64), lds, s, a, hist, totals, parts, bits);
  return hipGetLastError();
}

// ------------------------------------------------------------------- sum

namespace {

constexpr int CT = 256;  // threads of a workgroup
constexpr int CK = 8;    // rows of y under way together

}  // namespace

// A thread takes one 16-byte vector of one token; a workgroup takes CT
// consecutive ones of the tokens' rows laid end to end.
template <bool BF16>
__global__ __launch_bounds__(CT) void kc_combine(CombineArgs a, int64_t vecs) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N;
  const int64_t id = (int64_t)blockIdx.x * CT + threadIdx.x;
  const int64_t t = id / vecs;
  if (t >= a.tokens) return;
  const int64_t c = (id - t * vecs) * N;
  const int n = (int)lesser(N, a.dim - c);
  const T *y = static_cast<const T *>(a.y) + c;
  float sum[N];
#pragma unroll
  for (int q = 0; q < N; ++q) sum[q] = 0.f;
  for (int64_t j0 = 0; j0 < a.k; j0 += CK) {
    uint4 v[CK];
    float w[CK];
    bool has[CK];
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const int64_t at = t * a.k + j0 + j;
      const int64_t row = j0 + j < a.k ? a.place[at] : -1;
      has[j] = row >= 0 && row < a.rows;
      w[j] = has[j] && a.weights ? a.weights[at] : 1.f;
      if (has[j]) {
        const T *p = y + row * a.yld;
        if (n == N) {
          v[j] = load16(p);
        } else {
          T e[N];
          for (int q = 0; q < N; ++q) e[q] = q < n ? p[q] : T(0);
          __builtin_memcpy(&v[j], e, 16);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < CK; ++j)
      if (has[j]) {
        float f[N];
        E::unpack(v[j], f);
#pragma unroll
        for (int q = 0; q < N; ++q) sum[q] = fmaf(w[j], f[q], sum[q]);
      }
  }
  const T *res = a.residual ? static_cast<const T *>(a.residual) + t * a.rld + c : nullptr;
  T *out = static_cast<T *>(a.out) + t * a.old + c;
  if (n == N) {
    if (res) {
      float f[N];
      E::unpack(load16(res), f);
#pragma unroll
      for (int q = 0; q < N; ++q) sum[q] += f[q];
    }
    store16(out, E::pack(sum));
  } else {
    for (int q = 0; q < n; ++q) out[q] = E::put(res ? sum[q] + E::get(res[q]) : sum[q]);
  }
}

// A wave takes a token: its row of dout is read once, each of its rows of y
// once, each of its rows of dy written once.
template <bool BF16>
__global__ __launch_bounds__(CT) void kc_backward(CombineBwdArgs a) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (CT / 64) + uniform(threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const T *g = static_cast<const T *>(a.dout) + t * a.dold;
  for (int64_t j0 = 0; j0 < a.k; j0 += CK) {
    int64_t row[CK];
    float w[CK], dot[CK];
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const int64_t at = t * a.k + j0 + j;
      const int64_t r = j0 + j < a.k ? a.place[at] : -1;
      row[j] = r >= 0 && r < a.rows ? r : -1;
      w[j] = row[j] >= 0 && a.weights ? a.weights[at] : 1.f;
      dot[j] = 0.f;
    }
    for (int64_t c = lane * N; c < a.dim; c += 64 * N) {
      const int n = (int)lesser(N, a.dim - c);
      float d[N];
      if (n == N) {
        E::unpack(load16(g + c), d);
        uint4 v[CK];
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < CK; ++j)
            if (row[j] >= 0) v[j] = load16(static_cast<const T *>(a.y) + row[j] * a.yld + c);
        }
#pragma unroll
        for (int j = 0; j < CK; ++j) {
          if (row[j] < 0) continue;
          float f[N];
          if (a.dweights) {
            E::unpack(v[j], f);
#pragma unroll
            for (int q = 0; q < N; ++q) dot[j] = fmaf(d[q], f[q], dot[j]);
          }
          if (a.dy) {
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] = w[j] * d[q];
            stream16(static_cast<T *>(a.dy) + row[j] * a.dyld + c, E::pack(f));
          }
        }
      } else {
        for (int q = 0; q < n; ++q) d[q] = E::get(g[c + q]);
#pragma unroll
        for (int j = 0; j < CK; ++j) {
          if (row[j] < 0) continue;
          for (int q = 0; q < n; ++q) {
            if (a.dweights) dot[j] = fmaf(d[q], E::get(static_cast<const T *>(a.y)[row[j] * a.yld + c + q]), dot[j]);
            if (a.dy) static_cast<T *>(a.dy)[row[j] * a.dyld + c + q] = E::put(w[j] * d[q]);
          }
        }
      }
    }
    if (a.dweights) {
#pragma unroll
      for (int j = 0; j < CK; ++j) {
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) dot[j] += __shfl_xor(dot[j], m);
        if (lane == 0 && j0 + j < a.k) a.dweights[t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

hipError_t launch_combine(const CombineArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t n = bf16 ? 8 : 4, vecs = (a.dim + n - 1) / n;
  const int64_t grid = (a.tokens * vecs + CT - 1) / CT;
  if (bf16) hipLaunchKernelGGL(kc_combine<true>, dim3((unsigned)grid), dim3(CT), 0, s, a, vecs);
  else hipLaunchKernelGGL(kc_combine<false>, dim3((unsigned)grid), dim3(CT), 0, s, a, vecs);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineBwdArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t grid = (a.tokens + CT / 64 - 1) / (CT / 64);
  if (bf16) hipLaunchKernelGGL(kc_backward<true>, dim3((unsigned)grid), dim3(CT), 0, s, a);
  else hipLaunchKernelGGL(kc_backward<false>, dim3((unsigned)grid), dim3(CT), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
