// Dropout whose mask is never stored, on gfx950.
//
//   out = residual + (r >= threshold ? x * scale : 0),  threshold = p 2^32,
//   scale = 1 / (1 - p)
//
// r is a word of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): a block cipher of a counter, so
// any element's word is computed from where it stands and the backward pass is
// the same call on the gradient.  The counter is (column / 4, row, site, step)
// and the key the seed: four neighbours of a row share a block, whatever the
// row stride, and sites (layers) and steps never share one.
//
// Bound by HBM as long as the ten rounds (20 products of 32 x 32 bits for four
// elements) hide behind the loads: 16384 x 8192 bf16 with a residual 145 us,
// 5.55 TB/s.
#include <hip/hip_runtime.h>

#include "devops.hpp"
#include "layer_ops.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int DT = 256;    // threads of a workgroup
constexpr int DV = 4;      // vectors a thread

__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1,
                                       uint32_t *r) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(q >> 32) ^ c1 ^ k0, n2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  r[0] = c0;
  r[1] = c1;
  r[2] = c2;
  r[3] = c3;
}

// A workgroup takes DT * DV consecutive 16-byte vectors of the rows laid end
// to end; magic = 2^32 / vecs + 1 divides numbers below 2048 by vecs < 1024.
template <bool BF16>
__global__ __launch_bounds__(DT) void kd_dropout(DropoutArgs a, uint32_t vecs, uint32_t magic) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N;
  const int64_t base = (int64_t)blockIdx.x * (DT * DV);
  const int64_t row0 = base / vecs;
  const uint32_t col0 = (uint32_t)(base - row0 * vecs);
  const uint32_t step = a.device_step ? (uint32_t)*a.device_step : a.step;
  uint4 xv[DV], rv[DV];
  int64_t row[DV];
  uint32_t vec[DV];
#pragma unroll
  for (int u = 0; u < DV; ++u) {
    const uint32_t at = col0 + u * DT + threadIdx.x;
    const uint32_t over = vecs >= 1024 ? (at >= vecs ? 1u : 0u) : vecs == 1 ? at : __umulhi(at, magic);
    row[u] = row0 + over;
    vec[u] = at - over * vecs;
    const uint32_t c = vec[u] * N;
    if (row[u] < a.rows && c + N <= (uint32_t)a.cols) {
      xv[u] = load16(static_cast<const T *>(a.x) + row[u] * a.ld + c);
      if (a.residual) rv[u] = load16(static_cast<const T *>(a.residual) + row[u] * a.rld + c);
    }
  }
#pragma unroll
  for (int u = 0; u < DV; ++u) {
    if (row[u] >= a.rows) continue;
    const uint32_t c = vec[u] * N;
    uint32_t r[N];
#pragma unroll
    for (int q = 0; q < N / 4; ++q) philox(c / 4 + q, (uint32_t)row[u], a.site, step, a.key0, a.key1, r + 4 * q);
    T *out = static_cast<T *>(a.out) + row[u] * a.old + c;
    if (c + N <= (uint32_t)a.cols) {
      float v[N], w[N];
      E::unpack(xv[u], v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = r[j] >= a.threshold ? v[j] * a.scale : 0.f;
      if (a.residual) {
        E::unpack(rv[u], w);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += w[j];
      }
      stream16(out, E::pack(v));
    } else {
      const T *x = static_cast<const T *>(a.x) + row[u] * a.ld + c;
      const T *res = static_cast<const T *>(a.residual) + row[u] * a.rld + c;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j < (uint32_t)a.cols) {
          const float v = r[j] >= a.threshold ? E::get(x[j]) * a.scale : 0.f;
          out[j] = E::put(a.residual ? v + E::get(res[j]) : v);
        }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, bool bf16, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t n = bf16 ? 8 : 4, vecs = (a.cols + n - 1) / n;
  const uint32_t magic = vecs < 1024 ? (uint32_t)(((int64_t)1 << 32) / vecs + 1) : 0u;
  const int64_t grid = (a.rows * vecs + DT * DV - 1) / (DT * DV);
  if (bf16) hipLaunchKernelGGL(kd_dropout<true>, dim3((unsigned)grid), dim3(DT), 0, s, a, (uint32_t)vecs, magic);
  else hipLaunchKernelGGL(kd_dropout<false>, dim3((unsigned)grid), dim3(DT), 0, s, a, (uint32_t)vecs, magic);
  return hipGetLastError();
}

}  // namespace muon
