// The product of few rows with a weight matrix, or with one a group of rows,
// on gfx950: what a served model computes a token.
//
// Bound by the weights' bytes, which go from memory to registers once and
// never through LDS: the matrix instructions would have 16 rows to fill, the
// fp32 ones take longer than the bytes do, and a stage in LDS keeps fewer
// loads under way.  Sums are fp32 by multiply-adds, one order for each shape.
// One row by 4096 x 11008: bf16 20 us with K across and 17.7 with K adjacent
// (5.1 TB/s; 24 on tiles of 64 x 64), fp32 33 (5.5 TB/s; 71).
//
// Rows of the weights along N (K across): a workgroup of 8 waves takes 64
// columns; a lane 16 bytes of columns and 16 bytes of K, so that a row's x is
// one load.  Along K (K adjacent): a workgroup of 4 waves takes 8 columns, a
// lane 16 bytes of K of each.  The lanes' and the waves' sums meet at the end.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "linear_dev.hpp"
#include "linear_plan.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int AW = 8, AC = FEW_ACROSS;    // across: waves, columns
constexpr int BW = 4, BC = FEW_ADJACENT;  // adjacent

// Adds up v over the lanes that differ in bits D, D / 2 to LOW.  While several
// values are left, lanes D apart give each other half of theirs: a lane ends
// with those whose index begins with its bits, from the front of v; once one
// is left, all of the lanes have it.
template <int LEFT, int D, int LOW, int V>
__device__ __forceinline__ void add_lanes(float (&v)[V], int lane) {
  if constexpr (D >= LOW && LEFT > 1) {
    const bool up = lane & D;
#pragma unroll
    for (int i = 0; i < LEFT / 2; ++i) {
      const float give = up ? v[i] : v[i + LEFT / 2], keep = up ? v[i + LEFT / 2] : v[i];
      v[i] = keep + __shfl_xor(give, D);
    }
    add_lanes<LEFT / 2, D / 2, LOW>(v, lane);
  } else if constexpr (D >= LOW) {
    v[0] += __shfl_xor(v[0], D);
    add_lanes<1, D / 2, LOW>(v, lane);
  }
}

__device__ __forceinline__ uint4 if_in(bool in, uint4 v) { return make_uint4(in ? v.x : 0, in ? v.y : 0, in ? v.z : 0, in ? v.w : 0); }

// The sum of tile row r, column col: bias, activation, residual.
template <bool BF16>
__device__ __forceinline__ void leave(const LinearArgs &a, const LinTile &x, int r, int64_t col, float v) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  if (r >= x.rows || col >= a.N) return;
  const int64_t row = x.row0 + r;
  if (a.splits > 1) {
    a.partial[(x.split * a.M + row) * a.N + col] = v;
    return;
  }
  T *pre = static_cast<T *>(a.pre);
  if (a.mode == LIN_FORWARD) {
    if (a.bias) v += E::get(static_cast<const T *>(a.bias)[x.group * a.N + col]);
    if (pre) pre[row * a.pre_ld + col] = E::put(v);
    v = activate<BF16>(a.act, v);
  } else if (a.act != ACT_NONE) {
    v *= slope<BF16>(a.act, E::get(pre[row * a.pre_ld + col]));
  }
  if (a.residual) v += E::get(static_cast<const T *>(a.residual)[row * a.res_ld + col]);
  static_cast<T *>(a.out)[row * a.out_ld + col] = E::put(v);
}

template <bool BF16, int R>
__device__ __forceinline__ void few_across(const LinearArgs &a, const LinTile &x, float *red) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N, LC = AC / N, WK = 64 / LC * N;  // k of a wave's step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane % LC * N, kl = lane / LC * N;
  const int64_t col = x.col0 + c;
  // (a column that does not exist reads another one: its sums are left out)
  const T *w = static_cast<const T *>(a.b) + x.group * a.bstride + (col < a.N ? col : 0);
  const T *p = static_cast<const T *>(a.a) + x.row0 * a.lda;
  float acc[R * N];
#pragma unroll
  for (int i = 0; i < R * N; ++i) acc[i] = 0.f;
  for (int64_t kk = x.k0 + wave * WK; kk < x.k1; kk += AW * WK) {
    const bool in = kk + kl < x.k1;
    const int64_t k = in ? kk + kl : x.k0;
    uint4 wv[N], xv[R];
#pragma unroll
    for (int u = 0; u < N; ++u) wv[u] = load16(w + (k + u) * a.ldb);
#pragma unroll
    for (int r = 0; r < R; ++r) xv[r] = load16(p + (int64_t)min(r, x.rows - 1) * a.lda + k);
#pragma unroll
    for (int r = 0; r < R; ++r) xv[r] = if_in(in, xv[r]);
    float xf[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) E::unpack(xv[r], xf[r]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float wf[N];
      E::unpack(if_in(in, wv[u]), wf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[r * N + n] = fmaf(xf[r][u], wf[n], acc[r * N + n]);
    }
  }
  add_lanes<R * N, 32, LC>(acc, lane);
  constexpr int LEFT = R * N / (64 / LC) > 0 ? R * N / (64 / LC) : 1;
#pragma unroll
  for (int i = 0; i < LEFT; ++i) {
    const int f = lane / LC * LEFT + i;  // = r N + n
    red[wave * R * AC + f / N * AC + c + f % N] = acc[i];
  }
  __syncthreads();
  for (int t = threadIdx.x; t < R * AC; t += AW * 64) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < AW; ++i) sum += red[i * R * AC + t];
    leave<BF16>(a, x, t / AC, x.col0 + t % AC, sum);
  }
}

template <bool BF16, int R>
__device__ __forceinline__ void few_adjacent(const LinearArgs &a, const LinTile &x, float *red) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N, V = R * BC, H = V >= 64 ? 64 : V;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T *w = static_cast<const T *>(a.b) + x.group * a.bstride + x.col0 * a.ldb;
  const T *p = static_cast<const T *>(a.a) + x.row0 * a.lda;
  const int cols = (int)lesser(BC, a.N - x.col0);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int64_t kk = x.k0 + wave * 64 * N; kk < x.k1; kk += BW * 64 * N) {
    const bool in = kk + lane * N < x.k1;
    const int64_t k = in ? kk + lane * N : x.k0;
    uint4 wv[BC], xv[R];
#pragma unroll
    for (int c = 0; c < BC; ++c) wv[c] = load16(w + (int64_t)min(c, cols - 1) * a.ldb + k);
#pragma unroll
    for (int r = 0; r < R; ++r) xv[r] = load16(p + (int64_t)min(r, x.rows - 1) * a.lda + k);
    float xf[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) E::unpack(if_in(in, xv[r]), xf[r]);
#pragma unroll
    for (int c = 0; c < BC; ++c) {
      float wf[N];
      E::unpack(if_in(in, wv[c]), wf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[r * BC + c] = fmaf(xf[r][n], wf[n], acc[r * BC + c]);
    }
  }
  add_lanes<V, 32, 1>(acc, lane);
  if (lane % (64 / H) == 0) red[wave * V + lane / (64 / H)] = acc[0];
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= V) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < BW; ++i) sum += red[i * V + t];
  leave<BF16>(a, x, t / BC, x.col0 + t % BC, sum);
}

// Tiles of up to FEW_ROWS rows of a group, R of which there are at most.  (A
// step's loads alone are under way together: two steps' take the registers of
// other waves, 25.9 to 49.8 us at 8 rows.)
template <bool BF16, bool BX, int R>
__global__ __launch_bounds__(BX ? AW * 64 : BW * 64) void kl_few(LinearArgs a) {
  __shared__ float red[BX ? AW * R * AC : BW * R * BC];
  LinTile x;
  if (!find_tile<FEW_ROWS, true>(a, tile_groups<FEW_ROWS>(a), (int)blockIdx.x, FEW_PART, x)) return;
  x.col0 = x.col0 / FEW_ROWS * (BX ? AC : BC);
  if (R > 1 && x.rows == 1) {
    if constexpr (BX) few_across<BF16, 1>(a, x, red);
    else few_adjacent<BF16, 1>(a, x, red);
  } else {
    if constexpr (BX) few_across<BF16, R>(a, x, red);
    else few_adjacent<BF16, R>(a, x, red);
  }
}

template <bool BF16, bool BX>
void go(const LinearArgs &a, unsigned grid, hipStream_t s) {
  const dim3 threads(BX ? AW * 64 : BW * 64);
  if (a.M == 1) hipLaunchKernelGGL((kl_few<BF16, BX, 1>), dim3(grid), threads, 0, s, a);
  else if (a.M == 2) hipLaunchKernelGGL((kl_few<BF16, BX, 2>), dim3(grid), threads, 0, s, a);
  else if (a.M <= 4) hipLaunchKernelGGL((kl_few<BF16, BX, 4>), dim3(grid), threads, 0, s, a);
  else hipLaunchKernelGGL((kl_few<BF16, BX, FEW_ROWS>), dim3(grid), threads, 0, s, a);
}

}  // namespace

// Sets the launch's tiles and parts; the parts' sums are joined by the caller.
hipError_t launch_linear_few(LinearArgs &a, bool bf16, bool bx, hipStream_t s) {
  const FewPlan p = few_plan(a.M, a.N, a.K, a.groups, bf16, bx);
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.splits = p.splits;
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  const unsigned grid = (unsigned)(tiles * a.splits);
  if (bf16) bx ? go<true, true>(a, grid, s) : go<true, false>(a, grid, s);
  else bx ? go<false, true>(a, grid, s) : go<false, false>(a, grid, s);
  return hipGetLastError();
}

}  // namespace muon
