// The product with a weight matrix, or with one a group of rows, and its
// gradients, on gfx950: any size, type and alignment.
//
//   forwards       out = act(x w + bias) + residual
//   input          dx = (dy w') act'(pre) + residual
//   weights        dw (+)= x' dy,  dbias (+)= the sums of dy's columns
//
// A workgroup of 4 waves (2 x 2) takes a tile and walks K in stages of 128 bytes
// a row, double buffered in LDS: with loads straight into LDS where rows keep
// 16-byte alignment, through registers otherwise.  bf16 on
// v_mfma_f32_16x16x32_bf16, fp32 on v_mfma_f32_16x16x4_f32, sums in fp32.
// Few tiles with a long K are cut along K into parts, whose sums meet in the
// workspace and are added up in the order of the parts by a second launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "linear_dev.hpp"
#include "linear_plan.hpp"

namespace muon {

using namespace dev;

hipError_t launch_linear256(const LinearArgs &a, bool bx, hipStream_t s);

namespace {

// W x W blocks of 16 x 16 a wave: tiles of 128 x 128, or of 64 x 64 where
// larger ones would leave most of the chip idle.
template <bool BF16, bool AX, bool BX, bool DMA, int W>
__global__ __launch_bounds__(LIN_THREADS, 8 / W) void kl_linear(LinearArgs a) {
  constexpr int BT = 32 * W, OPB = BT * STAGE_BYTES;  // an operand's stage in LDS
  typedef Operand<BF16, BT, AX> OA;
  typedef Operand<BF16, BT, BX> OB;
  typedef typename OA::T T;
  constexpr int KS = OA::KS, L = OA::LOADS;
  __shared__ __attribute__((aligned(1024))) char lds[2 * 2 * OPB];
  LinTile x;
  if (!find_tile<BT, true>(a, tile_groups<BT>(a), (int)blockIdx.x, KS, x)) return;
  const OA oa{static_cast<const T *>(a.a) + (AX ? x.row0 : x.row0 * a.lda), a.lda, x.rows, x.k1};
  const OB ob{static_cast<const T *>(a.b) + x.group * a.bstride + (BX ? x.col0 : x.col0 * a.ldb), a.ldb,
              (int)lesser(BT, a.N - x.col0), x.k1};
  const int wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  f32x4_v acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) acc[i][j] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const int nk = (int)((x.k1 - x.k0 + KS - 1) / KS);
  uint32_t offa[L], offb[L];
  uint4 ra[L], rb[L];
  if constexpr (DMA) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      offa[j] = oa.offset(j);
      offb[j] = ob.offset(j);
    }
  }
  const T *qa[L], *qb[L];  // (not DMA) the next plain stage
  if constexpr (!DMA) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      qa[j] = oa.plain(x.k0, j);
      qb[j] = ob.plain(x.k0, j);
    }
  }
  // PLAIN: of a stage with another k behind it (see Operand)
  auto fetch = [&](int kt, int st, auto plain) {
    const int64_t k = x.k0 + (int64_t)kt * KS;
    char *la = lds + st * 2 * OPB, *lb = la + OPB;
    if constexpr (DMA) {
      const auto ars = OA::rsrc(oa.first(k), oa.bytes(k));
      const auto brs = OB::rsrc(ob.first(k), ob.bytes(k));
#pragma unroll
      for (int j = 0; j < L; ++j) {
        OA::dma(ars, oa.left(k), offa[j], la, j);
        OB::dma(brs, ob.left(k), offb[j], lb, j);
      }
    } else if constexpr (decltype(plain)::value) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        ra[j] = load16(qa[j]);
        rb[j] = load16(qb[j]);
        qa[j] += OA::step(a.lda) / (int)sizeof(T);
        qb[j] += OB::step(a.ldb) / (int)sizeof(T);
      }
    } else {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        ra[j] = oa.load(k, j);
        rb[j] = ob.load(k, j);
      }
    }
  };
  auto land = [&](int st) {
    if constexpr (!DMA) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        OA::put(lds + st * 2 * OPB, j, ra[j]);
        OB::put(lds + st * 2 * OPB + OPB, j, rb[j]);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  auto multiply = [&](int st) {
    const char *la = lds + st * 2 * OPB, *lb = la + OPB;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if constexpr (BF16) {
        bf16x8_v fa[W], fb[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          fa[i] = read_fragment<BT, AX>(la, wm * (BT / 2) + i * 16, ks);
          fb[i] = read_fragment<BT, BX>(lb, wn * (BT / 2) + i * 16, ks);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int j = 0; j < W; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      } else {
        f32x4_v fa[W], fb[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          fa[i] = read_fragment_f32<BT, AX>(la, wm * (BT / 2) + i * 16, ks);
          fb[i] = read_fragment_f32<BT, BX>(lb, wn * (BT / 2) + i * 16, ks);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j][c], fa[i][c], acc[i][j], 0, 0, 0);
      }
    }
  };
  // Plain stages, in a loop of their own, as loads under questions keep each
  // other waiting (2047 x 4095 x 4095 bf16: 107 us, 329 with questions in every
  // stage).
  int np = 0;
  if constexpr (!DMA) np = nk > 0 && oa.has_plain() && ob.has_plain() ? nk - 1 : 0;
  const std::true_type yes;
  const std::false_type no;
  if (nk > 0) {
    if (np > 0) fetch(0, 0, yes);
    else fetch(0, 0, no);
    land(0);
  }
  int kt = 0;
  if constexpr (!DMA)
    for (; kt + 1 < np; ++kt) {
      fetch(kt + 1, (kt & 1) ^ 1, yes);
      multiply(kt & 1);
      land((kt & 1) ^ 1);
    }
  for (; kt < nk; ++kt) {
    if (kt + 1 < nk) fetch(kt + 1, (kt & 1) ^ 1, no);
    multiply(kt & 1);
    if (kt + 1 < nk) land((kt & 1) ^ 1);
  }
  if constexpr (DMA) finish_aligned<BF16, W, AX ? (int)LIN_WEIGHT : -1, true>(a, x, acc, (int)threadIdx.x);
  else finish_any<BF16, W, AX>(a, x, acc, (int)threadIdx.x);
}

// Group of a row, by bisection; -1 for a row of none.
__device__ __forceinline__ int group_of(const LinearArgs &a, int64_t row) {
  if (!a.offsets.p) return 0;
  int lo = 0, hi = a.groups;  // start(lo) <= row < start(hi)
  if (row < group_start(a.offsets, 0, a.M) || row >= group_start(a.offsets, a.groups, a.M)) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (group_start(a.offsets, mid, a.M) <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr int JOINED = 4;

// Adds up the parts of the sums, in their order: a thread eight neighbours.
template <bool BF16>
__global__ __launch_bounds__(256) void kl_join(LinearArgs a, int64_t rows) {
  const int64_t chunks = (a.N + 7) / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t row = id / chunks;
  const int64_t col = (id - row * chunks) * 8;
  if (row >= rows) return;
  const int n = (int)lesser(8, a.N - col);
  int g;
  if (a.mode == LIN_WEIGHT) {
    g = (int)(row / a.M);
  } else {
    g = group_of(a, row);
    if (g < 0) return;
  }
  const float *p = a.partial + row * a.N + col;
  const int64_t part = rows * a.N;
  float v[8];
  load8<false>(p, 0, n, v);
  for (int s = 1; s < a.splits; s += JOINED) {
    // loads of several parts under way together: one at a time costs 2.5 us more with 16 parts, 5 with 32
    float w[JOINED][8];
    if (n == 8) {
#pragma unroll
      for (int u = 0; u < JOINED; ++u) load8<false>(p, lesser(s + u, a.splits - 1) * part, 8, w[u]);
    } else {
#pragma unroll
      for (int u = 0; u < JOINED; ++u) load8<false>(p, lesser(s + u, a.splits - 1) * part, n, w[u]);
    }
#pragma unroll
    for (int u = 0; u < JOINED; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s + u < a.splits) v[i] += w[u][i];
  }
  finish8<BF16>(a, g, a.mode == LIN_WEIGHT ? row - g * a.M : row, col, n, v);
}

// -------------------------------------------------------- sums of columns

constexpr int CS_THREADS = 256;

// A thread takes 16 bytes of columns over part of a group's rows.  Sums are
// fp64, as a thread may add up thousands of rows of one sign (131072 rows of
// 0.1 in one part are 6e-5 off in fp32); a part's leaves rounded to fp32.
template <bool BF16>
__global__ __launch_bounds__(CS_THREADS) void kl_column_sums(ColumnSumArgs a) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N;
  // 16 lanes across (256 bytes), 16 rows a round
  __shared__ double red[16][16 * N + 1];
  const int lx = threadIdx.x & 15, ly = threadIdx.x >> 4;
  const int64_t col = ((int64_t)blockIdx.x * 16 + lx) * N;
  const int g = (int)blockIdx.y / a.splits, part = (int)blockIdx.y % a.splits;
  int64_t lo = 0, hi = a.rows;
  if (a.offsets.p) {
    lo = group_start(a.offsets, g, a.rows);
    hi = greater(lo, group_start(a.offsets, g + 1, a.rows));
  }
  const int64_t r0 = lo + (hi - lo) * part / a.splits, r1 = lo + (hi - lo) * (part + 1) / a.splits;
  const int n = (int)lesser(N, a.cols - col);
  double sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.0;
  const T *p = static_cast<const T *>(a.dy) + col;
  if (n == N) {
#pragma unroll 4
    for (int64_t r = r0 + ly; r < r1; r += 16) {
      float v[N];
      E::unpack(load16(p + r * a.ld), v);
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += (double)v[i];
    }
  } else if (n > 0) {
    for (int64_t r = r0 + ly; r < r1; r += 16)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) sum[i] += (double)E::get(p[r * a.ld + i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) red[ly][lx * N + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;
  const int64_t at = (int64_t)blockIdx.x * 16 * N + c;
  if (c >= 16 * N || at >= a.cols) return;
  double v = 0.0;
#pragma unroll
  for (int y = 0; y < 16; ++y) v += red[y][c];
  if (a.splits > 1) a.partial[((int64_t)g * a.splits + part) * a.cols + at] = (float)v;
  else a.out[g * a.cols + at] = a.first ? (float)v : (float)((double)a.out[g * a.cols + at] + v);
}

__global__ __launch_bounds__(CS_THREADS) void kl_column_join(ColumnSumArgs a) {
  const int64_t at = (int64_t)blockIdx.x * CS_THREADS + threadIdx.x;
  if (at >= a.cols) return;
  const int g = (int)blockIdx.y;
  const float *p = a.partial + (int64_t)g * a.splits * a.cols + at;
  double v = 0.0;
  int s = 0;
  // eight loads under way together: one at a time 32 parts take 11 us
  for (; s + 8 <= a.splits; s += 8) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p[(s + i) * a.cols];
#pragma unroll
    for (int i = 0; i < 8; ++i) v += (double)w[i];
  }
  for (; s < a.splits; ++s) v += (double)p[s * a.cols];
  a.out[g * a.cols + at] = a.first ? (float)v : (float)((double)a.out[g * a.cols + at] + v);
}

// dy act'(pre)
template <bool BF16>
__global__ __launch_bounds__(256) void kl_activation_grad(ActivationGradArgs a, int64_t chunks) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = id / chunks, col = (id - row * chunks) * 8;
  if (row >= a.rows) return;
  const int n = (int)lesser(8, a.cols - col);
  float v[8], w[8];
  load8<BF16>(a.dy, row * a.dld + col, n, v);
  load8<BF16>(a.pre, row * a.pld + col, n, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= slope<BF16>(a.act, w[i]);
  store8<BF16>(a.out, row * a.old + col, n, v);
}

// ---------------------------------------------------------------- launches

bool aligned(const void *p, int64_t ld, int64_t extent, int64_t stride, int e) {
  return (uintptr_t)p % 16 == 0 && ld * e % 16 == 0 && extent * e % 16 == 0 && stride * e % 16 == 0 && ld < ((int64_t)1 << 20);
}

int64_t tiles_along(int64_t M, int32_t groups, bool grouped, int bt) {
  return (M + bt - 1) / bt + (grouped ? groups - 1 : 0);
}

template <bool BF16, bool AX, bool BX>
void go(const LinearArgs &a, bool dma, int w, unsigned grid, hipStream_t s) {
  if (w == 4) {
    if (dma) hipLaunchKernelGGL((kl_linear<BF16, AX, BX, true, 4>), dim3(grid), dim3(LIN_THREADS), 0, s, a);
    else hipLaunchKernelGGL((kl_linear<BF16, AX, BX, false, 4>), dim3(grid), dim3(LIN_THREADS), 0, s, a);
  } else {
    if (dma) hipLaunchKernelGGL((kl_linear<BF16, AX, BX, true, 2>), dim3(grid), dim3(LIN_THREADS), 0, s, a);
    else hipLaunchKernelGGL((kl_linear<BF16, AX, BX, false, 2>), dim3(grid), dim3(LIN_THREADS), 0, s, a);
  }
}

// Whether 256 x 256 tiles are many enough: 128 of them are 512 of 128 x 128,
// which fill the chip once (4096 x 4096 weights, on large and small tiles: 128
// large ones 113 and 69 us, 160 108 and 122, 208 108 and 129, 256 110 and 134).
bool large_tiles(const LinearArgs &a, bool weight) {
  const int64_t tiles = (a.M + 255) / 256 * ((a.N + 255) / 256) * (weight ? a.groups : 1);
  return tiles >= 160 && a.N >= 256 && (weight ? a.M >= 256 : a.M / a.groups >= 256);
}

}  // namespace

hipError_t launch_linear(LinearArgs a, bool bf16, int la, int lb, hipStream_t s) {
  const int e = bf16 ? 2 : 4;
  const bool ax = la == LIN_K_ACROSS, bx = lb == LIN_K_ACROSS, weight = a.mode == LIN_WEIGHT;
  const int eo = weight ? 4 : e;
  const bool dma = aligned(a.a, a.lda, ax ? a.M : a.K, 0, e) && aligned(a.b, a.ldb, bx ? a.N : a.K, a.groups > 1 ? a.bstride : 0, e) &&
                   a.N % 8 == 0 && aligned(a.out, a.out_ld, 0, a.groups > 1 ? a.out_stride : 0, eo) &&
                   (!a.pre || aligned(a.pre, a.pre_ld, 0, 0, e)) && (!a.residual || aligned(a.residual, a.res_ld, 0, 0, e));
  if (bf16 && dma && large_tiles(a, weight)) {
    a.splits = 1;
    a.tiles_m = (int32_t)tiles_along(a.M, a.groups, !weight && a.offsets.p, 256);
    a.tiles_n = (int32_t)((a.N + 255) / 256);
    return launch_linear256(a, bx, s);
  }
  hipError_t err;
  if (dma && !weight && few_rows(a.M, bf16, bx, a.offsets.p != nullptr)) {
    err = launch_linear_few(a, bf16, bx, s);
  } else {
    const LinearPlan p = linear_plan(a.M, a.N, a.K, a.groups, weight, bf16);
    const int bt = 32 * p.w;
    a.splits = p.splits;
    a.tiles_m = (int32_t)tiles_along(a.M, a.groups, !weight && a.offsets.p, bt);
    a.tiles_n = (int32_t)((a.N + bt - 1) / bt);
    const int64_t grid = (int64_t)a.tiles_m * a.tiles_n * (weight ? a.groups : 1) * a.splits;
    const unsigned g = (unsigned)grid;
    if (bf16) {
      if (ax) go<true, true, true>(a, dma, p.w, g, s);
      else if (bx) go<true, false, true>(a, dma, p.w, g, s);
      else go<true, false, false>(a, dma, p.w, g, s);
    } else {
      if (ax) go<false, true, true>(a, dma, p.w, g, s);
      else if (bx) go<false, false, true>(a, dma, p.w, g, s);
      else go<false, false, false>(a, dma, p.w, g, s);
    }
    err = hipGetLastError();
  }
  if (err != hipSuccess || a.splits == 1) return err;
  const int64_t rows = a.M * (weight ? a.groups : 1), threads = rows * ((a.N + 7) / 8);
  if (bf16) hipLaunchKernelGGL(kl_join<true>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, rows);
  else hipLaunchKernelGGL(kl_join<false>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, rows);
  return hipGetLastError();
}

// Parts of a group's rows for the sums of columns: enough for four workgroups
// a CU, of 64 rows each and more.
int32_t column_sum_splits(int64_t rows, int64_t cols, int32_t groups) {
  const int64_t wide = (cols + 127) / 128 * groups;
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({1024 / std::max<int64_t>(1, wide), rows / groups / 64, 64}));
}

hipError_t launch_column_sums(const ColumnSumArgs &a, bool bf16, hipStream_t s) {
  const int n = bf16 ? 128 : 64;
  const dim3 grid((unsigned)((a.cols + n - 1) / n), (unsigned)(a.groups * a.splits));
  if (bf16) hipLaunchKernelGGL(kl_column_sums<true>, grid, dim3(CS_THREADS), 0, s, a);
  else hipLaunchKernelGGL(kl_column_sums<false>, grid, dim3(CS_THREADS), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(kl_column_join, dim3((unsigned)((a.cols + CS_THREADS - 1) / CS_THREADS), (unsigned)a.groups),
                     dim3(CS_THREADS), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_activation_grad(const ActivationGradArgs &a, bool bf16, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t chunks = (a.cols + 7) / 8;
  const unsigned grid = (unsigned)((a.rows * chunks + 255) / 256);
  if (bf16) hipLaunchKernelGGL(kl_activation_grad<true>, dim3(grid), dim3(256), 0, s, a, chunks);
  else hipLaunchKernelGGL(kl_activation_grad<false>, dim3(grid), dim3(256), 0, s, a, chunks);
  return hipGetLastError();
}

}  // namespace muon
