// The product with a weight matrix and its gradients on 256 x 256 tiles, for
// large bf16 products whose rows keep 16-byte alignment, on gfx950.
//
// A workgroup of 4 waves (2 x 2), each 128 x 128 = 8 x 8 blocks of
// v_mfma_f32_16x16x32_bf16 with 256 fp32 sums a lane: 16 fragments of LDS feed
// 64 products, half of what 64 x 64 a wave needs, which is bound by LDS.  K in
// stages of 64, double buffered, loaded straight into LDS (buffer_load_dwordx4
// ... lds) with 16 loads a wave and stage, spread one a group of four products:
// issued together they stall the wave until the address unit has taken them.
// A stage has two barriers: one when every wave has read the stage's last
// fragments, which frees its buffer for the stage after the next, and one
// between its two k-steps, which waits for the next stage's loads alone.
// 8192 x 4096 x 11008: 630 us, 1.17 PFLOP/s, 1.45 us a stage and round.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_dev.hpp"

namespace muon {

using namespace dev;

namespace {

constexpr int BT = 256;
constexpr int OPB = BT * STAGE_BYTES;  // 32 KB an operand and stage

enum Kind { FIRST, MIDDLE, LAST };

// c (+)= b' a with the sums tied in place: left to itself the compiler rotates
// the 64 blocks through copies.  The first product of a block takes no sums.
// The compiler does not see the latency of an asm product, so the last one of
// every block goes through the builtin, and nothing but the next k-step's
// products, 64 instructions later, reads an asm one.
template <Kind KIND>
__device__ __forceinline__ void mfma(f32x4_v &c, const bf16x8_v &b, const bf16x8_v &a) {
  if constexpr (KIND == FIRST) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=a"(c) : "v"(b), "v"(a));
  else if constexpr (KIND == LAST) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
  else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// the stages, and the next place in the queue
__shared__ __attribute__((aligned(1024))) char lds[2 * 2 * OPB + 64];

// A workgroup takes several tiles, whose stages form one sequence: the next
// tile's first two are loaded while this tile's last two are multiplied and
// wait in LDS while its sums leave.  Tiles of equal K are taken `stride` apart;
// those of a grouped weight gradient (QUEUE) are of very different K, and each
// XCD's workgroups take theirs from a queue that begins with the longest
// group's.
template <int MODE, bool BX, bool QUEUE>
__global__ __launch_bounds__(LIN_THREADS, 1) void kl_linear256(LinearArgs a, int stride) {
  constexpr bool AX = MODE == LIN_WEIGHT;
  typedef Operand<true, BT, AX> OA;
  typedef Operand<true, BT, BX> OB;
  typedef typename OA::T T;
  constexpr int KS = OA::KS;
  // What a wave has under way when it waits: a stage's loads, and behind a tile
  // at least kStores stores of its sums (every row of blocks is stored, those
  // that do not exist outside the range).  Fewer would leave a wait too short.
  constexpr int kLoads = OA::LOADS + OB::LOADS, kStores = 32;
  static_assert(TileRows<MODE != LIN_WEIGHT, 8>::STORES >= kStores && kLoads + kStores < 64, "the vmcnt immediates behind a tile");
  // workgroup i runs on XCD i % 8: chunks of 256 tiles, 32 consecutive ones an XCD
  const int xcd = (int)blockIdx.x & 7, slot = (int)blockIdx.x >> 3;
  int t = (slot >> 5) * 256 + xcd * 32 + (slot & 31);
  LinTile x;
  // of each group's tiles, an XCD's: [q0, q0 + qn)
  const int each = a.tiles_m * a.tiles_n, q0 = xcd * ((each + 7) / 8), qn = min((each + 7) / 8, each - q0);
  LinearQueue *queue = reinterpret_cast<LinearQueue *>(a.queue);
  int *next_slot = reinterpret_cast<int *>(lds + 2 * 2 * OPB);
  auto queued = [&](int place, LinTile &y) {
    if (place >= qn * a.groups) return false;
    const int g = place / qn;
    weight_tile<BT>(a, uni32(queue->group[g]), q0 + place - g * qn, y);
    y.split = 0;
    return true;
  };
  if constexpr (QUEUE) {
    if (qn <= 0 || !queued(slot, x)) return;
    if (threadIdx.x == 0) *next_slot = atomicAdd(&queue->taken[xcd][0], 1);
  }
  TileGroups groups;
  if constexpr (MODE != LIN_WEIGHT) groups = tile_groups<BT>(a);
  auto find = [&](int t, LinTile &y) {
    if constexpr (MODE != LIN_WEIGHT) return find_tile<BT, false>(a, groups, t, KS, y);
    if (t >= each) return false;
    weight_tile<BT>(a, 0, t, y);
    y.split = 0;
    return true;
  };
  if (!QUEUE && !find(t, x)) return;
  const int wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  uint32_t offa[8], offb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    offa[j] = OA{nullptr, a.lda, 0, 0}.offset(j);
    offb[j] = OB{nullptr, a.ldb, 0, 0}.offset(j);
  }
  // The stage to be loaded next.
  struct Cursor {
    const char *a, *b;
    int64_t a_bytes, b_bytes, left;
  };
  auto start = [&](const LinTile &y) {
    const OA oa{static_cast<const T *>(a.a) + (AX ? y.row0 : y.row0 * a.lda), a.lda, y.rows, y.k1};
    const OB ob{static_cast<const T *>(a.b) + y.group * a.bstride + (BX ? y.col0 : y.col0 * a.ldb), a.ldb,
                (int)lesser(BT, a.N - y.col0), y.k1};
    return Cursor{oa.first(y.k0), ob.first(y.k0), oa.bytes(y.k0), ob.bytes(y.k0), y.k1 - y.k0};
  };
  struct Stage {
    __amdgpu_buffer_rsrc_t a, b;
    int left;
  };
  // The cursor's stage; behind a tile's last one a range of nothing, whose loads are zeros.
  auto take = [&](Cursor &c) {
    const bool any = c.left > 0;
    const Stage s{OA::rsrc(c.a, any ? c.a_bytes : 0), OB::rsrc(c.b, any ? c.b_bytes : 0), (int)lesser(c.left, KS)};
    c.a += OA::step(a.lda);
    c.b += OB::step(a.ldb);
    c.a_bytes -= OA::step(a.lda);
    c.b_bytes -= OB::step(a.ldb);
    c.left -= KS;
    return s;
  };
  auto dma1 = [&](const Stage &s, int st, int q) {
    char *la = lds + st * 2 * OPB;
    if (q < 8) OA::dma(s.a, s.left, offa[q], la, q);
    else OB::dma(s.b, s.left, offb[q - 8], la + OPB, q - 8);
  };
  Cursor at = start(x);
  int base = 0;        // buffer of the tile's first stage
  bool ready = false;  // whose loads, and the second one's, are under way
  for (;;) {
    // at least two stages: what is behind the last one is zeros
    const int nk = (int)greater(2, (x.k1 - x.k0 + KS - 1) / KS);
    bool chain;
    LinTile y;
    int taken = 0;
    f32x4_v acc[8][8];
    {
      bf16x8_v fa[2][8], fb[2][8];
      // fragment q of a k-step, in the order its products need them: A0, B0..B7, A1..A7
      auto read1 = [&](int set, int st, int ks, int q) {
        const char *la = lds + st * 2 * OPB, *lb = la + OPB;
        if (q == 0 || q > 8) {
          const int i = q == 0 ? 0 : q - 8;
          fa[set][i] = read_fragment<BT, AX>(la, wm * 128 + i * 16, ks);
        } else {
          fb[set][q - 1] = read_fragment<BT, BX>(lb, wn * 128 + (q - 1) * 16, ks);
        }
      };
      if (!ready) {
        const Stage s0 = take(at);
#pragma unroll
        for (int q = 0; q < 16; ++q) dma1(s0, base, q);
        const Stage s1 = take(at);
#pragma unroll
        for (int q = 0; q < 16; ++q) dma1(s1, base ^ 1, q);
      }
      // all but the second stage's loads, and behind a tile its stores
      if (ready) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads + kStores) : "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
      if constexpr (QUEUE) {
        chain = queued(uni32(*next_slot), y);
        if (threadIdx.x == 0 && chain) taken = atomicAdd(&queue->taken[xcd][0], 1);
      } else {
        t += stride;
        chain = find(t, y);
      }
      const Cursor then = chain ? start(y) : at;
#pragma unroll
      for (int q = 0; q < 16; ++q) read1(0, base, 0, q);
      constexpr int kBar1 = 9;           // group of k-step 0 that ends with the first barrier
      constexpr int kDma0 = 15 - kBar1;  // loads in k-step 0
      constexpr int kDma1 = kLoads - kDma0;  // in k-step 1
      static_assert(kLoads == 16 && kDma0 > 0, "the loads' places among the products");
      auto body = [&](int kt, auto kind) {
        constexpr Kind KIND = decltype(kind)::value;
        const int st = (kt ^ base) & 1;
        if (chain && kt == nk - 2) at = then;
        const Stage nn = take(at);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int i = n >> 1, j = (n & 1) * 4;
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) mfma<KIND == FIRST ? FIRST : MIDDLE>(acc[i][j + jj], fb[0][j + jj], fa[0][i]);
          __builtin_amdgcn_sched_barrier(0);
          if (n < 8) {
            read1(1, st, 1, 2 * n);
            read1(1, st, 1, 2 * n + 1);
          }
          if (n == kBar1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          if (n > kBar1) dma1(nn, st, n - kBar1 - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (KIND != LAST) {
          // the next stage's loads: all but those of this k-step, and behind a tile its stores
          if (KIND == FIRST && ready) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kDma0 + kStores) : "memory");
          else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kDma0) : "memory");
        }
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int i = n >> 1, j = (n & 1) * 4;
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) mfma<KIND == LAST ? LAST : MIDDLE>(acc[i][j + jj], fb[1][j + jj], fa[1][i]);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (KIND != LAST) {
            if (n < 4) {
              read1(0, st ^ 1, 0, 2 * n);
              read1(0, st ^ 1, 0, 2 * n + 1);
            } else if (n < 12) {
              read1(0, st ^ 1, 0, n + 4);
            }
          }
          // the q-th of the last kDma1 loads in the group where n kDma1 / 16 steps up
          if (((n + 1) * kDma1) / 16 > (n * kDma1) / 16) dma1(nn, st, kDma0 + (n * kDma1) / 16);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      body(0, std::integral_constant<Kind, FIRST>());
      for (int kt = 1; kt < nk - 1; ++kt) body(kt, std::integral_constant<Kind, MIDDLE>());
      body(nk - 1, std::integral_constant<Kind, LAST>());
      // the loads of zeros behind the last tile must not outlive the workgroup
      if (!chain) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    // What the sums' way needs is read and computed here, tile by tile: kept
    // over the products it does not fit the registers.
    typedef __attribute__((address_space(4))) const LinearArgs KernelArgs;
    KernelArgs *args = (KernelArgs *)__builtin_amdgcn_kernarg_segment_ptr();  // the first argument
    int tid = (int)threadIdx.x;
    asm volatile("" : "+s"(args), "+v"(tid));
    LinearArgs b;
    __builtin_memcpy(&b, (const void *)args, sizeof b);
    finish_aligned<true, 8, MODE, false>(b, x, acc, tid);
    if (!chain) return;
    if constexpr (QUEUE) {
      if (threadIdx.x == 0) *next_slot = taken;
    }
    ready = true;
    base = (nk + base) & 1;
    x = y;
  }
}

}  // namespace

// Sorts the groups by their rows, and clears the queues: each XCD's first 32
// places are its workgroups' own.
__global__ __launch_bounds__(1024) void kl_queue(LinearArgs a) {
  __shared__ int64_t size[1024];
  LinearQueue *queue = reinterpret_cast<LinearQueue *>(a.queue);
  const int g = threadIdx.x;
  int64_t mine = 0;
  if (g < a.groups) mine = group_start(a.offsets, g + 1, a.K) - group_start(a.offsets, g, a.K);
  size[g] = mine;
  if (g < 8) queue->taken[g][0] = 32;
  __syncthreads();
  if (g >= a.groups) return;
  int before = 0;
  for (int h = 0; h < a.groups; ++h) before += size[h] > mine || (size[h] == mine && h < g);
  queue->group[before] = g;
}

template <int MODE, bool BX, bool QUEUE>
void go(const LinearArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((kl_linear256<MODE, BX, QUEUE>), dim3(256), dim3(LIN_THREADS), 0, s, a, 256);
}

hipError_t launch_linear256(const LinearArgs &a, bool bx, hipStream_t s) {
  if (a.mode == LIN_WEIGHT && a.offsets.p) {
    static_assert(sizeof(LinearQueue::group) / 4 == 1024, "a group a thread");
    hipLaunchKernelGGL(kl_queue, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    go<LIN_WEIGHT, true, true>(a, s);
  } else if (a.mode == LIN_WEIGHT) {
    go<LIN_WEIGHT, true, false>(a, s);
  } else if (a.mode == LIN_FORWARD) {
    bx ? go<LIN_FORWARD, true, false>(a, s) : go<LIN_FORWARD, false, false>(a, s);
  } else {
    bx ? go<LIN_INPUT, true, false>(a, s) : go<LIN_INPUT, false, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace muon
