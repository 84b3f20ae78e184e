// Device parts that the kernels of the product with a weight matrix share:
// where a workgroup's tile lies, how a stage of an operand is laid out in LDS,
// activations, and the way of a tile's sums from registers to memory.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "devops.hpp"
#include "linear.hpp"

namespace muon {
namespace dev {

typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x4_v __attribute__((ext_vector_type(4)));
typedef short i16x4_v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_v lds_i16x4;
typedef __attribute__((address_space(3))) void lds_any;

constexpr int LIN_THREADS = 256;
constexpr int STAGE_BYTES = 128;  // of K a stage holds: 64 bf16 or 32 fp32

// ------------------------------------------------------------- activations

enum : int32_t { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// exp(x).  The rounding of x log2(e) moves it by |x| 2^-24 of itself: hidden
// by a bf16 result's rounding, while for an fp32 result what the product
// leaves over is multiplied in.
template <bool BF16>
__device__ __forceinline__ float exp_of(float x) {
  const float p = x * kLog2e, e = __builtin_amdgcn_exp2f(p);
  if (BF16) return e;
  const float low = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p));
  return fabsf(p) < 256.f ? e * fmaf(low, 0.69314718f, 1.f) : e;  // further out 0 or infinity, and low no number
}

// Phi(v) = (1 + erf(v / sqrt 2)) / 2.  For bf16 results Phi(-x) = exp(-x^2 / 2)
// times a polynomial of degree 6 in 1 / (1 + 0.29 x), a minimax fit over
// [0, 14]: off by at most 7.8e-8 and by at most 7.8e-5 of Phi(-x), so that
// gelu's tail keeps bf16's digits (a tenth of the instructions of erfcf, of
// which a tile's thread would spend 256).  fp32 results take erfcf.
template <bool BF16>
__device__ __forceinline__ float normal_cdf(float v) {
  if constexpr (BF16) {
    const float x = fabsf(v);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.29f, x, 1.f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, fmaf(t, -0.08837444317f, 0.2833175835f), -0.09105694498f), 0.1781477883f), 0.1011390706f), 0.1168270219f);
    const float tail = p * exp_of<true>(-0.5f * v * v);
    return v < 0.f ? tail : 1.f - tail;
  } else {
    return 0.5f * erfcf(-0.70710678f * v);
  }
}
template <bool BF16>
__device__ __forceinline__ float quotient(float d) {
  return BF16 ? __builtin_amdgcn_rcpf(d) : 1.f / d;
}
// q = 1 / (1 + exp(-u)), and 1 - q: for an fp32 result from the exponential
// where q is near 1, which leaves 1 - q few digits.
template <bool BF16>
__device__ __forceinline__ float logistic(float u, float &rest) {
  const float e = exp_of<BF16>(-u), q = quotient<BF16>(1.f + e);
  rest = !BF16 && u > 0.f ? e * q : 1.f - q;
  return q;
}
// 2 sqrt(2 / pi) (v + 0.044715 v^3): (1 + tanh(half of it)) / 2 is its logistic
__device__ __forceinline__ float tanh_argument(float v) { return v * fmaf(0.0713548163f, v * v, 1.5957691216f); }

template <bool BF16>
__device__ __forceinline__ float activate(int32_t act, float v) {
  float rest;
  switch (act) {
    case ACT_RELU: return v < 0.f ? 0.f : v;
    case ACT_SILU: return v * logistic<BF16>(v, rest);
    case ACT_GELU: return v * normal_cdf<BF16>(v);
    case ACT_GELU_TANH: return v * logistic<BF16>(tanh_argument(v), rest);
    default: return v;
  }
}
template <bool BF16>
__device__ __forceinline__ float slope(int32_t act, float v) {
  float rest;
  switch (act) {
    case ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case ACT_SILU: {
      const float q = logistic<BF16>(v, rest);
      return q * fmaf(v, rest, 1.f);
    }
    case ACT_GELU: return fmaf(v * 0.39894228f, exp_of<BF16>(-0.5f * v * v), normal_cdf<BF16>(v));
    case ACT_GELU_TANH: {
      v = v < -64.f ? -64.f : v > 64.f ? 64.f : v;  // 0 and 1 from there on, where v^2 is still finite
      const float q = logistic<BF16>(tanh_argument(v), rest);
      return fmaf(v * q * rest, fmaf(0.2140644489f, v * v, 1.5957691216f), q);
    }
    default: return 1.f;
  }
}

// -------------------------------------------------------------------- tiles

__device__ __forceinline__ int uni32(int v) { return __builtin_amdgcn_readfirstlane(v); }

// First row of group g, and of group `groups` the end; what falls outside
// [0, rows] is cut off.
__device__ __forceinline__ int64_t group_start(const IndexVec &o, int g, int64_t rows) {
  const int64_t v = index_at(o, g);
  return v < 0 ? 0 : v > rows ? rows : v;
}

struct LinTile {
  int64_t row0, col0;  // of C (in LIN_WEIGHT: of its group's C)
  int64_t k0, k1;
  int rows;            // of the tile that exist
  int group, split;
};

// Tiles are counted in panels of 8 tile rows, column by column, so that 32
// consecutive ones, which the 32 CUs of an XCD take, share 8 + 4 panels of
// operands.
__device__ __forceinline__ void tile_at(int tiles_m, int tiles_n, int t, int &tm, int &tn) {
  const int panel = t / (8 * tiles_n), in = t - panel * 8 * tiles_n;
  const int high = min(8, tiles_m - panel * 8);
  tn = in / high;
  tm = panel * 8 + in - tn * high;
}

// Tile t of a group's weight gradient.
template <int BT>
__device__ __forceinline__ void weight_tile(const LinearArgs &a, int group, int t, LinTile &x) {
  int tm, tn;
  tile_at(a.tiles_m, a.tiles_n, t, tm, tn);
  x.group = group;
  x.col0 = (int64_t)tn * BT;
  x.row0 = (int64_t)tm * BT;
  x.rows = (int)lesser(BT, a.M - x.row0);
  x.k0 = 0;
  x.k1 = a.K;
  if (a.offsets.p) {
    x.k0 = uniform(group_start(a.offsets, group, a.K));
    x.k1 = greater(x.k0, uniform(group_start(a.offsets, group + 1, a.K)));
  }
}

// The tile's part of K.
__device__ __forceinline__ void cut_tile(const LinearArgs &a, int stage_k, LinTile &x) {
  if (a.splits <= 1) return;
  const int64_t stages = (x.k1 - x.k0 + stage_k - 1) / stage_k, start = x.k0, end = x.k1;
  x.k0 = lesser(end, start + stages * x.split / a.splits * stage_k);
  x.k1 = lesser(end, start + stages * (x.split + 1) / a.splits * stage_k);
}

// A product's tile rows are those of its groups one after the other: where
// they begin, for the first 64 groups a lane each, and how many there are.
struct TileGroups {
  int64_t lo, hi;  // the group's rows
  int first, tiles;
  int total;       // of all groups
};

// The tile rows of groups [g0, g0 + 64), behind `before` ones.
template <int BT>
__device__ __forceinline__ void scan_groups(const LinearArgs &a, int g0, int before, TileGroups &r) {
  const int lane = threadIdx.x & 63, g = g0 + lane;
  r.lo = r.hi = 0;
  if (g < a.groups) {
    r.lo = group_start(a.offsets, g, a.M);
    r.hi = group_start(a.offsets, g + 1, a.M);
  }
  r.tiles = r.hi > r.lo ? (int)((r.hi - r.lo + BT - 1) / BT) : 0;
  int sum = r.tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  r.first = before + sum - r.tiles;
  r.total = before + uni32(__shfl(sum, 63));
}
template <int BT>
__device__ __forceinline__ TileGroups tile_groups(const LinearArgs &a) {
  TileGroups r{0, 0, 0, 0, a.tiles_m};
  if (a.mode == LIN_WEIGHT || !a.offsets.p) return r;
  scan_groups<BT>(a, 0, 0, r);
  TileGroups more = r;
  for (int g0 = 64; g0 < a.groups; g0 += 64) scan_groups<BT>(a, g0, more.total, more);
  r.total = more.total;
  return r;
}

// Tile t of a launch of BT x BT tiles; false if there is none.  PARTS: of one
// that may be cut along K.
template <int BT, bool PARTS>
__device__ __forceinline__ bool find_tile(const LinearArgs &a, const TileGroups &groups, int t, int stage_k, LinTile &x) {
  const int per_split = groups.total * a.tiles_n * (a.mode == LIN_WEIGHT ? a.groups : 1);
  if (t >= per_split * (PARTS ? a.splits : 1)) return false;
  x.split = PARTS ? t / per_split : 0;
  t -= x.split * per_split;
  if (a.mode == LIN_WEIGHT) {
    const int group = t / (a.tiles_m * a.tiles_n);
    weight_tile<BT>(a, group, t - group * a.tiles_m * a.tiles_n, x);
    if (PARTS) cut_tile(a, stage_k, x);
    return true;
  }
  int tm, tn;
  tile_at(groups.total, a.tiles_n, t, tm, tn);
  x.group = 0;
  x.col0 = (int64_t)tn * BT;
  x.k0 = 0;
  x.k1 = a.K;
  if (!a.offsets.p) {
    x.row0 = (int64_t)tm * BT;
    x.rows = (int)lesser(BT, a.M - x.row0);
  } else {
    TileGroups r = groups;
    uint64_t has = __ballot(tm >= r.first && tm < r.first + r.tiles);
    int g0 = 0;
    if (!has) {
      // a group behind the 64th: the scan again
      int before = uni32(__shfl(r.first + r.tiles, 63));
      for (g0 = 64; !has && g0 < a.groups; g0 += 64) {
        scan_groups<BT>(a, g0, before, r);
        before = r.total;
        has = __ballot(tm >= r.first && tm < r.first + r.tiles);
      }
      g0 -= 64;
    }
    const int who = __ffsll((unsigned long long)has) - 1;
    x.group = g0 + who;
    const int first = uni32(__shfl(r.first, who));
    const int64_t lo = uniform((int64_t)__shfl((long long)r.lo, who)), hi = uniform((int64_t)__shfl((long long)r.hi, who));
    x.row0 = lo + (int64_t)(tm - first) * BT;
    x.rows = (int)lesser(BT, hi - x.row0);
  }
  if (PARTS) cut_tile(a, stage_k, x);
  return true;
}

// ----------------------------------------------------- operands in LDS
//
// K adjacent: a row of the tile is 128 bytes of a stage, 16-byte chunk c of
// row r at position c ^ (r / 2 % 8): the 16 rows that a quarter of a fragment
// read touches spread over all banks.
// K across: a row is one k of the stage with the tile's BT elements.  bf16
// fragments are read with transposing reads (ds_read_b64_tr_b16: lane i of 16
// gets element i % 4 of the 8 bytes that lanes i / 4, 4 + i / 4, ... address),
// four k x 16 elements a group of 16 lanes: 32-byte pieces are XORed with
// f(k) = k % 4 + 4 (k / 8 % 2), so that the eight k of half a wave fall on
// different banks.  fp32 elements are read one by one, 64-byte pieces XORed
// with k / 4 % 4.

__device__ __forceinline__ int adjacent_chunk(int r, int c) { return c ^ (r >> 1 & 7); }
template <bool BF16, int BT>
__device__ __forceinline__ int across_chunk(int k, int c) {
  if (!BF16) return c ^ (k >> 2 & 3) << 2;
  // rows of 128 bytes lie two to the banks' 256
  return BT == 64 ? c ^ ((k >> 1 & 1) << 1 | (k >> 3 & 1) << 2) : c ^ ((k & 3) << 1 | (k >> 3 & 1) << 3);
}

// One operand of a BT-wide tile as a stage's loads see it: BT / 32 loads of 16
// bytes a thread, load j of wave w covering the LDS bytes from (w BT / 32 + j)
// KB on, lane l its 16 bytes l.
template <bool BF16, int BT, bool ACROSS>
struct Operand {
  typedef typename Elem<BF16>::type T;
  static constexpr int E = (int)sizeof(T), N = 16 / E, LOADS = BT / 32, KS = STAGE_BYTES / E;
  static constexpr int CPR = ACROSS ? BT * E / 16 : 8;  // 16-byte chunks of a row in LDS
  static constexpr int RPL = 64 / CPR;                  // rows of a load
  const T *p;       // the operand's element (tile, k = 0)
  int64_t ld;
  int extent;       // elements of the tile that exist
  int64_t k1;

  static __device__ __forceinline__ int row(int j) { return ((threadIdx.x >> 6) * LOADS + j) * RPL + (threadIdx.x & 63) / CPR; }
  static __device__ __forceinline__ int chunk(int j) {
    const int r = row(j), c = (threadIdx.x & 63) % CPR;
    return ACROSS ? across_chunk<BF16, BT>(r, c) : adjacent_chunk(r, c);
  }
  // 32-bit byte offset of load j from the stage's first element
  __device__ __forceinline__ uint32_t offset(int j) const { return (uint32_t)(row(j) * ld * E) + chunk(j) * 16; }

  // The operand's first element of k, and the bytes from there to its last one.
  __device__ __forceinline__ const char *first(int64_t k) const { return reinterpret_cast<const char *>(p + (ACROSS ? k * ld : k)); }
  __device__ __forceinline__ int64_t bytes(int64_t k) const {
    return k >= k1 ? 0 : ACROSS ? ((k1 - k - 1) * ld + extent) * E : ((int64_t)(extent - 1) * ld + (k1 - k)) * E;
  }
  // From a stage's first element to the next one's.
  static __device__ __forceinline__ int64_t step(int64_t ld) { return ACROSS ? KS * ld * E : STAGE_BYTES; }
  // A descriptor of a stage, whose range ends with the operand's last element:
  // what lies behind it (rows of the tile or k that do not exist) loads as 0.
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const char *base, int64_t bytes) {
    const uint64_t v = reinterpret_cast<uint64_t>(base);
    const uint64_t b = (uint64_t)uni32((int)(v >> 32)) << 32 | (uint32_t)uni32((int)v);
    const int limit = uni32((int)(bytes < 0 ? 0 : lesser(bytes, 0x7fffffff)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(b), (short)0, limit, 0x00020000);
  }
  // Load j of a stage, into LDS; left: k from its first one on that exist, or more than a stage has.
  static __device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t rs, int left, uint32_t off, char *lds, int j) {
    // the last stage of adjacent K: chunks behind it are no rows' ends but the last one's
    if (!ACROSS && chunk(j) * N >= left) off = 0x80000000u;
    const int w = uni32((int)(threadIdx.x >> 6));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_any *)(lds + (w * LOADS + j) * 1024), 16, off, 0, 0, 0);
  }
  __device__ __forceinline__ int left(int64_t k) const { return (int)lesser(k1 - k, KS); }
  // The same through registers, at any alignment.  A stage with another k
  // behind it is loaded by sixteen bytes without a question: a row that does
  // not exist repeats the last one, and of columns that do not exist the first
  // ones or what lies behind the row's end; their sums are not stored.  (Rows
  // across K have to be 16 bytes apart for that to stay inside the operand.)
  __device__ __forceinline__ const T *plain(int64_t k, int j) const {
    const int r = row(j), c = chunk(j) * N;
    return p + (ACROSS ? (k + r) * ld + (c < extent ? c : 0) : lesser(r, extent - 1) * ld + c + k);
  }
  __device__ __forceinline__ bool has_plain() const { return !ACROSS || ld >= N; }
  // Any stage.  Sixteen bytes that do not all exist are loaded as a whole too,
  // unless they go past the operand's last element, and what does not exist
  // along K becomes 0.
  __device__ __forceinline__ uint4 load(int64_t k, int j) const {
    const int r = row(j), c = chunk(j) * N;
    const int64_t have = ACROSS ? (k + r < k1 ? (int64_t)extent - c : 0) : (r < extent ? k1 - k - c : 0);
    const int64_t at = ACROSS ? (k + r) * ld + c : r * ld + k + c;
    if (have >= N) return load16(p + at);
    if (have <= 0) return make_uint4(0, 0, 0, 0);
    if (at + N <= (ACROSS ? (k1 - 1) * ld + extent : (int64_t)(extent - 1) * ld + k1)) {
      const uint4 v = load16(p + at);
      return ACROSS ? v : first_of(v, (int)have);
    }
    T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = i < have ? p[at + i] : T(0);
    uint4 v;
    __builtin_memcpy(&v, e, 16);
    return v;
  }
  // The first n elements (0 < n < N), and zeros.
  static __device__ __forceinline__ uint4 first_of(uint4 v, int n) {
    uint64_t q[2];
    __builtin_memcpy(q, &v, 16);
    const int bits = n * E * 8;
    q[0] &= bits >= 64 ? ~0ull : (1ull << bits) - 1;
    q[1] &= bits <= 64 ? 0ull : (1ull << (bits - 64)) - 1;
    __builtin_memcpy(&v, q, 16);
    return v;
  }
  static __device__ __forceinline__ void put(char *lds, int j, uint4 v) {
    *reinterpret_cast<uint4 *>(lds + ((threadIdx.x >> 6) * LOADS + j) * 1024 + (threadIdx.x & 63) * 16) = v;
  }
};

// The compiler waits for all loads into LDS before a transposing read, unless
// the read carries alias information, as ordinary ones do: `restrict` gives
// it some.  The kernels wait for the loads themselves.
__device__ __forceinline__ i16x4_v read_across(const char *__restrict p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p);
}

// bf16 fragment of 16 tile elements from `at` on and 32 k from 32 ks on: lane l
// holds element l % 16, k 8 (l / 16) to + 7.
template <int BT, bool ACROSS>
__device__ __forceinline__ bf16x8_v read_fragment(const char *lds, int at, int ks) {
  const int lr = threadIdx.x & 15, lg = threadIdx.x >> 4 & 3;
  if constexpr (!ACROSS) {
    return *reinterpret_cast<const bf16x8_v *>(lds + (at + lr) * STAGE_BYTES + adjacent_chunk(lr, 4 * ks + lg) * 16);
  } else {
    const int k = 32 * ks + 8 * lg + (lr >> 2);
    const char *q = lds + k * (BT * 2) + across_chunk<true, BT>(k, at >> 3) * 16 + (lr & 3) * 8;
    union {
      i16x4_v h[2];
      bf16x8_v v;
    } u;
    u.h[0] = read_across(q);
    u.h[1] = read_across(q + 4 * (BT * 2));
    return u.v;
  }
}

// fp32 fragment of 16 tile elements and 16 k from 16 ks on: lane l holds
// element l % 16, k 4 (l / 16) to + 3 (of which product c takes the c-th).
template <int BT, bool ACROSS>
__device__ __forceinline__ f32x4_v read_fragment_f32(const char *lds, int at, int ks) {
  const int lr = threadIdx.x & 15, lg = threadIdx.x >> 4 & 3;
  if constexpr (!ACROSS) {
    return *reinterpret_cast<const f32x4_v *>(lds + (at + lr) * STAGE_BYTES + adjacent_chunk(lr, 4 * ks + lg) * 16);
  } else {
    f32x4_v v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = 16 * ks + 4 * lg + c;
      v[c] = *reinterpret_cast<const float *>(lds + k * (BT * 4) + across_chunk<false, BT>(k, (at + lr) >> 2) * 16 + (lr & 3) * 4);
    }
    return v;
  }
}

// ------------------------------------------------------ sums to memory

// Eight neighbours of a row, n of which exist, as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, int64_t at, int n, float *v) {
  typedef typename Elem<BF16>::type T;
  const T *p = static_cast<const T *>(base) + at;
  if (n >= 8) {
    constexpr int N = Elem<BF16>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) Elem<BF16>::unpack(load16(p + i), v + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<BF16>::get(p[i]) : 0.f;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t at, int n, const float *v) {
  typedef typename Elem<BF16>::type T;
  T *p = static_cast<T *>(base) + at;
  if (n >= 8) {
    constexpr int N = Elem<BF16>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) store16(p + i, Elem<BF16>::pack(v + i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem<BF16>::put(v[i]);
  }
}

// Eight sums of row `row` (in LIN_WEIGHT: of the group's C), columns col to
// col + 7, n of which exist: bias, activation, residual; rounded once.
template <bool BF16>
__device__ __forceinline__ void finish8(const LinearArgs &a, int group, int64_t row, int64_t col, int n, float *v) {
  if (a.mode == LIN_WEIGHT) {
    const int64_t at = group * a.out_stride + row * a.out_ld + col;
    if (!a.first) {
      float w[8];
      load8<false>(a.out, at, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    store8<false>(a.out, at, n, v);
    return;
  }
  float w[8];
  if (a.mode == LIN_FORWARD) {
    if (a.bias) {
      load8<BF16>(a.bias, group * a.N + col, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    if (a.pre) store8<BF16>(a.pre, row * a.pre_ld + col, n, v);
    if (a.act != ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate<BF16>(a.act, v[i]);
    }
  } else if (a.act != ACT_NONE) {
    load8<BF16>(a.pre, row * a.pre_ld + col, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= slope<BF16>(a.act, w[i]);
  }
  if (a.residual) {
    load8<BF16>(a.residual, row * a.res_ld + col, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += w[i];
  }
  store8<BF16>(a.out, row * a.out_ld + col, n, v);
}

// Eight neighbours of a row as they come from memory.
template <bool BF16>
struct Raw8 {
  uint4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void *base, int64_t at) {
    typedef typename Elem<BF16>::type T;
    const T *p = static_cast<const T *>(base) + at;
    v[0] = load16(p);
    if constexpr (!BF16) v[1] = load16(p + 4);
  }
  __device__ __forceinline__ void get(float *f) const {
    Elem<BF16>::unpack(v[0], f);
    if constexpr (!BF16) Elem<BF16>::unpack(v[1], f + 4);
  }
};

// A tile's sums on their way to memory.  Wave (wm, wn) of 2 x 2 holds W x W
// blocks of 16 x 16, lane l of a block row l % 16, columns 4 (l / 16) to + 3.
// Two neighbouring blocks exchange quads between lanes 16 apart
// (v_permlane16_swap), after which a lane has eight neighbours of its row: of
// the first block where l / 16 is even, of the second one where it is odd.

// Column of the tile that a lane's eight of the first pair of blocks begin at;
// the next pairs' are 32 apart.
template <int W>
__device__ __forceinline__ int pair_column(int tid) {
  const int lg = tid >> 4 & 3, wn = tid >> 6 & 1;
  return wn * (16 * W) + (lg & 1) * 16 + (lg >> 1) * 8;
}

// q = row i of blocks, I <= i < W.
template <int W, int I>
__device__ __forceinline__ void pick_row(const f32x4_v (&acc)[W][W], int i, f32x4_v (&q)[W]) {
  if (I == W - 1 || i == I) {
    // (the asm keeps the rows apart: merged, they would index the sums in memory)
#pragma unroll
    for (int j = 0; j < W; ++j) {
      q[j] = acc[I][j];
      asm volatile("" : "+v"(q[j]));
    }
  } else if constexpr (I < W - 1) {
    pick_row<W, I + 1>(acc, i, q);
  }
}

// Row i of blocks, as a lane's eights.
template <int W>
__device__ __forceinline__ void take_row(const f32x4_v (&acc)[W][W], int i, float (&v)[W / 2][8]) {
  f32x4_v q[W];
  pick_row<W, 0>(acc, i, q);
#pragma unroll
  for (int jj = 0; jj < W / 2; ++jj)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto two = __builtin_amdgcn_permlane16_swap(__float_as_uint(q[2 * jj][e]), __float_as_uint(q[2 * jj + 1][e]), false, false);
      v[jj][e] = __uint_as_float(two[0]);
      v[jj][4 + e] = __uint_as_float(two[1]);
    }
}

// Calls f with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_activation(int32_t act, F f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>()); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>()); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>()); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, ACT_NONE>()); break;
  }
}

// A matrix beside the sums, rows of blocks at a time, as buffer accesses: a
// range that ends with the tile's last element leaves out the rows that do not
// exist, and columns that do not are given an offset outside it, so that no
// lane branches.  One wave's half of the tile.
template <bool BF16, int W>
struct TileRows {
  static constexpr int E = BF16 ? 2 : 4, P = W / 2;
  static constexpr int STORES = W * P * (E / 2);  // of a whole tile, by a wave
  const char *base;
  int64_t step;  // bytes of 16 rows
  int64_t range;
  uint32_t off[P];

  __device__ __forceinline__ void init(const void *p, int64_t at, int64_t ld, const LinTile &x, int64_t cols, int tid) {
    const int half = uni32(tid >> 7) * (16 * W), column = pair_column<W>(tid);
    base = static_cast<const char *>(p) + (at + (x.row0 + half) * ld + x.col0) * E;
    step = 16 * ld * E;
    range = ((int64_t)(x.rows - half - 1) * ld + (cols - x.col0)) * E;
    if (x.rows <= half) range = 0;
#pragma unroll
    for (int jj = 0; jj < P; ++jj)
      off[jj] = x.col0 + column + 32 * jj < cols ? (uint32_t)(((tid & 15) * ld + column + 32 * jj) * E) : 0x80000000u;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const { return Operand<BF16, 32 * W, false>::rsrc(base, range); }
  __device__ __forceinline__ void next() {
    base += step;
    range -= step;
  }
  // A row of blocks, then on to the next one (behind the last row: nothing).
  __device__ __forceinline__ void take(Raw8<BF16> (&r)[P]) {
    const auto rs = rsrc();
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int jj = 0; jj < P; ++jj)
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off[jj] + 16 * h, 0, 0));
        r[jj].v[h] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    next();
  }
  __device__ __forceinline__ void store(const float (&v)[P][8]) const {
    const auto rs = rsrc();
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int jj = 0; jj < P; ++jj)
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        const uint4 w = Elem<BF16>::pack(v[jj] + h * Elem<BF16>::N);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{w.x, w.y, w.z, w.w}, rs, off[jj] + 16 * h, 0, 0);
      }
  }
};

// The way of a whole tile whose matrices keep 16-byte alignment, with a
// multiple of 8 columns.  PARTS: of a launch that may be
// cut along K.  What is read beside the sums goes out two rows of blocks ahead.
// MODE: a LinearMode, or -1 for either of the products.
template <bool BF16, int W, int MODE, bool PARTS>
__device__ __forceinline__ void finish_aligned(const LinearArgs &a, const LinTile &x, const f32x4_v (&acc)[W][W], int tid) {
  constexpr int P = W / 2;
  constexpr bool WEIGHT = MODE == LIN_WEIGHT;
  if (PARTS && a.splits > 1) {
    const int64_t all = WEIGHT ? a.M * a.groups : a.M;
    TileRows<false, W> out;
    out.init(a.partial, ((int64_t)x.split * all + (WEIGHT ? x.group * a.M : 0)) * a.N, a.N, x, a.N, tid);
#pragma unroll 1
    for (int i = 0; i < W; ++i) {
      float v[P][8];
      take_row(acc, i, v);
      out.store(v);
      out.next();
    }
  } else if constexpr (WEIGHT) {
    TileRows<false, W> out, old;
    Raw8<false> r[2][P];
    out.init(a.out, x.group * a.out_stride, a.out_ld, x, a.N, tid);
    old = out;
    if (!a.first) {
      old.take(r[0]);
      old.take(r[1]);
    }
#pragma unroll 1
    for (int i = 0; i < W; i += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v[P][8];
        take_row(acc, i + u, v);
        if (!a.first) {
#pragma unroll
          for (int jj = 0; jj < P; ++jj) {
            float f[8];
            r[u][jj].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[jj][e] += f[e];
          }
          old.take(r[u]);
        }
        out.store(v);
        out.next();
      }
    }
  } else {
    const bool forward = MODE < 0 ? a.mode == LIN_FORWARD : MODE == LIN_FORWARD, biased = forward && a.bias, kept = forward && a.pre;
    const bool sloped = !forward && a.act != ACT_NONE;
    TileRows<BF16, W> out, pre, res;
    Raw8<BF16> bias[P], br[2][P], rr[2][P];
    out.init(a.out, 0, a.out_ld, x, a.N, tid);
    if (kept || sloped) pre.init(a.pre, 0, a.pre_ld, x, a.N, tid);
    if (a.residual) res.init(a.residual, 0, a.res_ld, x, a.N, tid);
    if (biased) {
      const int64_t col = x.col0 + pair_column<W>(tid);
#pragma unroll
      for (int jj = 0; jj < P; ++jj) bias[jj].load(a.bias, x.group * a.N + lesser(col + 32 * jj, a.N - 8));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (sloped) pre.take(br[u]);
      if (a.residual) res.take(rr[u]);
    }
    with_activation(a.act, [&](auto act) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act)::value;
#pragma unroll 1
      for (int i = 0; i < W; i += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v[P][8], f[8];
          take_row(acc, i + u, v);
          if (forward) {
            if (biased) {
#pragma unroll
              for (int jj = 0; jj < P; ++jj) {
                bias[jj].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[jj][e] += f[e];
              }
            }
            if (kept) {
              pre.store(v);
              pre.next();
            }
#pragma unroll
            for (int jj = 0; jj < P; ++jj)
#pragma unroll
              for (int e = 0; e < 8; ++e) v[jj][e] = activate<BF16>(ACT, v[jj][e]);
          } else if constexpr (ACT != ACT_NONE) {
#pragma unroll
            for (int jj = 0; jj < P; ++jj) {
              br[u][jj].get(f);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[jj][e] *= slope<BF16>(ACT, f[e]);
            }
            pre.take(br[u]);
          }
          if (a.residual) {
#pragma unroll
            for (int jj = 0; jj < P; ++jj) {
              rr[u][jj].get(f);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[jj][e] += f[e];
            }
            res.take(rr[u]);
          }
          out.store(v);
          out.next();
        }
      }
    });
  }
}

// The same without assumptions.
template <bool BF16, int W, bool WEIGHT>
__device__ __forceinline__ void finish_any(const LinearArgs &a, const LinTile &x, const f32x4_v (&acc)[W][W], int tid) {
  const int64_t col = x.col0 + pair_column<W>(tid);
  float *part = nullptr;
  if (a.splits > 1) part = a.partial + ((int64_t)x.split * (WEIGHT ? a.M * a.groups : a.M) + (WEIGHT ? x.group * a.M : 0)) * a.N;
#pragma unroll 1
  for (int i = 0; i < W; ++i) {
    const int r = (tid >> 7) * (16 * W) + i * 16 + (tid & 15);
    const int64_t row = x.row0 + r;
    float v[W / 2][8];
    take_row(acc, i, v);
    if (r >= x.rows) continue;
#pragma unroll
    for (int jj = 0; jj < W / 2; ++jj) {
      const int64_t c = col + 32 * jj;
      if (c >= a.N) continue;
      const int n = (int)lesser(8, a.N - c);
      if (part) store8<false>(part, row * a.N + c, n, v[jj]);
      else finish8<BF16>(a, x.group, row, c, n, v[jj]);
    }
  }
}

}  // namespace dev
}  // namespace muon
