// Device helpers of the training-step operators: 16-byte element vectors,
// bf16 conversion, index loads and fixed-order reductions.
#pragma once

#include <hip/hip_runtime.h>

#include "train_ops.hpp"

namespace muon {
namespace dev {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);  // what fp32 leaves of it
// Start of a running maximum: the lowest finite value, so that a row of
// -inf keeps a finite maximum and sums to exactly 0 instead of NaN.
constexpr float kLowest = -3.402823466e+38f;

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// fp32 pair -> packed bf16, round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Elements of one 16-byte vector, and their conversion.
template <bool BF16>
struct Elem;
template <>
struct Elem<true> {
  typedef uint16_t type;
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(type x) { return bf16_f32(x); }
  static __device__ __forceinline__ type put(float x) { return (type)pack_bf16(x, 0.f); }
  static __device__ __forceinline__ uint4 none() {  // -inf in every element
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __forceinline__ void unpack(uint4 w, float *v) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(x[k] << 16);
      v[2 * k + 1] = __uint_as_float(x[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <>
struct Elem<false> {
  typedef float type;
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(type x) { return x; }
  static __device__ __forceinline__ type put(float x) { return x; }
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ __forceinline__ void unpack(uint4 w, float *v) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// 16-byte accesses at element alignment (the hardware takes any alignment of
// a 16-byte global access; an access off its own 16 bytes only costs more).
template <class T>
__device__ __forceinline__ uint4 load16(const T *p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
template <class T>
__device__ __forceinline__ void store16(T *p, uint4 v) {
  __builtin_memcpy(p, &v, 16);
}
// A store that leaves the caches to what is read again.
template <class T>
__device__ __forceinline__ void stream16(T *p, uint4 v) {
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
  const words w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<words *>(p));
}

__device__ __forceinline__ int64_t index_at(const IndexVec &v, int64_t i) {
  return v.is64 ? static_cast<const int64_t *>(v.p)[i] : (int64_t)static_cast<const int32_t *>(v.p)[i];
}

// exp of a non-positive shifted logit: the difference is taken before the
// change of base, so values at either end of the fp32 range cannot turn an
// infinite product into NaN.
__device__ __forceinline__ float exp_shift(float x, float m) { return __builtin_amdgcn_exp2f((x - m) * kLog2e); }

// The same for terms of a row's sum.  log2(e) rounded to fp32 is low by 1.3e-8
// of itself, an error of one sign in every term: a sequence adds up hundreds
// of rows' log-probabilities, so the constant's rest is added back.
__device__ __forceinline__ float exp_term(float x, float m) {
  const float d = x - m;
  return __builtin_amdgcn_exp2f(fmaf(d, kLog2e, d * kLog2eLow));
}

// And for the elements of a gradient of either type: a bf16 result's rounding
// (2^-8) hides the constant's rest, fp32 ones would all be off to one side.
template <bool BF16>
__device__ __forceinline__ float exp_grad(float x, float m) {
  return BF16 ? exp_shift(x, m) : exp_term(x, m);
}

// A value that is the same in all lanes of a wave, moved to scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double shfl_f64(double v, int lane) {
  union {
    double d;
    int i[2];
  } u;
  u.d = v;
  u.i[0] = __shfl(u.i[0], lane);
  u.i[1] = __shfl(u.i[1], lane);
  return u.d;
}

__device__ __forceinline__ double shfl_xor_f64(double v, int m) {
  union {
    double d;
    int i[2];
  } u;
  u.d = v;
  u.i[0] = __shfl_xor(u.i[0], m);
  u.i[1] = __shfl_xor(u.i[1], m);
  return u.d;
}

// A row of a matrix as the kernels walk it: 16-byte vectors from its first
// 128-byte line on, and what is left at either end (less than a line before
// them, less than a vector after them) element by element.  Over 50257-column
// bf16 rows, reads off 4 bytes cost a quarter of the bandwidth (4.9 against
// 6.1 TB/s), and streamed stores off their line write it in two parts: the
// policy loss took 541 us on odd rows, 466 on rows at 4 bytes, 446 at 8.
template <bool BF16>
struct Row {
  int head, vecs, n;
  __device__ __forceinline__ Row(const void *p, int64_t cols) {
    n = (int)cols;
    head = min((int)((0u - (uint32_t)(uintptr_t)p) & 127u) / (int)sizeof(typename Elem<BF16>::type), n);
    vecs = (n - head) / Elem<BF16>::N;
  }
  // column of a vector's first element
  __device__ __forceinline__ uint32_t col(int vec) const { return (uint32_t)(head + vec * Elem<BF16>::N); }
  // single elements (fewer than 80), and the column of the i-th
  __device__ __forceinline__ int singles() const { return n - vecs * Elem<BF16>::N; }
  __device__ __forceinline__ uint32_t single(int i) const {
    return (uint32_t)(i < head ? i : vecs * Elem<BF16>::N + i);
  }
};

// Values passed between workgroups of one launch, past the caches that are not
// shared by all of them.  arrive() counts a wave in after its stores have
// reached memory, and returns how many came before it: whoever learns that
// all did may read what they put.  (A release and an acquire fence of device
// scope would write back and invalidate a whole L2: the sums of the embedding
// gradient of 16384 tokens took 195 us so, 76 without.)
template <class T>
__device__ __forceinline__ void put_shared(T *p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get_shared(const T *p) {
  return __hip_atomic_load(const_cast<T *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int arrive(int32_t *count) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  const int before = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("" ::: "memory");
  return before;
}

// Sum over a workgroup of WAVES waves in a fixed order; every thread gets
// it.  `red` holds WAVES doubles and is free again after the call.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += shfl_xor_f64(v, m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += red[w];
  __syncthreads();
  return t;
}

}  // namespace dev
}  // namespace muon
