// Embedding lookup with scaling and its gradient, on gfx950.
//
//   lookup     out[t] = scale * table[ids[t]]
//   gradient   acc[v] (+)= scale * sum of dout[t] over the tokens t with
//              ids[t] = v, added in a fixed order
//
// An id outside the table (padding) has no row: its output is 0 and it adds
// nothing.  The gradient uses no float atomics: the tokens are sorted by row
// (stably, so in token order within a row) and every sum has a fixed order,
// so results are bitwise the same from run to run.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "devops.hpp"
#include "train_ops.hpp"

namespace muon {

using namespace dev;

// ---------------------------------------------------------------- lookup

// HBM-bound: the distinct rows are read once, the rest of the reads hit the
// caches.  `lanes` (a power of two) consecutive threads copy one row, 16
// bytes a thread and step, so a narrow table fills a workgroup with several
// tokens and a wide one gives a token to the whole workgroup.  An output that
// the memory-side cache could not hold beside the table is streamed past it:
// 32768 tokens of 8192 bf16 columns out of 131072 rows take 137 us for the 727
// MB they cannot do without, 5.3 TB/s (a large copy: 4.95), with ordinary
// stores 149; 32768 of 1024 fp32 columns out of 32000 rows 29 and 49.  7 tokens
// of 4096: 3 us, a launch.
template <bool BF16, bool STREAM>
__global__ __launch_bounds__(256) void ke_lookup(EmbedFwdArgs a, int lanes) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  const int per = 256 / lanes;
  const int64_t t = a.token0 + (int64_t)blockIdx.x * per + threadIdx.x / lanes;
  if (t >= a.tokens) return;
  const int64_t id = index_at(a.ids, t);
  const bool has = id >= 0 && id < a.vocab;
  const T *src = static_cast<const T *>(a.table) + (has ? id : 0) * a.table_ld;
  T *dst = static_cast<T *>(a.out) + t * a.out_ld;
  const int64_t step = (int64_t)lanes * E::N;
#pragma unroll 4
  for (int64_t c = (int64_t)(threadIdx.x & (lanes - 1)) * E::N; c < a.dim; c += step) {
    if (c + E::N <= a.dim) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (has) {
        float v[E::N];
        E::unpack(load16(src + c), v);
#pragma unroll
        for (int k = 0; k < E::N; ++k) v[k] *= a.scale;
        w = E::pack(v);
      }
      if constexpr (STREAM) stream16(dst + c, w);
      else store16(dst + c, w);
    } else {
      for (int64_t j = c; j < a.dim; ++j) dst[j] = has ? E::put(E::get(src[j]) * a.scale) : T(0);
    }
  }
}

hipError_t launch_embed_forward(const EmbedFwdArgs &a, bool bf16, hipStream_t s) {
  const int64_t vecs = (a.dim + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);
  int lanes = 1;
  while (lanes < 256 && lanes < vecs) lanes *= 2;
  const int64_t per = 256 / lanes;
  // a grid holds fewer than 2^32 threads: more tokens take several launches
  const int64_t most = ((int64_t)1 << 23) * per;
  // (smaller outputs take the same time either way, and their reader finds them in the cache)
  const bool stream = a.tokens * a.dim * (bf16 ? 2 : 4) >= (64 << 20);
  EmbedFwdArgs b = a;
  for (b.token0 = 0; b.token0 < a.tokens; b.token0 += most) {
    const dim3 grid((unsigned)((std::min(most, a.tokens - b.token0) + per - 1) / per));
    if (bf16 && stream) hipLaunchKernelGGL((ke_lookup<true, true>), grid, dim3(256), 0, s, b, lanes);
    else if (bf16) hipLaunchKernelGGL((ke_lookup<true, false>), grid, dim3(256), 0, s, b, lanes);
    else if (stream) hipLaunchKernelGGL((ke_lookup<false, true>), grid, dim3(256), 0, s, b, lanes);
    else hipLaunchKernelGGL((ke_lookup<false, false>), grid, dim3(256), 0, s, b, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------- sorting the tokens

// One workgroup a bucket (the rows congruent to it modulo EB_BUCKETS, so the
// frequent low ids spread over the buckets).  Every workgroup reads all ids:
// while it collects its own tokens it counts those of the lower buckets, and
// so knows where its part of the sorted order starts without a pass between
// the workgroups.  A bucket of at most ES_SMALL tokens is sorted by counting,
// for each token, the smaller keys in LDS; a larger one by a stable
// least-digit-first radix sort whose digit of 10 bits covers a table of 2^18
// rows in one pass.  Bound by the latency of its dependent steps: 27 us at
// 16384 tokens, 46 with half of the zeros of 32000 x 4096 beside it.
//
// At the first call of a step, as many workgroups more write zeros into rows
// without a token, one bucket's each: the sort waits for memory and the zeros
// for bandwidth, so they fit beside each other on a CU.  The rest of the zeros
// is written beside the sums.
namespace {

constexpr int ES_WAVES = 16, ES_THREADS = 64 * ES_WAVES;
constexpr int ES_BITS = 10, ES_DIGITS = 1 << ES_BITS;
constexpr int ES_MAP_BITS = 1 << 17;  // local rows that one presence map covers
constexpr int ES_HELD = 16;           // ids that a thread reads at a time
constexpr int ES_SMALL = 512;
constexpr int ES_LARGE = 32;          // rows of a bucket that the workgroup cuts into chunks together

struct EsLarge {
  int32_t slot, row, start, len, parts, slot0, tok0;
};
static_assert(ES_DIGITS == ES_THREADS, "one thread a digit in the scan");
static_assert(ES_MAP_BITS / 32 <= ES_WAVES * ES_DIGITS, "the map shares the counts' memory");
static_assert((EB_BUCKETS & (EB_BUCKETS - 1)) == 0, "bucket and key are bits of the row");
constexpr int EB_SHIFT = 8;
static_assert(EB_BUCKETS == 1 << EB_SHIFT, "");

// Rows from here on get their zeros beside the sums.  16384 tokens of 4096
// columns into 32000 rows take 157 us so; with a quarter beside the sort 165,
// with two thirds 164, with all 162.  (Every workgroup that sorts or writes
// zeros reads all ids: 256, and in a first call 256 and 1024 more.  2^20 tokens
// of 1024 bf16 columns take 1.7 ms, in a first call 3.1; the bytes that they
// cannot do without 0.5 at a copy's rate.)
__device__ __forceinline__ int64_t zeros_beside_sort(int64_t vocab) { return vocab / 2; }

constexpr int EF_ZERO_SHIFT = 10;  // log2 of the workgroups that write zeros beside sums

__device__ __forceinline__ uint64_t lanes_below() { return (1ull << (threadIdx.x & 63)) - 1; }

// A token's table row, -1 if it has none.
__device__ __forceinline__ int row_of(const EmbedBwdArgs &a, int64_t t) {
  const int64_t id = index_at(a.ids, t);
  return id >= 0 && id < a.vocab ? (int)id : -1;
}

// Exclusive sum over the workgroup; *total gets the sum.
__device__ __forceinline__ int scan_exclusive(int v, int *wsum, int *total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  int base = 0, sum = 0;
  for (int i = 0; i < ES_WAVES; ++i) {
    if (i == w) base = sum;
    sum += wsum[i];
  }
  *total = sum;
  __syncthreads();
  return base + x - v;
}

// Zeros into the rows of [from, to) congruent to b modulo 2^SHIFT that no token
// meets; map: MAP_BITS bits of LDS.
template <int THREADS, int SHIFT, int MAP_BITS>
__device__ __forceinline__ void zero_rows(const EmbedBwdArgs &a, int b, int64_t from, int64_t to, uint32_t *map) {
  constexpr int MASK = (1 << SHIFT) - 1, ROUND = 8;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rows = (int)((to - b + MASK) >> SHIFT);
  for (int r0 = (int)((from - b + MASK) >> SHIFT); r0 < rows; r0 += MAP_BITS) {
    const int m = min(rows - r0, MAP_BITS);
    for (int i = threadIdx.x; i < (m + 31) / 32; i += THREADS) map[i] = 0;
    __syncthreads();
    for (int64_t t = threadIdx.x; t < a.tokens; t += ROUND * THREADS) {
      int id[ROUND];
#pragma unroll
      for (int q = 0; q < ROUND; ++q) id[q] = t + q * THREADS < a.tokens ? row_of(a, t + q * THREADS) : -1;
#pragma unroll
      for (int q = 0; q < ROUND; ++q) {
        const int r = (id[q] >> SHIFT) - r0;
        if (id[q] >= 0 && (id[q] & MASK) == b && r >= 0 && r < m) atomicOr(&map[r >> 5], 1u << (r & 31));
      }
    }
    __syncthreads();
    for (int r = w; r < m; r += THREADS / 64) {
      if ((map[r >> 5] >> (r & 31)) & 1) continue;
      float *dst = a.acc + (((int64_t)(r0 + r) << SHIFT) + b) * a.acc_ld;
      const Row<false> row(dst, a.dim);
#pragma unroll 4
      for (int i = lane; i < row.vecs; i += 64) stream16(dst + row.col(i), make_uint4(0, 0, 0, 0));
      if (lane < row.singles()) dst[row.single(lane)] = 0.f;
    }
    __syncthreads();
  }
}

}  // namespace

__global__ __launch_bounds__(ES_THREADS, 8) void ke_sort(EmbedBwdArgs a, int passes, int col_blocks) {
  __shared__ __attribute__((aligned(16))) int count[ES_WAVES][ES_DIGITS];
  __shared__ int base[ES_DIGITS];
  __shared__ int wsum[ES_WAVES], wsum2[ES_WAVES];
  __shared__ int n_heavy, n_light, n_parts, n_large;
  __shared__ EsLarge large[ES_LARGE];
  const int b = blockIdx.x, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (b >= EB_BUCKETS) {
    zero_rows<ES_THREADS, EB_SHIFT, ES_MAP_BITS>(a, b - EB_BUCKETS, 0, zeros_beside_sort(a.vocab), reinterpret_cast<uint32_t *>(&count[0][0]));
    return;
  }
  // a wave takes a contiguous span of the tokens, so wave order is token
  // order; up to 16384 tokens its part of the ids is read once
  const int span = (int)((a.tokens + ES_THREADS - 1) / ES_THREADS) * 64;
  const int64_t t0 = min((int64_t)w * span, a.tokens), t1 = min(t0 + span, a.tokens);
  int held[ES_HELD];
  auto read_ids = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < ES_HELD; ++k) {
      held[k] = -1;
      if (t + 64 * k < t1 && t + 64 * k + lane < t1) held[k] = row_of(a, t + 64 * k + lane);
    }
  };
  int mine = 0, lower = 0;
  for (int64_t t = t0; t < t1; t += 64 * ES_HELD) {
    read_ids(t);
#pragma unroll
    for (int k = 0; k < ES_HELD; ++k) {
      if (t + 64 * k < t1) {
        const int bk = held[k] & (EB_BUCKETS - 1);
        mine += __popcll(__ballot(held[k] >= 0 && bk == b));
        lower += __popcll(__ballot(held[k] >= 0 && bk < b));
      }
    }
  }
  if (lane == 0) {
    wsum[w] = mine;
    wsum2[w] = lower;
  }
  if (threadIdx.x == 0) n_heavy = n_light = n_parts = n_large = 0;
  __syncthreads();
  int first = 0, n = 0, at = 0;
  for (int i = 0; i < ES_WAVES; ++i) {
    first += wsum2[i];
    if (i == w) at = n;
    n += wsum[i];
  }
  const bool small = n <= ES_SMALL;
  int *const lkey = &count[0][0], *const ltok = &count[ES_WAVES / 2][0];
  int32_t *key = passes & 1 ? a.key_b : a.key_a, *tok = passes & 1 ? a.tok_b : a.perm;
  int32_t *key2 = passes & 1 ? a.key_a : a.key_b, *tok2 = passes & 1 ? a.perm : a.tok_b;
  key += first;
  tok += first;
  key2 += first;
  tok2 += first;
  if (mine) {
    for (int64_t t = t0; t < t1; t += 64 * ES_HELD) {
      if (span > 64 * ES_HELD) read_ids(t);
#pragma unroll
      for (int k = 0; k < ES_HELD; ++k) {
        if (t + 64 * k < t1) {
          const bool in = held[k] >= 0 && (held[k] & (EB_BUCKETS - 1)) == b;
          const uint64_t m = __ballot(in);
          if (in) {
            const int p = at + __popcll(m & lanes_below());
            (small ? lkey : key)[p] = held[k] >> EB_SHIFT;
            (small ? ltok : tok)[p] = (int32_t)(t + 64 * k + lane);
          }
          at += __popcll(m);
        }
      }
    }
  }
  if (small && threadIdx.x < 4) lkey[n + threadIdx.x] = INT32_MAX;  // no row's key
  __syncthreads();

  // a row's tokens in chunks of EB_CHUNK: chunks of rows with many tokens from
  // the front of the bucket's slots, others from the back.  Neither their
  // order nor that of the slots for partial sums touches the results.  (A row
  // of several chunks has 33 tokens or more and so at most tokens / 16 of
  // them: the bucket's slots are its own from first / 16 on.)
  auto chunk = [&](int slot, int row, int s, int len, int parts, int slot0, int tok0, int i) {
    a.chunks[slot + i] = EbChunk{row, first + s + i * EB_CHUNK, min(EB_CHUNK, len - i * EB_CHUNK), parts, i, slot0, tok0, 0};
    if (parts > 1) {
      for (int j = 0; j < col_blocks; ++j) {
        a.arrive[((int64_t)slot0 + i) * 2 * col_blocks + j] = 0;
        a.arrive[((int64_t)slot0 + i) * 2 * col_blocks + col_blocks + j] = 0;
      }
    }
  };
  auto emit = [&](int k, int s, int len, int tok0) {
    const int parts = (len + EB_CHUNK - 1) / EB_CHUNK, row = k * EB_BUCKETS + b;
    if (len <= EB_LIGHT) {
      chunk(first + n - 1 - atomicAdd(&n_light, 1), row, s, len, 1, 0, tok0, 0);
      return;
    }
    const int slot = first + atomicAdd(&n_heavy, parts);
    const int slot0 = parts > 1 ? first / (EB_CHUNK / 2) + atomicAdd(&n_parts, parts) : 0;
    // a row of very many tokens is left to the whole workgroup
    const int at = parts > 4 ? atomicAdd(&n_large, 1) : ES_LARGE;
    if (at < ES_LARGE) {
      large[at] = EsLarge{slot, row, s, len, parts, slot0, tok0};
    } else {
      for (int i = 0; i < parts; ++i) chunk(slot, row, s, len, parts, slot0, tok0, i);
    }
  };
  auto finish = [&]() {
    __syncthreads();
    for (int j = 0; j < min(n_large, ES_LARGE); ++j) {
      const EsLarge l = large[j];
      for (int i = threadIdx.x; i < l.parts; i += ES_THREADS) chunk(l.slot, l.row, l.start, l.len, l.parts, l.slot0, l.tok0, i);
    }
    if (threadIdx.x == 0) a.buckets[b] = EbBucket{first, n, n_heavy, n_light};
  };

  if (small) {
    const int p = threadIdx.x;
    if (p < n) {
      const int k = lkey[p];
      int less = 0, same = 0, before = 0;
#pragma unroll 4
      for (int q = 0; q < n; q += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(lkey + q);
        less += (o.x < k) + (o.y < k) + (o.z < k) + (o.w < k);
        same += (o.x == k) + (o.y == k) + (o.z == k) + (o.w == k);
        before += (o.x == k && q < p) + (o.y == k && q + 1 < p) + (o.z == k && q + 2 < p) + (o.w == k && q + 3 < p);
      }
      a.perm[first + less + before] = ltok[p];
      if (before == 0) emit(k, less, same, ltok[p]);
    }
    finish();
    return;
  }

  const int span2 = (n + ES_THREADS - 1) / ES_THREADS * 64;
  const int p0 = min(w * span2, n), p1 = min(p0 + span2, n);
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * ES_BITS;
    for (int i = 0; i < ES_WAVES; ++i) count[i][threadIdx.x] = 0;
    __syncthreads();
    for (int p = p0 + lane; p < p1; p += 64) atomicAdd(&count[w][(key[p] >> shift) & (ES_DIGITS - 1)], 1);
    __syncthreads();
    int run = 0, total;
    for (int i = 0; i < ES_WAVES; ++i) {
      const int c = count[i][threadIdx.x];
      count[i][threadIdx.x] = run;
      run += c;
    }
    base[threadIdx.x] = scan_exclusive(run, wsum, &total);
    __syncthreads();
    for (int p = p0; p < p1; p += 64) {
      const bool in = p + lane < p1;
      const int k = in ? key[p + lane] : 0, v = in ? tok[p + lane] : 0;
      const int d = (k >> shift) & (ES_DIGITS - 1);
      uint64_t same = __ballot(in);
#pragma unroll
      for (int i = 0; i < ES_BITS; ++i) {
        const uint64_t m = __ballot((d >> i) & 1);
        same &= (d >> i) & 1 ? m : ~m;
      }
      if (in) {
        const int rank = __popcll(same & lanes_below());
        const int off = count[w][d];
        // the lanes of a digit read before its last lane moves the count on
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if ((same >> lane) == 1) count[w][d] = off + rank + 1;
        key2[base[d] + off + rank] = k;
        tok2[base[d] + off + rank] = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    int32_t *x = key;
    key = key2;
    key2 = x;
    x = tok;
    tok = tok2;
    tok2 = x;
  }

  // the first positions of the rows, in order, into the spare key list
  int32_t *head = key2;
  int heads = 0;
  for (int p = p0; p < p1; p += 64) {
    const int i = p + lane;
    heads += __popcll(__ballot(i < p1 && (i == 0 || key[i] != key[i - 1])));
  }
  if (lane == 0) wsum[w] = heads;
  __syncthreads();
  int n_heads = 0, hat = 0;
  for (int i = 0; i < ES_WAVES; ++i) {
    if (i == w) hat = n_heads;
    n_heads += wsum[i];
  }
  for (int p = p0; p < p1; p += 64) {
    const int i = p + lane;
    const bool is = i < p1 && (i == 0 || key[i] != key[i - 1]);
    const uint64_t m = __ballot(is);
    if (is) head[hat + __popcll(m & lanes_below())] = i;
    hat += __popcll(m);
  }
  __syncthreads();
  for (int h = threadIdx.x; h < n_heads; h += ES_THREADS) {
    const int s = head[h];
    emit(key[s], s, (h + 1 < n_heads ? head[h + 1] : n) - s, tok[s]);
  }
  finish();
}

// ------------------------------------------------------- adding them up

// Units of work, a wave each: (chunk, column block) adds up to EB_CHUNK rows
// of dout, VECS 16-byte vectors a lane.  HBM-bound: each live dout row is
// read once, each gradient row with a token written once.  The units run over
// the buckets' first chunks, then over their second ones, and so on: the
// chunks of many tokens come first and the light ones fill the end.  A wave
// meets another bucket at each turn (141 us a call against 167 with always the
// same, at 16384 tokens of 4096 columns, as the frequent rows' buckets are
// fuller).  At that size the kernel takes 80 us beside half of the zeros, for
// 440 MB: 5.5 TB/s.  Chunk sums of one row are joined 32 at a time and then the
// groups: of 32768 tokens of 4096 columns with 30% in one row a call takes 265
// us, 410 if its last chunk adds up all the others (and one thread of the sort
// lists them).
template <bool BF16, int VECS>
__global__ __launch_bounds__(256) void ke_add(EmbedBwdArgs a, int col_blocks, int zeros) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N, AHEAD = 8 / VECS;
  __shared__ EbBucket bucket[EB_BUCKETS];
  __shared__ int most;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // `zeros` of the workgroups, spread over the grid, write zeros
  const int z = (int)((int64_t)blockIdx.x * zeros / gridDim.x);
  if (z != (int)((int64_t)(blockIdx.x + 1) * zeros / gridDim.x)) {
    zero_rows<256, EF_ZERO_SHIFT, 32 * EB_BUCKETS>(a, z, zeros_beside_sort(a.vocab), a.vocab, reinterpret_cast<uint32_t *>(bucket));
    return;
  }
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  bucket[threadIdx.x] = a.buckets[threadIdx.x];
  atomicMax(&most, bucket[threadIdx.x].heavy + bucket[threadIdx.x].light);
  __syncthreads();
  const uint64_t n_q = (uint64_t)most * EB_BUCKETS;
  const T *dout = static_cast<const T *>(a.dout);
  const uint32_t waves = (gridDim.x - zeros) * 4 / (uint32_t)col_blocks * (uint32_t)col_blocks;
  const uint32_t wave = (blockIdx.x - z) * 4 + w;
  if (wave >= waves) return;
  const int cb = (int)(wave % (uint32_t)col_blocks);
  for (uint64_t q = wave / (uint32_t)col_blocks; q < n_q; q += waves / (uint32_t)col_blocks) {
    const EbBucket bk = bucket[(q + 37 * (q >> EB_SHIFT)) & (EB_BUCKETS - 1)];
    const int at = (int)(q >> EB_SHIFT);
    if (at >= bk.heavy + bk.light) continue;
    const int slot = bk.first + (at < bk.heavy ? at : bk.tokens - 1 - (at - bk.heavy));
    const EbChunk ch = a.chunks[__builtin_amdgcn_readfirstlane(slot)];
    const int count = ch.count;
    const int64_t c0 = (int64_t)cb * (64 * N * VECS) + lane * N;
    int cols[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v) cols[v] = (int)max((int64_t)0, min((int64_t)N, a.dim - c0 - v * 64 * N));
    const int toks = count == 1 && ch.parts == 1 ? ch.tok0 : lane < count ? a.perm[ch.start + lane] : 0;
    float *dst = a.acc + ch.row * a.acc_ld + c0;
    float sum[VECS][N] = {};
    uint4 old[VECS][N / 4];
    const bool add_old = !a.first && ch.parts == 1;
    if (add_old) {
#pragma unroll
      for (int v = 0; v < VECS; ++v)
        if (cols[v] == N) {
#pragma unroll
          for (int j = 0; j < N; j += 4) old[v][j / 4] = load16(dst + v * 64 * N + j);
        }
    }
    auto add = [&](int k, auto steps) {
      constexpr int STEPS = decltype(steps)::value;
      uint4 in[STEPS][VECS];
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        const T *row = dout + (int64_t)__builtin_amdgcn_readlane(toks, k + q) * a.dout_ld + c0;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          in[q][v] = make_uint4(0, 0, 0, 0);
          if (cols[v] == N) in[q][v] = load16(row + v * 64 * N);
        }
      }
#pragma unroll
      for (int q = 0; q < STEPS; ++q)
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          float x[N];
          E::unpack(in[q][v], x);
#pragma unroll
          for (int j = 0; j < N; ++j) sum[v][j] += x[j];
        }
    };
    int k = 0;
    for (; k + AHEAD <= count; k += AHEAD) add(k, std::integral_constant<int, AHEAD>());
    for (; k < count; ++k) add(k, std::integral_constant<int, 1>());
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      if (cols[v] > 0 && cols[v] < N) {  // the row's last elements
        for (k = 0; k < count; ++k) {
          const T *row = dout + (int64_t)__builtin_amdgcn_readlane(toks, k) * a.dout_ld + c0 + v * 64 * N;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j < cols[v]) sum[v][j] += E::get(row[j]);
        }
      }
    }
    if (ch.parts > 1) {
      // the row's chunks meet here: each leaves its sum, the last of a group
      // adds the group's in their order, and the last of the groups the
      // groups' (which one is last does not matter).  A lane's elements lie
      // 64 apart, so that the lanes' stores touch.
      const int64_t width = (int64_t)col_blocks * (64 * N * VECS);
      float *part = a.partials + ch.slot0 * width + (int64_t)cb * (64 * N * VECS) + lane;
      int32_t *count2 = a.arrive + ((int64_t)ch.slot0 * 2 * col_blocks + cb);
      auto leave = [&](int slot) {
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
          for (int j = 0; j < N; ++j) put_shared(part + slot * width + 64 * (v * N + j), sum[v][j]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // of all lanes
      };
      auto join = [&](int slot, int slots, int step) {
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
          for (int j = 0; j < N; ++j) sum[v][j] = 0.f;
#pragma unroll 2
        for (int i = 0; i < slots; ++i) {
          const float *p = part + (int64_t)(slot + i * step) * width;
#pragma unroll
          for (int v = 0; v < VECS; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) sum[v][j] += get_shared(p + 64 * (v * N + j));
        }
      };
      auto count_in = [&](int32_t *c) {
        int before = 0;
        if (lane == 0) before = arrive(c);
        return __builtin_amdgcn_readfirstlane(before);
      };
      const int g0 = ch.index / EB_GROUP * EB_GROUP, members = min(EB_GROUP, ch.parts - g0);
      const int groups = (ch.parts + EB_GROUP - 1) / EB_GROUP;
      leave(ch.index);
      if (count_in(count2 + (int64_t)g0 * 2 * col_blocks) != members - 1) continue;
      join(g0, members, 1);
      if (groups > 1) {
        leave(g0);
        if (count_in(count2 + col_blocks) != groups - 1) continue;
        join(0, groups, EB_GROUP);
      }
    }
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      float *out = dst + v * 64 * N;
#pragma unroll
      for (int j = 0; j < N; ++j) sum[v][j] *= a.scale;
      if (cols[v] == N) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          float o[4] = {};
          if (!a.first) Elem<false>::unpack(add_old ? old[v][j / 4] : load16(out + j), o);
          for (int q = 0; q < 4; ++q) o[q] += sum[v][j + q];
          store16(out + j, Elem<false>::pack(o));
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j < cols[v]) out[j] = a.first ? sum[v][j] : out[j] + sum[v][j];
      }
    }
  }
}

// ------------------------------------------------------- few tokens

// Up to EB_FEW tokens need no sort: a workgroup takes (token t, column block),
// finds the tokens of the same row among all ids, ends if one of them comes
// before t, and otherwise adds them up, each wave those of its quarter of the
// ids; the waves' sums are joined in their order.  Bound by the latency of
// its dependent loads (ids, then dout rows) and the launch.  The other
// workgroups write the zeros of a first call.  In us, so and with a sort, ids
// at word frequencies: 1021 tokens of 64 bf16 columns 8.3 16.6, of 1024 fp32
// ones 8.8 17.6, of 4096 bf16 14.3 24.6, of 8192 21.9 26.9; 1000 tokens into a
// first call's 32000 rows of 1024 30 33.  Every workgroup reads all ids, so
// twice the tokens are four times the reads, and more ids a lane slow the
// smaller calls too: with 2048 as the limit 2000 tokens of 64 columns take 9.6
// (sorted 19.5) and of 1024 14.7 (23.2), but of 4096 29.6 (28.9), 1500 of 8192
// 38.8 (29.7), and 1021 of 8192 29.2.  One workgroup a column block adds up a
// row's tokens however many they are: 1000 tokens of 4096 bf16 columns take 31
// (sorted 35) with 30% of them in one row, 74 (32) with all.
namespace {

constexpr int EF_IDS = EB_FEW / 256;  // ids that a lane holds

}  // namespace

template <bool BF16, int VECS>
__global__ __launch_bounds__(256) void ke_few(EmbedBwdArgs a, int zeros) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int N = E::N, COLS = 64 * N * VECS, AHEAD = 8 / VECS;
  __shared__ __attribute__((aligned(16))) float part[3][COLS];  // sums of waves 1 to 3
  __shared__ int before, has[4];
  if ((int)blockIdx.x < zeros) {
    __shared__ uint32_t map[1 << 8];
    zero_rows<256, EF_ZERO_SHIFT, 32 << 8>(a, blockIdx.x, 0, a.vocab, map);
    return;
  }
  const uint32_t i0 = blockIdx.x - zeros;
  const int t = (int)(i0 % (uint32_t)a.tokens), cb = (int)(i0 / (uint32_t)a.tokens), lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mine = row_of(a, t);
  int id[EF_IDS];
#pragma unroll
  for (int k = 0; k < EF_IDS; ++k) {
    const int j = (w * EF_IDS + k) * 64 + lane;
    id[k] = j < a.tokens ? row_of(a, j) : -1;
  }
  if (mine < 0) return;
  if (threadIdx.x == 0) before = 0;
  __syncthreads();
  uint64_t same[EF_IDS];
  int n = 0;
  bool late = false;
#pragma unroll
  for (int k = 0; k < EF_IDS; ++k) {
    same[k] = __ballot(id[k] == mine);
    n += __popcll(same[k]);
    late = late || (same[k] && (w * EF_IDS + k) * 64 + __builtin_ctzll(same[k]) < t);
  }
  if (lane == 0) {
    has[w] = n;
    if (late) before = 1;
  }
  const int64_t c0 = (int64_t)cb * COLS + lane * N;
  float *dst = a.acc + mine * a.acc_ld + c0;
  int cols[VECS];
  uint4 old[VECS][N / 4];
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    cols[v] = (int)max((int64_t)0, min((int64_t)N, a.dim - c0 - v * 64 * N));
    if (w == 0 && !a.first && cols[v] == N) {
#pragma unroll
      for (int j = 0; j < N; j += 4) old[v][j / 4] = load16(dst + v * 64 * N + j);
    }
  }
  __syncthreads();
  if (before) return;
  float sum[VECS][N] = {};
  const T *dout = static_cast<const T *>(a.dout) + c0;
  // the wave's tokens in order: the k-th set bit of the masks
  int word = 0;
  uint64_t left = same[0];
  auto pop = [&]() {
    while (!left) {
      ++word;
#pragma unroll
      for (int k = 1; k < EF_IDS; ++k)
        if (word == k) left = same[k];
    }
    const int j = (w * EF_IDS + word) * 64 + __builtin_ctzll(left);
    left &= left - 1;
    return j;
  };
  for (int k = 0; k < n; k += AHEAD) {
    uint4 in[AHEAD][VECS];
    const int m = min(AHEAD, n - k);
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const T *row = dout;
      if (q < m) row += (int64_t)pop() * a.dout_ld;
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        in[q][v] = make_uint4(0, 0, 0, 0);
        if (q < m) {
          if (cols[v] == N) {
            in[q][v] = load16(row + v * 64 * N);
          } else if (cols[v] > 0) {  // the row's last elements
            float x[N];
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = j < cols[v] ? E::get(row[v * 64 * N + j]) : 0.f;
            in[q][v] = E::pack(x);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        float x[N];
        E::unpack(in[q][v], x);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[v][j] += x[j];
      }
  }
  if (w > 0 && n > 0) {
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
      for (int j = 0; j < N; j += 4)
        *reinterpret_cast<uint4 *>(&part[w - 1][(v * 64 + lane) * N + j]) = Elem<false>::pack(&sum[v][j]);
  }
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (!has[i]) continue;
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
      for (int j = 0; j < N; ++j) sum[v][j] += part[i - 1][(v * 64 + lane) * N + j];
  }
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    float *out = dst + v * 64 * N;
#pragma unroll
    for (int j = 0; j < N; ++j) sum[v][j] *= a.scale;
    if (cols[v] == N) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        float o[4] = {};
        if (!a.first) Elem<false>::unpack(old[v][j / 4], o);
        for (int q = 0; q < 4; ++q) o[q] += sum[v][j + q];
        store16(out + j, Elem<false>::pack(o));
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j < cols[v]) out[j] = a.first ? sum[v][j] : out[j] + sum[v][j];
    }
  }
}

EbLayout embed_layout(int64_t tokens, int64_t vocab, int64_t dim) {
  (void)vocab;
  EbLayout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t n = (size_t)tokens, slots = n / (EB_CHUNK / 2) + 1;  // of partial sums
  l.buckets = take(EB_BUCKETS * sizeof(EbBucket));
  l.perm = take(4 * n);
  l.key_a = take(4 * n);
  l.key_b = take(4 * n);
  l.tok_b = take(4 * n);
  l.chunks = take(sizeof(EbChunk) * n);
  // a row of at most EB_CHUNK tokens leaves no partial sums; a slot holds the
  // columns up to whole column blocks, of either type's width
  const size_t width = dim > 512 ? ((size_t)dim + 1023) / 1024 * 1024 : 512;
  l.partials = take(n > EB_CHUNK ? slots * width * 4 : 0);
  l.arrive = take(n > EB_CHUNK ? slots * 2 * (width / 256) * 4 : 0);  // a chunk's group, and its row's groups
  l.total = at;
  return l;
}

namespace {

template <bool BF16>
hipError_t add_launch(const EmbedBwdArgs &a, int passes, hipStream_t s) {
  constexpr int WAVE_COLS = 64 * Elem<BF16>::N;
  const bool wide = a.dim > WAVE_COLS;
  const int cols = WAVE_COLS * (wide ? 2 : 1), col_blocks = (int)((a.dim + cols - 1) / cols);
  if (a.tokens <= EB_FEW && a.tokens * col_blocks <= (1 << 23)) {
    const int zeros = a.first ? (int)std::min<int64_t>(a.vocab, 1 << EF_ZERO_SHIFT) : 0;
    const unsigned grid = (unsigned)(zeros + a.tokens * col_blocks);
    if (grid == 0) return hipSuccess;
    if (wide) hipLaunchKernelGGL((ke_few<BF16, 2>), dim3(grid), dim3(256), 0, s, a, zeros);
    else hipLaunchKernelGGL((ke_few<BF16, 1>), dim3(grid), dim3(256), 0, s, a, zeros);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(ke_sort, dim3(EB_BUCKETS + (a.first ? (unsigned)std::min<int64_t>(a.vocab, EB_BUCKETS) : 0)),
                     dim3(ES_THREADS), 0, s, a, passes, col_blocks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.tokens == 0) return e;
  const unsigned grid = (unsigned)std::max<int64_t>(col_blocks, std::min<int64_t>((a.tokens * col_blocks + 7) / 8, 4096));
  const int zeros = a.first ? (int)std::min<int64_t>(a.vocab, 1 << EF_ZERO_SHIFT) : 0;
  if (wide) hipLaunchKernelGGL((ke_add<BF16, 2>), dim3(grid + zeros), dim3(256), 0, s, a, col_blocks, zeros);
  else hipLaunchKernelGGL((ke_add<BF16, 1>), dim3(grid + zeros), dim3(256), 0, s, a, col_blocks, zeros);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_backward(const EmbedBwdArgs &a, bool bf16, hipStream_t s) {
  int passes = 1;
  while (((a.vocab - 1) >> EB_SHIFT) >> (passes * ES_BITS)) ++passes;
  return bf16 ? add_launch<true>(a, passes, s) : add_launch<false>(a, passes, s);
}

}  // namespace muon
