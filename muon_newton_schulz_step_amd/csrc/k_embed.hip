// Embedding lookup with scaling and its gradient, on gfx950.
//
//   lookup     out[t] = scale * table[ids[t]]
//   gradient   acc[v] (+)= scale * sum of dout[t] over the tokens t with
//              ids[t] = v, added in token order
//
// An id outside the table (padding) has no row: its output is 0 and it adds
// nothing.  The gradient uses no float atomics: the tokens are sorted by row
// (stably, so in token order within a row) and every sum has a fixed order,
// so results are bitwise the same from run to run.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "devops.hpp"
#include "train_ops.hpp"

namespace muon {

using namespace dev;

// ---------------------------------------------------------------- lookup

// HBM-bound: the distinct rows are read once, the rest of the reads hit the
// caches.  `lanes` (a power of two) consecutive threads copy one row, 16
// bytes a thread and step, so a narrow table fills a workgroup with several
// tokens and a wide one gives a token to the whole workgroup.
template <bool BF16>
__global__ __launch_bounds__(256) void ke_lookup(EmbedFwdArgs a, int lanes) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  const int per = 256 / lanes;
  const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
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
      store16(dst + c, w);
    } else {
      for (int64_t j = c; j < a.dim; ++j) dst[j] = has ? E::put(E::get(src[j]) * a.scale) : T(0);
    }
  }
}

hipError_t launch_embed_forward(const EmbedFwdArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t vecs = (a.dim + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);
  int lanes = 1;
  while (lanes < 256 && lanes < vecs) lanes *= 2;
  const int64_t per = 256 / lanes, grid = (a.tokens + per - 1) / per;
  if (bf16) hipLaunchKernelGGL(ke_lookup<true>, dim3((unsigned)grid), dim3(256), 0, s, a, lanes);
  else hipLaunchKernelGGL(ke_lookup<false>, dim3((unsigned)grid), dim3(256), 0, s, a, lanes);
  return hipGetLastError();
}

// ---------------------------------------------------- sorting the tokens

// One workgroup a bucket (the rows congruent to it modulo EB_BUCKETS, so the
// frequent low ids spread over the buckets).  Every workgroup reads all ids:
// while it collects its own tokens it counts those of the lower buckets, and
// so knows where its part of the sorted order starts without a pass between
// the workgroups.  Inside the bucket the tokens go through a stable
// least-digit-first radix sort; a digit of 10 bits covers a table of 2^18
// rows in one pass.
namespace {

constexpr int ES_WAVES = 16, ES_THREADS = 64 * ES_WAVES;
constexpr int ES_BITS = 10, ES_DIGITS = 1 << ES_BITS;
constexpr int ES_MAP_BITS = 1 << 17;  // local rows that one presence map covers
static_assert(ES_DIGITS == ES_THREADS, "one thread a digit in the scan");
static_assert(ES_MAP_BITS / 32 <= ES_WAVES * ES_DIGITS, "the map shares the counts' memory");

__device__ __forceinline__ uint64_t lanes_below() { return (1ull << (threadIdx.x & 63)) - 1; }

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

}  // namespace

__global__ __launch_bounds__(ES_THREADS) void ke_sort(EmbedBwdArgs a, int passes, int col_blocks) {
  __shared__ int count[ES_WAVES][ES_DIGITS];
  __shared__ int base[ES_DIGITS];
  __shared__ int wsum[ES_WAVES], wsum2[ES_WAVES];
  __shared__ int n_chunks, n_empty;
  const int b = blockIdx.x, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t span = (a.tokens + ES_THREADS - 1) / ES_THREADS * 64;
  const int64_t t0 = min((int64_t)w * span, a.tokens), t1 = min(t0 + span, a.tokens);

  // a wave takes a contiguous span of the tokens, so wave order is token order
  int mine = 0, lower = 0;
#pragma unroll 4
  for (int64_t t = t0; t < t1; t += 64) {
    const int64_t id = t + lane < t1 ? index_at(a.ids, t + lane) : -1;
    const bool ok = id >= 0 && id < a.vocab;
    const int bk = (int)(id & (EB_BUCKETS - 1));
    mine += __popcll(__ballot(ok && bk == b));
    lower += __popcll(__ballot(ok && bk < b));
  }
  if (lane == 0) {
    wsum[w] = mine;
    wsum2[w] = lower;
  }
  if (threadIdx.x == 0) n_chunks = n_empty = 0;
  __syncthreads();
  int first = 0, n = 0, at = 0;
  for (int i = 0; i < ES_WAVES; ++i) {
    first += wsum2[i];
    if (i == w) at = n;
    n += wsum[i];
  }
  int32_t *key = passes & 1 ? a.key_b : a.key_a, *tok = passes & 1 ? a.tok_b : a.perm;
  int32_t *key2 = passes & 1 ? a.key_a : a.key_b, *tok2 = passes & 1 ? a.perm : a.tok_b;
  key += first;
  tok += first;
  key2 += first;
  tok2 += first;
  if (mine) {
#pragma unroll 4
    for (int64_t t = t0; t < t1; t += 64) {
      const int64_t id = t + lane < t1 ? index_at(a.ids, t + lane) : -1;
      const bool in = id >= 0 && id < a.vocab && (int)(id & (EB_BUCKETS - 1)) == b;
      const uint64_t m = __ballot(in);
      if (in) {
        const int p = at + __popcll(m & lanes_below());
        key[p] = (int32_t)(id / EB_BUCKETS);
        tok[p] = (int32_t)(t + lane);
      }
      at += __popcll(m);
    }
  }
  __syncthreads();

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

  // work chunks: a row's tokens in nearly equal parts of at most EB_CHUNK
  // (their order in the list does not touch the results)
  for (int h = threadIdx.x; h < n_heads; h += ES_THREADS) {
    const int s = head[h], len = (h + 1 < n_heads ? head[h + 1] : n) - s;
    const int parts = (len + EB_CHUNK - 1) / EB_CHUNK;
    const int slot = atomicAdd(&n_chunks, parts);
    const int row = key[s] * EB_BUCKETS + b;
    for (int i = 0; i < parts; ++i) {
      const int lo = (int)((int64_t)len * i / parts), hi = (int)((int64_t)len * (i + 1) / parts);
      a.chunks[first + slot + i] = EbChunk{row, first + s + lo, hi - lo, parts, first + s, len};
    }
    if (parts > 1) {
      for (int j = 0; j < col_blocks; ++j) a.arrive[(int64_t)((first + s) / (EB_CHUNK / 2)) * col_blocks + j] = 0;
    }
  }

  // the bucket's rows without a token
  if (a.first) {
    const int per = (int)((a.vocab + EB_BUCKETS - 1) / EB_BUCKETS);
    const int rows = (int)((a.vocab - b + EB_BUCKETS - 1) / EB_BUCKETS);
    uint32_t *map = reinterpret_cast<uint32_t *>(&count[0][0]);
    for (int r0 = 0; r0 < rows; r0 += ES_MAP_BITS) {
      const int m = min(rows - r0, ES_MAP_BITS);
      for (int i = threadIdx.x; i < (m + 31) / 32; i += ES_THREADS) map[i] = 0;
      __syncthreads();
      for (int h = threadIdx.x; h < n_heads; h += ES_THREADS) {
        const int r = key[head[h]] - r0;
        if (r >= 0 && r < m) atomicOr(&map[r >> 5], 1u << (r & 31));
      }
      __syncthreads();
      for (int r = threadIdx.x; r < m; r += ES_THREADS) {
        if (!((map[r >> 5] >> (r & 31)) & 1)) {
          a.empty[(int64_t)b * per + atomicAdd(&n_empty, 1)] = (r0 + r) * EB_BUCKETS + b;
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.buckets[b] = EbBucket{first, n, n_chunks, n_empty};
}

// ------------------------------------------------------- adding them up

// Units of work, a wave each: (chunk, column block) adds up to EB_CHUNK rows
// of dout, (empty row, column block) writes zeros.  HBM-bound: each live
// dout row is read once, each gradient row written once.
template <bool BF16>
__global__ __launch_bounds__(256) void ke_add(EmbedBwdArgs a, int col_blocks) {
  typedef Elem<BF16> E;
  typedef typename E::type T;
  constexpr int COLS = 64 * E::N;   // columns of a wave
  constexpr int ZCOLS = 2048;       // columns of a wave that writes zeros
  __shared__ int chunk0[EB_BUCKETS + 1], empty0[EB_BUCKETS + 1];
  {
    // exclusive sums of the buckets' unit counts (256 threads, 256 buckets)
    const EbBucket k = a.buckets[threadIdx.x];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int x = k.chunks, y = k.empty;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int u = __shfl_up(x, d), v = __shfl_up(y, d);
      if (lane >= d) {
        x += u;
        y += v;
      }
    }
    __shared__ int wx[4], wy[4];
    if (lane == 63) {
      wx[w] = x;
      wy[w] = y;
    }
    __syncthreads();
    for (int i = 0; i < w; ++i) {
      x += wx[i];
      y += wy[i];
    }
    chunk0[threadIdx.x + 1] = x;
    empty0[threadIdx.x + 1] = y;
    if (threadIdx.x == 0) chunk0[0] = empty0[0] = 0;
    __syncthreads();
  }
  auto bucket_of = [](const int *start, int i) {
    int lo = 0, hi = EB_BUCKETS - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  const int lane = threadIdx.x & 63;
  const int zblocks = (int)((a.dim + ZCOLS - 1) / ZCOLS);
  const int64_t n_chunk_units = (int64_t)chunk0[EB_BUCKETS] * col_blocks;
  const int64_t n_units = n_chunk_units + (int64_t)empty0[EB_BUCKETS] * zblocks;
  const int per = (int)((a.vocab + EB_BUCKETS - 1) / EB_BUCKETS);
  const T *dout = static_cast<const T *>(a.dout);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < n_units; u += (int64_t)gridDim.x * 4) {
    if (u >= n_chunk_units) {
      const int64_t z = u - n_chunk_units;
      const int i = (int)(z / zblocks);
      const int bk = bucket_of(empty0, i);
      float *dst = a.acc + a.empty[(int64_t)bk * per + i - empty0[bk]] * a.acc_ld;
      const int64_t c0 = z % zblocks * ZCOLS, c1 = min(c0 + ZCOLS, a.dim);
      for (int64_t c = c0 + 4 * lane; c < c1; c += 256) {
        if (c + 4 <= c1) store16(dst + c, make_uint4(0, 0, 0, 0));
        else
          for (int64_t j = c; j < c1; ++j) dst[j] = 0.f;
      }
      continue;
    }
    const int i = (int)(u / col_blocks), cb = (int)(u % col_blocks);
    const int bk = bucket_of(chunk0, i);
    const EbChunk ch = a.chunks[a.buckets[bk].first + i - chunk0[bk]];
    const int64_t c = (int64_t)cb * COLS + lane * E::N;
    const int cols = (int)max((int64_t)0, min((int64_t)E::N, a.dim - c));
    float sum[E::N] = {};
    if (cols == E::N) {
#pragma unroll 4
      for (int k = 0; k < ch.count; ++k) {
        float v[E::N];
        E::unpack(load16(dout + a.perm[ch.start + k] * a.dout_ld + c), v);
#pragma unroll
        for (int j = 0; j < E::N; ++j) sum[j] += v[j];
      }
    } else if (cols > 0) {
      for (int k = 0; k < ch.count; ++k) {
        const T *row = dout + a.perm[ch.start + k] * a.dout_ld + c;
#pragma unroll
        for (int j = 0; j < E::N; ++j)
          if (j < cols) sum[j] += E::get(row[j]);
      }
    }
    if (ch.parts > 1) {
      // the row's chunks meet here: each leaves its sum, the last to arrive
      // adds them in their order (which one is last does not matter)
      const int slot0 = ch.seg / (EB_CHUNK / 2);
      float *mine = a.partials + (int64_t)(ch.start / (EB_CHUNK / 2)) * a.dim + c;
#pragma unroll
      for (int j = 0; j < E::N; ++j)
        if (j < cols) mine[j] = sum[j];
      int before = 0;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
      if (lane == 0)
        before = __hip_atomic_fetch_add(&a.arrive[(int64_t)slot0 * col_blocks + cb], 1, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
      before = __builtin_amdgcn_readfirstlane(before);
      if (before != ch.parts - 1) continue;
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
#pragma unroll
      for (int j = 0; j < E::N; ++j) sum[j] = 0.f;
      for (int k = 0; k < ch.parts; ++k) {
        const int st = ch.seg + (int)((int64_t)ch.seg_count * k / ch.parts);
        const float *p = a.partials + (int64_t)(st / (EB_CHUNK / 2)) * a.dim + c;
#pragma unroll
        for (int j = 0; j < E::N; ++j)
          if (j < cols) sum[j] += p[j];
      }
    }
    float *dst = a.acc + ch.row * a.acc_ld + c;
#pragma unroll
    for (int j = 0; j < E::N; ++j) sum[j] *= a.scale;
    if (cols == E::N) {
#pragma unroll
      for (int j = 0; j < E::N; j += 4) {
        float4 v = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
        if (!a.first) {
          float4 o;
          __builtin_memcpy(&o, dst + j, 16);
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        __builtin_memcpy(dst + j, &v, 16);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E::N; ++j)
        if (j < cols) dst[j] = a.first ? sum[j] : dst[j] + sum[j];
    }
  }
}

EbLayout embed_layout(int64_t tokens, int64_t vocab, int64_t dim) {
  EbLayout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t n = (size_t)tokens, slots = n / (EB_CHUNK / 2) + 1;
  l.buckets = take(EB_BUCKETS * sizeof(EbBucket));
  l.perm = take(4 * n);
  l.key_a = take(4 * n);
  l.key_b = take(4 * n);
  l.tok_b = take(4 * n);
  l.chunks = take(sizeof(EbChunk) * n);
  l.empty = take(4 * ((size_t)vocab + EB_BUCKETS));
  // a row of at most EB_CHUNK tokens leaves no partial sums
  l.partials = take(n > EB_CHUNK ? slots * (size_t)dim * 4 : 0);
  l.arrive = take(n > EB_CHUNK ? slots * (((size_t)dim + 255) / 256) * 4 : 0);
  l.total = at;
  return l;
}

hipError_t launch_embed_backward(const EmbedBwdArgs &a, bool bf16, hipStream_t s) {
  const int cols = bf16 ? 512 : 256;
  const int col_blocks = (int)((a.dim + cols - 1) / cols);
  int passes = 1;
  while (((a.vocab - 1) / EB_BUCKETS) >> (passes * ES_BITS)) ++passes;
  hipLaunchKernelGGL(ke_sort, dim3(EB_BUCKETS), dim3(ES_THREADS), 0, s, a, passes, col_blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t units = a.tokens * col_blocks + (a.first ? a.vocab * ((a.dim + 2047) / 2048) : 0);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((units + 3) / 4, 2048));
  if (bf16) hipLaunchKernelGGL(ke_add<true>, dim3(grid), dim3(256), 0, s, a, col_blocks);
  else hipLaunchKernelGGL(ke_add<false>, dim3(grid), dim3(256), 0, s, a, col_blocks);
  return hipGetLastError();
}

}  // namespace muon
