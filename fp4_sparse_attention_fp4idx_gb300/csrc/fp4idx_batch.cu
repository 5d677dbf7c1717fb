// fp4idx_batch.cu -- pages and maps of a step (fp4idx_batch_extend,
// fp4idx_pages_release, defined in include/fp4idx_step.h).
//
// What bounds it.  24 bytes written for each token (8 of page table and stack
// for each 64), 8 to 20 read and written for each sequence: for a decode step
// nothing but latency, so everything is one launch.  Both calls are a running
// sum over the sequences and then, for every token (every page), the search for
// its sequence in those sums.  Measured, an extension in a captured graph: 7
// sequences by 4 tokens 3.4 us, 2.6 of it the launch; 3,000 by 2 tokens 10.9 (sums 3.3,
// search and maps 5.0); 256 by 230 tokens 13.2 (sums 0.7, 1.4 MB written 5.2, search
// and maps 4.7).
//
// Layout.  One cluster of 1 or 8 CTAs.  Every CTA makes the running sums of all
// sequences, four to a thread and 4,096 at a time in shared memory, and the
// cluster's threads share out the tokens, four to a thread.  What the call reads
// and also changes (the count of free pages) is written behind a barrier of the
// cluster, so that no CTA sees it changed and the call needs neither a workspace
// nor a second launch.

#include "fp4idx_attn.cuh"
#include "fp4idx_step.h"

namespace fp4idx_impl {
namespace {

constexpr int kPage = FP4IDX_KV_BLOCK;
constexpr int kThreads = 1024;      // of a CTA; 256 for a small call
constexpr int kEach = 4;            // sequences of a thread
constexpr int kChunk = kThreads * kEach;
constexpr unsigned kClusterMax = 8;  // the largest portable cluster

struct ExtendArgs {
  const int32_t* cached;
  const int32_t* added;
  int32_t* table;
  int64_t tstride;
  int32_t pages;
  const int32_t* free_pages;
  int32_t* free_count;
  int64_t capacity;
  int32_t* q_starts;
  int32_t* context;
  int64_t* slots;
  int64_t* positions;
  int32_t* seq_ids;
  int32_t* row_lens;
  int32_t batch, T;
  int32_t vec;  // the token outputs are 16-byte aligned
  uint32_t* err;
};

struct ReleaseArgs {
  const int32_t* held;
  const int32_t* kept;
  int32_t* table;
  int64_t tstride;
  int32_t pages;
  int32_t* free_pages;
  int32_t* free_count;
  int64_t capacity;
  int32_t batch;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// a + b, at most `cap` (which leaves the sum of two such within 32 bits).
__device__ __forceinline__ uint32_t capped(uint32_t a, uint32_t b, uint32_t cap) {
  return min(a + b, cap);
}

// The sum of x over the threads before this one, capped; `total`, over all of the
// CTA.  `part` holds 32 words and may be used again after the next barrier of the
// CTA.
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t cap, uint32_t* part,
                                               uint32_t& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  uint32_t incl = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl = capped(incl, o, cap);
  }
  uint32_t before = __shfl_up_sync(kFull, incl, 1);
  if (lane == 0) before = 0;
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  uint32_t w = lane < warps ? part[lane] : 0u;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(kFull, w, d);
    if (lane >= d) w = capped(w, o, cap);
  }
  total = __shfl_sync(kFull, w, 31);
  const uint32_t base = __shfl_sync(kFull, w, (warp + 31) % 32);
  return capped(before, warp > 0 ? base : 0u, cap);
}

// The first of n ascending ends that is above x (there is one).
__device__ __forceinline__ int find(const uint32_t* ends, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (ends[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Four words from p (at, ..), zero from n on.
__device__ __forceinline__ void load4(const int32_t* p, int64_t at, int64_t n, int32_t (&v)[kEach]) {
#pragma unroll
  for (int j = 0; j < kEach; ++j) v[j] = at + j < n ? max(__ldg(p + at + j), 0) : 0;
}

__device__ __forceinline__ uint32_t pages_of(uint32_t tokens) {
  return tokens / kPage + (tokens % kPage != 0);
}

// The count of free pages as the calls take it.
__device__ __forceinline__ uint32_t count_of(const int32_t* free_count, int64_t capacity) {
  return (uint32_t)min((int64_t)max(*free_count, 0), capacity);
}

__global__ __launch_bounds__(kThreads) void extend_kernel(const ExtendArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ uint32_t part[3][32];
  const int tid = threadIdx.x, threads = blockDim.x, chunk = threads * kEach;
  uint32_t* const ends = smem;            // of a sequence's tokens, in the call
  uint32_t* const first = smem + chunk;   // position of its first new token; ~0: not served
  uint32_t* const taken = first + chunk;  // pages taken before it
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const uint32_t count = count_of(a.free_count, a.capacity);
  // sums stop where nothing fits any more
  const uint32_t T = a.T, token_cap = T + 1, page_cap = count + 1;
  uint32_t done = 0;   // tokens of the chunks before this one
  uint32_t asked = 0;  // pages that they asked for
  uint32_t used = 0;   // and that were taken
  uint32_t turn = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += chunk, ++turn) {
    const int64_t b = b0 + tid * kEach;
    int32_t old[kEach], add[kEach];
    load4(a.cached, b, a.batch, old);
    load4(a.added, b, a.batch, add);
    uint32_t own = 0, tokens, pages;
#pragma unroll
    for (int j = 0; j < kEach; ++j) own = capped(own, min((uint32_t)add[j], token_cap), token_cap);
    uint32_t at = capped(done, sum_before(own, token_cap, part[0], tokens), token_cap);
    // where each one's tokens start and end, and the pages it needs
    uint32_t start[kEach], end[kEach], need[kEach], asks = 0;
    bool fits[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      start[j] = at;
      at = end[j] = capped(at, min((uint32_t)add[j], token_cap), token_cap);
      const uint32_t want = pages_of((uint32_t)old[j] + (uint32_t)add[j]);
      fits[j] = want <= (uint32_t)a.pages && end[j] <= T;
      need[j] = fits[j] ? want - pages_of(old[j]) : 0;
      asks = capped(asks, min(need[j], page_cap), page_cap);
    }
    uint32_t upto = capped(asked, sum_before(asks, page_cap, part[1], pages), page_cap);
    uint32_t most = 0;
    bool full = false;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t before = upto;
      upto = capped(upto, min(need[j], page_cap), page_cap);
      const bool served = fits[j] && (need[j] == 0 || upto <= count);
      if (served && need[j] > 0) most = upto;
      end[j] = min(end[j], T);
      start[j] = min(start[j], T);
      need[j] = before;
      // (from here on the length after the call, and the first new token's position)
      add[j] = served ? old[j] + add[j] : old[j];
      old[j] = served ? old[j] : -1;
      if (b + j < a.batch) {
        full = full || !served;
        if (turn % ctas == rank) {
          if (a.q_starts) a.q_starts[b + j] = (int32_t)start[j];
          if (a.context) a.context[b + j] = add[j];
        }
      }
    }
    reinterpret_cast<uint4*>(ends)[tid] = make_uint4(end[0], end[1], end[2], end[3]);
    reinterpret_cast<int4*>(first)[tid] = make_int4(old[0], old[1], old[2], old[3]);
    reinterpret_cast<uint4*>(taken)[tid] = make_uint4(need[0], need[1], need[2], need[3]);
    if (full && turn % ctas == rank) flag_error(a.err, FP4IDX_ERRFLAG_FULL);
    most = __reduce_max_sync(kFull, most);
    if (tid % 32 == 0) part[2][tid / 32] = most;
    __syncthreads();
    for (int w = 0; w < threads / 32; ++w) used = max(used, part[2][w]);
    // ---- the chunk's tokens, four to a thread
    const int n = (int)min((int64_t)chunk, a.batch - b0);
    const uint32_t t0 = min(done, T);
    done = capped(done, tokens, token_cap);
    asked = capped(asked, pages, page_cap);
    const uint32_t t1 = min(done, T);
    for (uint32_t g = t0 / 4 + rank * threads + tid; g < (t1 + 3) / 4; g += ctas * threads) {
      const uint32_t t = g * 4;
      int s = find(ends, n, max(t, t0));
      const bool whole = a.vec && t >= t0 && t + 3 < t1;
      {  // four tokens of one page, as most are in a prompt
        const uint32_t f = first[s], p = f + (t - (s > 0 ? ends[s - 1] : t0));
        if (whole && ends[s] > t + 3 && f != ~0u && p % kPage <= kPage - 4) {
          const uint32_t idx = p / kPage, held = pages_of(f);
          int32_t* const place = a.table + (b0 + s) * a.tstride + idx;
          const int32_t page =
              idx < held ? *place : a.free_pages[count - 1 - (taken[s] + (idx - held))];
          if (idx >= held && p % kPage == 0) *place = page;
          const int64_t slot = (int64_t)page * kPage + p % kPage;
          const int32_t id = (int32_t)b0 + s;
          if (a.slots) {
            reinterpret_cast<longlong2*>(a.slots + t)[0] = make_longlong2(slot, slot + 1);
            reinterpret_cast<longlong2*>(a.slots + t)[1] = make_longlong2(slot + 2, slot + 3);
          }
          if (a.positions) {
            reinterpret_cast<longlong2*>(a.positions + t)[0] = make_longlong2(p, p + 1);
            reinterpret_cast<longlong2*>(a.positions + t)[1] = make_longlong2(p + 2, p + 3);
          }
          if (a.seq_ids) *reinterpret_cast<int4*>(a.seq_ids + t) = make_int4(id, id, id, id);
          if (a.row_lens)
            *reinterpret_cast<int4*>(a.row_lens + t) = make_int4(p + 1, p + 2, p + 3, p + 4);
          continue;
        }
      }
      int32_t seq[4], pos[4];  // pos -1: nothing
      const int32_t* from[4];  // its page's number
      int32_t* entry[4];       // its place in the table, if it is new and begins here
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = t + j;
        pos[j] = -1;
        seq[j] = 0;
        from[j] = nullptr;
        entry[j] = nullptr;
        if (x < t0 || x >= t1) continue;
        if (ends[s] <= x && ends[++s] <= x) s = find(ends, n, x);
        seq[j] = (int32_t)b0 + s;
        const uint32_t f = first[s];
        if (f == ~0u) continue;
        const uint32_t p = f + (x - (s > 0 ? ends[s - 1] : t0));
        const uint32_t idx = p / kPage, held = pages_of(f);
        pos[j] = (int32_t)p;
        int32_t* const place = a.table + (b0 + s) * a.tstride + idx;
        from[j] = idx < held ? place : a.free_pages + (count - 1 - (taken[s] + (idx - held)));
        if (idx >= held && p % kPage == 0) entry[j] = place;
      }
      int32_t page[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        page[j] = !from[j] ? 0 : j > 0 && from[j] == from[j - 1] ? page[j - 1] : *from[j];
      int64_t slot[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        slot[j] = pos[j] < 0 ? -1 : (int64_t)page[j] * kPage + pos[j] % kPage;
        if (entry[j]) *entry[j] = page[j];
      }
      if (whole) {
        if (a.slots) {
          reinterpret_cast<longlong2*>(a.slots + t)[0] = make_longlong2(slot[0], slot[1]);
          reinterpret_cast<longlong2*>(a.slots + t)[1] = make_longlong2(slot[2], slot[3]);
        }
        if (a.positions) {
          reinterpret_cast<longlong2*>(a.positions + t)[0] =
              make_longlong2(max(pos[0], 0), max(pos[1], 0));
          reinterpret_cast<longlong2*>(a.positions + t)[1] =
              make_longlong2(max(pos[2], 0), max(pos[3], 0));
        }
        if (a.seq_ids)
          *reinterpret_cast<int4*>(a.seq_ids + t) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        if (a.row_lens)
          *reinterpret_cast<int4*>(a.row_lens + t) =
              make_int4(pos[0] + 1, pos[1] + 1, pos[2] + 1, pos[3] + 1);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (t + j < t0 || t + j >= t1) continue;
          if (a.slots) a.slots[t + j] = slot[j];
          if (a.positions) a.positions[t + j] = max(pos[j], 0);
          if (a.seq_ids) a.seq_ids[t + j] = seq[j];
          if (a.row_lens) a.row_lens[t + j] = pos[j] + 1;
        }
      }
    }
    __syncthreads();
  }
  // ---- the tokens behind the last one
  const uint32_t end = min(done, T);
  for (uint32_t t = end + rank * threads + tid; t < T; t += ctas * threads) {
    if (a.slots) a.slots[t] = -1;
    if (a.positions) a.positions[t] = 0;
    if (a.seq_ids) a.seq_ids[t] = 0;
    if (a.row_lens) a.row_lens[t] = 0;
  }
  cluster_sync();  // every CTA has read the count
  if (rank == 0 && tid == 0) {
    if (a.q_starts) a.q_starts[a.batch] = (int32_t)end;
    *a.free_count = (int32_t)(count - used);
  }
}

__global__ __launch_bounds__(kThreads) void release_kernel(const ReleaseArgs a) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t part[2][32];
  const int tid = threadIdx.x, threads = blockDim.x, chunk = threads * kEach;
  uint32_t* const upto = smem;          // pages given back up to a sequence of the chunk
  uint32_t* const keep = smem + chunk;  // pages that it keeps
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const uint32_t count = count_of(a.free_count, a.capacity);
  // (a batch's pages of a chunk stay below 2^31; sums of several stop there)
  constexpr uint32_t kCap = 0x7fffffffu;
  const auto gone = [&](int64_t b, uint32_t (&k)[kEach], uint32_t (&n)[kEach]) {
    int32_t held[kEach], kept[kEach];
    load4(a.held, b, a.batch, held);
    load4(a.kept, b, a.batch, kept);
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      k[j] = pages_of(min(kept[j], held[j]));
      const uint32_t has = min(pages_of(held[j]), (uint32_t)a.pages);
      n[j] = has > k[j] ? has - k[j] : 0;
      sum = capped(sum, n[j], kCap);
    }
    return sum;
  };
  // the first page goes on top, so their number is needed first
  uint32_t k[kEach], n[kEach], all = 0, done = 0;
  if (a.batch > chunk) {
    uint32_t own = 0;
    for (int64_t b = tid * kEach; b < a.batch; b += chunk) own = capped(own, gone(b, k, n), kCap);
    sum_before(own, kCap, part[1], all);
  }
  for (int64_t b0 = 0; b0 < a.batch; b0 += chunk) {
    const uint32_t own = gone(b0 + tid * kEach, k, n);
    uint32_t pages;
    uint32_t at = sum_before(own, kCap, part[0], pages);
    if (a.batch <= chunk) all = pages;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      at = capped(at, n[j], kCap);
      upto[tid * kEach + j] = at;
      keep[tid * kEach + j] = k[j];
    }
    __syncthreads();
    for (uint32_t i = rank * threads + tid; i < pages; i += ctas * threads) {
      const int s = find(upto, chunk, i);
      int32_t* const entry =
          a.table + (b0 + s) * a.tstride + keep[s] + (i - (s > 0 ? upto[s - 1] : 0));
      const int64_t to = (int64_t)count + all - 1 - done - i;
      if (to < a.capacity) a.free_pages[to] = *entry;
      *entry = -1;
    }
    done += pages;
    __syncthreads();
  }
  cluster_sync();  // every CTA has read the count
  if (rank == 0 && tid == 0) {
    const int64_t now = (int64_t)count + all;
    if (now > a.capacity) flag_error(a.err, FP4IDX_ERRFLAG_FULL);
    *a.free_count = (int32_t)min(now, a.capacity);
  }
}

// One small CTA where its threads are enough, a cluster of 8 large ones for `many`
// tokens or pages.
template <typename Args>
fp4idx_status launch_cluster(void (*kern)(Args), int64_t batch, int64_t elements, int words,
                             cudaStream_t stream, const Args& a) {
  // (a CTA's threads take 150 instructions for a token of its own: 4,096 tokens of
  // one sequence 9.2 us in one CTA)
  const bool many = elements > kThreads;
  const int threads = elements <= 8 * kThreads && batch <= 256 * kEach ? 256 : kThreads;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = many ? kClusterMax : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attr.val.clusterDim.x);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)threads * kEach * words * 4;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA;
}

bool pool_shape_ok(int64_t batch, int64_t stride, int64_t pages, int64_t capacity) {
  return batch < (1ll << 31) - 8192 && pages >= 0 && pages < (1ll << 25) &&
         (batch <= 1 || stride >= pages) && stride < (1ll << 40) && capacity >= 0 &&
         capacity < (1ll << 31) - 1;
}

}  // namespace
}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" fp4idx_status fp4idx_batch_extend(
    const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table,
    int64_t block_table_stride, int64_t block_table_pages, const int32_t* free_pages,
    int32_t* free_count, int64_t free_capacity, int32_t* q_starts, int32_t* context_lens,
    int64_t* slot_mapping, int64_t* positions, int32_t* seq_ids, int32_t* row_lens, int64_t batch,
    int64_t num_tokens, uint32_t* err_flags, void* stream) {
  if (batch < 0 || num_tokens < 0 || num_tokens >= (1ll << 31) - 4 ||
      !pool_shape_ok(batch, block_table_stride, block_table_pages, free_capacity))
    return FP4IDX_ERR_SHAPE;
  if (!free_count || (free_capacity > 0 && !free_pages) ||
      (batch > 0 && (!cached_lens || !new_lens || (block_table_pages > 0 && !block_table))))
    return FP4IDX_ERR_NULL;
  for (const int32_t* out : {q_starts, context_lens})
    if (out && (out == cached_lens || out == new_lens)) return FP4IDX_ERR_ARG;
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(q_starts, 4) ||
      !aligned(context_lens, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 8) ||
      !aligned(seq_ids, 4) || !aligned(row_lens, 4) || !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  ExtendArgs a = {};
  a.cached = cached_lens;
  a.added = new_lens;
  a.table = block_table;
  a.tstride = block_table_stride;
  a.pages = (int32_t)block_table_pages;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.capacity = free_capacity;
  a.q_starts = q_starts;
  a.context = context_lens;
  a.slots = slot_mapping;
  a.positions = positions;
  a.seq_ids = seq_ids;
  a.row_lens = row_lens;
  a.batch = (int32_t)batch;
  a.T = (int32_t)num_tokens;
  a.vec = aligned(slot_mapping, 16) && aligned(positions, 16) && aligned(seq_ids, 16) &&
          aligned(row_lens, 16);
  a.err = err_flags;
  static SmemOnce once;  // (48 KB beside the static words)
  if (!once.set(extend_kernel, kChunk * 3 * 4)) return FP4IDX_ERR_CUDA;
  return launch_cluster(extend_kernel, batch, num_tokens, 3, static_cast<cudaStream_t>(stream), a);
}

extern "C" fp4idx_status fp4idx_pages_release(const int32_t* held_lens, const int32_t* kept_lens,
                                              int32_t* block_table, int64_t block_table_stride,
                                              int64_t block_table_pages, int32_t* free_pages,
                                              int32_t* free_count, int64_t free_capacity,
                                              int64_t batch, uint32_t* err_flags, void* stream) {
  if (batch < 0 || !pool_shape_ok(batch, block_table_stride, block_table_pages, free_capacity))
    return FP4IDX_ERR_SHAPE;
  if (batch == 0) return FP4IDX_OK;
  if (!held_lens || !kept_lens || (block_table_pages > 0 && !block_table) ||
      (free_capacity > 0 && !free_pages) || !free_count)
    return FP4IDX_ERR_NULL;
  if (!aligned(held_lens, 4) || !aligned(kept_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  ReleaseArgs a = {};
  a.held = held_lens;
  a.kept = kept_lens;
  a.table = block_table;
  a.tstride = block_table_stride;
  a.pages = (int32_t)block_table_pages;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.capacity = free_capacity;
  a.batch = (int32_t)batch;
  a.err = err_flags;
  // (a page or two of each sequence, or all of a few)
  return launch_cluster(release_kernel, batch, batch * block_table_pages / 4, 2,
                        static_cast<cudaStream_t>(stream), a);
}
