// fp4idx_batch.cu -- pages and maps of a step (fp4idx_batch_extend,
// fp4idx_pages_release, defined in include/fp4idx_step.h).
//
// What bounds it.  24 bytes written for each token (8 of page table and stack
// for each 64), 8 to 20 read and written for each sequence: for a decode step
// nothing but latency, so everything is one launch.  Both calls are a running
// sum over the sequences and then, for every token (every page), the search for
// its sequence in those sums.
//
// Layout.  One cluster of 1 or 8 CTAs.  Every CTA makes the running sums of all
// sequences, 1,024 at a time in shared memory, and the cluster's threads share
// out the tokens.  What the call reads and also changes (the count of free
// pages) is written behind a barrier of the cluster, so that no CTA sees it
// changed and the call needs neither a workspace nor a second launch.

#include "fp4idx_attn.cuh"
#include "fp4idx_step.h"

namespace fp4idx_impl {
namespace {

constexpr int kPage = FP4IDX_KV_BLOCK;
constexpr int kThreads = 1024;  // sequences summed at a time, one per thread
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
  int64_t batch, T;
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
  int64_t batch;
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

// The sum of x over this thread and those before it; `total`, over all of the
// CTA.  `part` holds a place per warp and may be used again after the next
// barrier of the CTA.
__device__ __forceinline__ int64_t running_sum(int64_t x, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += o;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int64_t w = part[lane];  // kThreads / 32 = 32 warps
  const int64_t own = w;
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(kFull, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(kFull, w, 31);
  return x + __shfl_sync(kFull, w - own, warp);
}

// The first of n ascending ends that is above x (there is one).
__device__ __forceinline__ int find(const int32_t* ends, int n, int32_t x) {
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

__global__ __launch_bounds__(kThreads) void extend_kernel(const ExtendArgs a) {
  __shared__ int64_t part[2][32];
  __shared__ int32_t ends[kThreads];   // of a sequence's tokens, from the chunk's first
  __shared__ int32_t first[kThreads];  // position of its first new token; -1: not served
  __shared__ int32_t taken[kThreads];  // pages taken before it
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int64_t count = min(max((int64_t)*a.free_count, (int64_t)0), a.capacity);
  int64_t done = 0;   // tokens of the chunks before this one
  int64_t asked = 0;  // pages that they asked for
  int64_t used = 0;   // and that were taken
  uint32_t turn = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kThreads, ++turn) {
    const int64_t b = b0 + tid;
    const bool real = b < a.batch;
    const int64_t old = real ? max(a.cached[b], 0) : 0;
    const int64_t add = real ? max(a.added[b], 0) : 0;
    const int64_t has = (old + kPage - 1) / kPage, want = (old + add + kPage - 1) / kPage;
    int64_t tokens, pages;
    const int64_t end = done + running_sum(add, part[0], tokens);
    const bool fits = want <= a.pages && end <= a.T;
    const int64_t need = fits ? want - has : 0;
    const int64_t upto = asked + running_sum(need, part[1], pages);
    const bool served = fits && (need == 0 || upto <= count);
    ends[tid] = (int32_t)(min(end, a.T) - min(done, a.T));
    first[tid] = served ? (int32_t)old : -1;
    taken[tid] = (int32_t)min(upto - need, (int64_t)INT32_MAX);
    if (real && turn % ctas == rank) {
      if (a.q_starts) a.q_starts[b] = (int32_t)min(end - add, a.T);
      if (a.context) a.context[b] = (int32_t)(served ? old + add : old);
      if (!served) flag_error(a.err, FP4IDX_ERRFLAG_FULL);
    }
    __syncthreads();
    // what was taken: up to the last sequence served
    int64_t most = served && need > 0 ? upto : 0;
    for (int d = 16; d > 0; d /= 2) most = max(most, __shfl_xor_sync(kFull, most, d));
    if (tid % 32 == 0) part[0][tid / 32] = most;
    // ---- the chunk's tokens, four to a thread
    const int n = (int)min((int64_t)kThreads, a.batch - b0);
    const int64_t t0 = min(done, a.T), t1 = min(done + tokens, a.T);
    for (int64_t g = t0 / 4 + rank * kThreads + tid; g * 4 < t1; g += ctas * kThreads) {
      int64_t slot[4], pos[4];
      int32_t seq[4], len[4];
      int s = -1;
      int64_t page = 0;
      int at = -1;  // the page's index in its sequence
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = g * 4 + j;
        slot[j] = -1;
        pos[j] = 0;
        seq[j] = len[j] = 0;
        if (t < t0 || t >= t1) continue;
        const int32_t x = (int32_t)(t - t0);
        if (s < 0 || ends[s] <= x) {
          s = find(ends, n, x);
          at = -1;
        }
        seq[j] = (int32_t)(b0 + s);
        const int32_t f = first[s];
        if (f < 0) continue;
        const int32_t p = f + (x - (s > 0 ? ends[s - 1] : 0));
        const int idx = p / kPage, held = (int)(((int64_t)f + kPage - 1) / kPage);
        if (idx != at) {
          at = idx;
          int32_t* entry = a.table + (b0 + s) * a.tstride + idx;
          if (idx < held) {
            page = *entry;
          } else {
            page = a.free_pages[count - 1 - (taken[s] + (idx - held))];
            if (p % kPage == 0) *entry = (int32_t)page;
          }
        }
        slot[j] = page * kPage + p % kPage;
        pos[j] = p;
        len[j] = p + 1;
      }
      const int64_t t = g * 4;
      if (a.vec && t >= t0 && t + 3 < t1) {
        if (a.slots) {
          reinterpret_cast<longlong2*>(a.slots + t)[0] = make_longlong2(slot[0], slot[1]);
          reinterpret_cast<longlong2*>(a.slots + t)[1] = make_longlong2(slot[2], slot[3]);
        }
        if (a.positions) {
          reinterpret_cast<longlong2*>(a.positions + t)[0] = make_longlong2(pos[0], pos[1]);
          reinterpret_cast<longlong2*>(a.positions + t)[1] = make_longlong2(pos[2], pos[3]);
        }
        if (a.seq_ids)
          *reinterpret_cast<int4*>(a.seq_ids + t) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        if (a.row_lens)
          *reinterpret_cast<int4*>(a.row_lens + t) = make_int4(len[0], len[1], len[2], len[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (t + j < t0 || t + j >= t1) continue;
          if (a.slots) a.slots[t + j] = slot[j];
          if (a.positions) a.positions[t + j] = pos[j];
          if (a.seq_ids) a.seq_ids[t + j] = seq[j];
          if (a.row_lens) a.row_lens[t + j] = len[j];
        }
      }
    }
    __syncthreads();
    for (int w = 0; w < 32; ++w) used = max(used, part[0][w]);
    done += tokens;
    asked += pages;
    __syncthreads();
  }
  // ---- the tokens behind the last one
  const int64_t end = min(done, a.T);
  for (int64_t t = end + rank * kThreads + tid; t < a.T; t += ctas * kThreads) {
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
  __shared__ int64_t part[2][32];
  __shared__ int64_t upto[kThreads];  // pages given back up to a sequence of the chunk
  __shared__ int32_t keep[kThreads];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int64_t count = min(max((int64_t)*a.free_count, (int64_t)0), a.capacity);
  // pages of sequence b that go, behind the k first
  const auto gone = [&](int64_t b, int64_t& k) -> int64_t {
    k = 0;
    if (b >= a.batch) return 0;
    const int64_t held = max(a.held[b], 0), kept = min((int64_t)max(a.kept[b], 0), held);
    k = (kept + kPage - 1) / kPage;
    return max(min((held + kPage - 1) / kPage, (int64_t)a.pages) - k, (int64_t)0);
  };
  // the first page goes on top, so their number is needed first
  int64_t k, own = 0, all;
  for (int64_t b = tid; b < a.batch; b += kThreads) own += gone(b, k);
  running_sum(own, part[1], all);
  int64_t done = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int64_t n = gone(b0 + tid, k);
    int64_t pages;
    upto[tid] = running_sum(n, part[0], pages);
    keep[tid] = (int32_t)k;
    __syncthreads();
    for (int64_t i = (int64_t)rank * kThreads + tid; i < pages; i += ctas * kThreads) {
      int lo = 0, hi = kThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (upto[mid] > i)
          hi = mid;
        else
          lo = mid + 1;
      }
      int32_t* entry =
          a.table + (b0 + lo) * a.tstride + keep[lo] + (i - (lo > 0 ? upto[lo - 1] : 0));
      const int64_t to = count + all - 1 - (done + i);
      if (to < a.capacity) a.free_pages[to] = *entry;
      *entry = -1;
    }
    done += pages;
    __syncthreads();
  }
  cluster_sync();  // every CTA has read the count
  if (rank == 0 && tid == 0) {
    if (count + all > a.capacity) flag_error(a.err, FP4IDX_ERRFLAG_FULL);
    *a.free_count = (int32_t)min(count + all, a.capacity);
  }
}

template <typename Args>
fp4idx_status launch_cluster(void (*kern)(Args), bool many, void* stream, const Args& a) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = many ? kClusterMax : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attr.val.clusterDim.x);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA;
}

bool pool_shape_ok(int64_t batch, int64_t stride, int64_t pages, int64_t capacity) {
  return batch < (1ll << 31) && pages >= 0 && pages < (1ll << 25) &&
         (batch <= 1 || stride >= pages) && stride < (1ll << 40) && capacity >= 0 &&
         capacity < (1ll << 31);
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
  if (batch < 0 || num_tokens < 0 || num_tokens >= (1ll << 31) ||
      !pool_shape_ok(batch, block_table_stride, block_table_pages, free_capacity))
    return FP4IDX_ERR_SHAPE;
  if (!free_count || (free_capacity > 0 && !free_pages) ||
      (batch > 0 && (!cached_lens || !new_lens || (block_table_pages > 0 && !block_table))))
    return FP4IDX_ERR_NULL;
  if (context_lens && context_lens == cached_lens) return FP4IDX_ERR_ARG;
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
  a.batch = batch;
  a.T = num_tokens;
  a.vec = aligned(slot_mapping, 16) && aligned(positions, 16) && aligned(seq_ids, 16) &&
          aligned(row_lens, 16);
  a.err = err_flags;
  return launch_cluster(extend_kernel, num_tokens > 4 * kThreads || batch > kThreads, stream, a);
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
  a.batch = batch;
  a.err = err_flags;
  return launch_cluster(release_kernel, batch * block_table_pages > 16 * kThreads, stream, a);
}
