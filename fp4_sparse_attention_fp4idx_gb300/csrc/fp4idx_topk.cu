// fp4idx_topk.cu -- the selection of the k largest logits of each row
// (fp4idx_topk_tokens, defined in include/fp4idx_attention.h): the step
// between the index scorer's logits and attention over the selected tokens.
//
// A logit becomes an unsigned key that orders like the float (0 for what can
// never be selected).  One CTA per row, bound by reading the row once:
//   1. 2,048 samples of the row (4,096 beyond 65,536 entries) give a threshold
//      that about k + 4 sigma of its entries reach; where no more samples than
//      that can be selected at all (a row mostly of -inf, as the scorer leaves
//      those of a prompt's first tokens), every entry that can be reaches it;
//   2. one pass over the row keeps the entries that reach it (a few
//      thousand) with their places, in shared memory;
//   3. the k-th largest of those is found exactly, 11 bits of the remaining
//      range at a time, by histograms in shared memory;
//   4. the selected places become a bit map, which is read out in order: the
//      result is ascending and does not depend on the order of step 2.
// Equal keys at the border are taken from a bit map of their own, lowest
// first.  Whatever the samples say, the result is exact: if fewer than k or
// more entries than fit reach the threshold (rows with many equal logits, or
// laid out against the samples), the row is selected by the general method,
// four histogram passes of 8 bits over the row and an ordered one.
//
// The steps but the second are chains of short phases between barriers, so
// what counts is how many rows an SM works on at once: the candidates stay in
// shared memory rather than in registers, four CTAs of 512 threads to an SM.
// Few long rows are given a cluster of eight CTAs each: all of them find the
// threshold, each filters an eighth of the row, and the first one's shared
// memory collects the candidates.  Measured: 512 rows of up to 65,536, k =
// 2,048, in 34 us with the logits in L2, 44 from HBM (13 for the bytes), 2 rows of
// 100,003, k = 1,024, in 12 (a CTA each 25).  Rows of more than 262,144 columns,
// for which the bit map has no room, always take the general method, 2.9 us per
// 1,000 entries and CTA: 878 us for a row of 300,007, 2,910 for 1,000,000.

#include <float.h>

#include <algorithm>

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;           // 11 bits
constexpr int kMaxMapCols = 1 << 18;  // a bit map of 32 KB
constexpr int kCluster = 8;

// Samples of a row of n entries.
__host__ __device__ constexpr int samples_of(int n) { return (n > 65536 ? 8 : 4) * kThreads; }

// Candidates that fit.  A sample stands for r entries, and the sampled rank is
// w = k / r + 4 sqrt(k / r) + 4, so about w r entries reach the threshold, 1.6 k at
// k = 2048 of 65,536.  More than C do if fewer than w samples lie among the C
// largest, of which C / r are expected with a deviation of sqrt(C / r): C is
// taken where w is four deviations below, since a row with more takes the
// general method, 7 to 40 times as long.  (9/4 k alone is up to two deviations
// from k = 1025 on: 512 rows of 65,536 took 248 us at k = 1100, 35 at 1024; 64 of
// 262,144 took 785 at k = 2048, now 35.)
constexpr int kMaxCap = 9600;
int cap_of(int k, int cols) {
  int r = (cols + samples_of(cols) - 1) / samples_of(cols);
  if (cols > 65536 && r < 32) r = 32;  // a row may be shorter
  const double w = (double)k / r + 4 * sqrt((double)k / r) + 4;
  const int most = (int)(r * (w + 8 + 4 * sqrt(w + 4)));
  return std::min(kMaxCap, std::max(most, std::max(3200, k * 9 / 4)));
}

struct TopkArgs {
  const float* logits;
  int64_t stride;
  const int32_t* lens;
  int32_t* indices;
  int64_t istride;
  int32_t* counts;
  int32_t cols, k;
  int32_t map_words;  // words of the bit map; 0: columns beyond kMaxMapCols
  int32_t cap;        // candidates that fit
};

// Orders like x; 0 for -inf and NaN; -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float float_of(uint32_t key) {  // key != 0
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

struct Shared {
  uint32_t bins[kBins];  // histograms; afterwards the bit map of equal keys
  uint32_t part[kWarps + 1];
  uint32_t part2[kWarps];
  uint32_t found[4];
  uint32_t lo, hi;   // least and largest key
  uint32_t live;     // samples that can be selected
  uint32_t few[32];  // the keys of a bin of few
  uint32_t count;
};

// Exclusive prefix sum over the block, and the sum of all.  (Every instruction
// that all threads execute costs an SM with four CTAs 16 cycles, so the first
// warp alone sums over the warps.)
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t& all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const uint32_t own = lane < kWarps ? part[lane] : 0u;
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < kWarps; d *= 2) {
      const uint32_t o = __shfl_up_sync(kFull, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane < kWarps) part[lane] = sum - own;
    if (lane == kWarps - 1) part[kWarps] = sum;
  }
  __syncthreads();
  all = part[kWarps];
  return part[warp] + incl - v;
}

// Of the bins' counts, which sum to `want` at least: the bin that holds the
// want-th largest (found[0]), the number above it (found[1]) and in it
// (found[2]).
__device__ __forceinline__ void find_bin(uint32_t want, Shared& sh) {
  const int tid = threadIdx.x;
  // thread t sums the bins from the top: 4t .. 4t + 3 counted downwards
  constexpr int kEach = kBins / kThreads;
  uint32_t c[kEach], own = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    c[i] = sh.bins[kBins - 1 - (tid * kEach + i)];
    own += c[i];
  }
  uint32_t all;
  uint32_t above = block_scan(own, sh.part, all);
  if (above < want && above + own >= want) {
    int i = 0;
#pragma unroll
    for (; i < kEach - 1; ++i) {
      if (above + c[i] >= want) break;
      above += c[i];
    }
    uint32_t n = c[0];
#pragma unroll
    for (int j = 1; j < kEach; ++j) n = i == j ? c[j] : n;
    sh.found[0] = (uint32_t)(kBins - 1 - (tid * kEach + i));
    sh.found[1] = above;
    sh.found[2] = n;
  }
  __syncthreads();
}

// Narrows [lo, hi] to where the want-th largest key lies, by at most `passes`
// histograms; keys outside [lo, hi] do not count, and `want` at least lie
// within.  On return the keys > hi
// are all selected and `want` of those in [lo, hi] are; `in` is their number.
// each(f): calls f for each of the thread's keys.
template <typename Each>
__device__ __forceinline__ void narrow(const Each& each, uint32_t& lo, uint32_t& hi,
                                       uint32_t& want, uint32_t& in, int passes, Shared& sh) {
  const int tid = threadIdx.x;
  for (int p = 0; p < passes && lo < hi && in != want; ++p) {
    const int bits = 32 - __clz((int)(hi - lo));
    const int shift = bits > 11 ? bits - 11 : 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) sh.bins[tid + i * kThreads] = 0;
    __syncthreads();
    each([&](uint32_t key) {
      if (key >= lo && key <= hi) atomicAdd(&sh.bins[(key - lo) >> shift], 1u);
    });
    __syncthreads();
    find_bin(want, sh);
    const uint32_t bin = sh.found[0];
    want -= sh.found[1];
    in = sh.found[2];
    lo += bin << shift;
    const uint32_t top = lo + ((1u << shift) - 1u);
    hi = top < hi && top >= lo ? top : hi;
    if (in <= 32 && in != want && lo < hi) {  // few: ranked by one warp
      if (tid == 0) sh.found[3] = 0;
      if (tid < 32) sh.few[tid] = 0;
      __syncthreads();
      each([&](uint32_t key) {
        if (key >= lo && key <= hi) sh.few[atomicAdd(&sh.found[3], 1u) % 32u] = key;
      });
      __syncthreads();
      if (tid < 32) {
        const uint32_t own = sh.few[tid];
        uint32_t above = 0, same = 0;
#pragma unroll 8
        for (int l = 0; l < 32; ++l) {
          const uint32_t o = __shfl_sync(kFull, own, l);
          above += o > own;
          same += o == own;
        }
        if (own != 0 && above < want && above + same >= want) {
          sh.found[0] = own;
          sh.found[1] = above;
          sh.found[2] = same;
        }
      }
      __syncthreads();
      lo = hi = sh.found[0];
      want -= sh.found[1];
      in = sh.found[2];
    }
    __syncthreads();
  }
}

// The general method: any row, any number of equal keys.
__device__ __noinline__ void select_general(const TopkArgs& a, const float* x, int n, int32_t* out,
                                            int64_t row, Shared& sh) {
  uint32_t* const hist = sh.bins;
  uint32_t* const found = sh.found;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  uint32_t prefix = 0, want = (uint32_t)a.k;  // `want` of the keys that share `prefix`
  bool all = false;  // fewer than k candidates: every one is selected
  for (int shift = 24; shift >= 0 && !all; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t key = key_of(__ldg(x + i));
      if (key != 0 && (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))))
        atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // lane l sums digits 8l .. 8l+7, from the top
      uint32_t own = 0;
      for (int j = 0; j < 8; ++j) own += hist[lane * 8 + j];
      uint32_t above = own;  // inclusive suffix sum
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_down_sync(kFull, above, d);
        if (lane + d < 32) above += o;
      }
      if (lane == 0) found[2] = above < want;  // the row has fewer candidates
      above -= own;
      if (above < want && above + own >= want) {
        int j = 7;
        for (; j > 0 && above + hist[lane * 8 + j] < want; --j) above += hist[lane * 8 + j];
        found[0] = (uint32_t)(lane * 8 + j);
        found[1] = above;
      }
    }
    __syncthreads();
    if (shift == 24 && found[2]) {
      all = true;
    } else {
      prefix |= found[0] << shift;
      want -= found[1];
    }
    __syncthreads();
  }
  // selected: key > prefix, or key == prefix and among the first `want` such
  if (all) {
    prefix = 0;
    want = 0;
  }
  uint32_t done = 0, ties = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const uint32_t key = i < n ? key_of(__ldg(x + i)) : 0u;
    const uint32_t meq = __ballot_sync(kFull, key == prefix && key != 0);
    const uint32_t mgt = __ballot_sync(kFull, key > prefix);
    if (lane == 0) {
      sh.part[warp] = __popc(mgt);
      sh.part2[warp] = __popc(meq);
    }
    __syncthreads();
    uint32_t gt = 0, eq = 0, gt_all = 0, eq_all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        gt += sh.part[w];
        eq += sh.part2[w];
      }
      gt_all += sh.part[w];
      eq_all += sh.part2[w];
    }
    const uint32_t below = (1u << lane) - 1u;
    gt += __popc(mgt & below);
    eq += ties + __popc(meq & below);
    const uint32_t before = eq < want ? eq : want;  // equal keys selected before this one
    const bool take = (mgt >> lane & 1u) || ((meq >> lane & 1u) && eq < want);
    const uint32_t eq_before_chunk = ties < want ? ties : want;
    if (take) out[done + gt + (before - eq_before_chunk)] = i;
    ties += eq_all;
    const uint32_t eq_now = ties < want ? ties : want;
    done += gt_all + (eq_now - eq_before_chunk);
    __syncthreads();
  }
  for (int i = (int)done + tid; i < a.k; i += kThreads) out[i] = -1;
  if (tid == 0 && a.counts) a.counts[row] = (int32_t)done;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The address of the first CTA's copy of a shared-memory word.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
  return a;
}

// Appends the places of the entries of x[from, from + n) that reach thr to a
// list of the CTA, *count of them so far.  What does not fit is counted only.
// A lane takes 16 entries at a time: a bit for each, one prefix sum over the
// warp, and a loop over the few that are set.
__device__ __forceinline__ void filter(const float* x, int from, int n, float thr,
                                       uint32_t* places, uint32_t* count, uint32_t cap) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  x += from;
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) / 4 % 4), n);
  const int nv = (n - head) / 4;
  const float4* xv = reinterpret_cast<const float4*>(x + head);
  const auto append = [&](uint32_t hits, const auto& place_of) {
    const uint32_t own = __popc(hits);
    uint32_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    uint32_t at = 0;
    if (lane == 31 && incl != 0) at = atomicAdd(count, incl);
    at = __shfl_sync(kFull, at, 31) + incl - own;
    for (; hits != 0; hits &= hits - 1, ++at)
      if (at < cap) places[at] = (uint32_t)place_of(__ffs((int)hits) - 1);
  };
  constexpr int kLoads = 4;
  for (int base = warp * 32 * kLoads; base < nv; base += kThreads * kLoads) {
    float4 w[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = base + i * 32 + lane;
      w[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < nv) w[i] = __ldg(xv + e);
    }
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (w[i].x >= thr) hits |= 1u << (4 * i);
      if (w[i].y >= thr) hits |= 2u << (4 * i);
      if (w[i].z >= thr) hits |= 4u << (4 * i);
      if (w[i].w >= thr) hits |= 8u << (4 * i);
    }
    const int first = from + head + (base + lane) * 4;
    append(hits, [&](int b) { return first + b / 4 * 128 + b % 4; });
  }
  if (warp == 0) {  // the ends that are not on 16-byte words: at most 3 + 3
    const int rest = head + nv * 4;
    const int e = lane < head ? lane : rest + lane - head;
    const bool hit = e < n && (lane < head || e >= rest) && __ldg(x + e) >= thr;
    append(hit, [&](int) { return from + e; });
  }
}

template <bool kClustered>
__global__ __launch_bounds__(kThreads, kClustered ? 1 : 4) void topk_kernel(const TopkArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint32_t* const ckey = reinterpret_cast<uint32_t*>(smem);  // candidates
  uint32_t* const cidx = ckey + a.cap;
  uint32_t* const map = cidx + a.cap;  // selected places
  const int tid = threadIdx.x, lane = tid % 32;
  const int64_t row = kClustered ? blockIdx.x / kCluster : blockIdx.x;
  const uint32_t rank = kClustered ? cluster_rank() : 0;
  const float* x = a.logits + row * a.stride;
  int32_t* out = a.indices + row * a.istride;
  int n = a.lens ? a.lens[row] : a.cols;
  n = n < 0 ? 0 : n > a.cols ? a.cols : n;
  if (!kClustered && a.map_words == 0) return select_general(a, x, n, out, row, sh);
  const int words = (n + 31) / 32;
  for (int i = tid; i < words; i += kThreads) map[i] = 0;
  if (tid == 0) sh.count = 0;

  float thr = -FLT_MAX;  // what reaches it can be selected: neither NaN nor -inf
  if (tid == 0) {
    sh.lo = kFull;
    sh.hi = 0;
    sh.live = 0;
  }
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) sh.bins[tid + i * kThreads] = 0;
  __syncthreads();
  if (n > a.cap) {
    // ---- the threshold: the sample of rank k/n * samples + 4 sigma.  Groups
    // of 8 neighbours, a lane four of them: a load that meets 32 lines holds
    // the L1 for as many cycles.
    const int samples = samples_of(n);
    const bool twice = samples > 4 * kThreads;
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) / 4 % 4);
    const float4* xv = reinterpret_cast<const float4*>(x + head);
    const int groups = (n - head) / 4 - 1;  // a group may begin at any of these words
    uint32_t s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 1 && !twice) break;
      const int g = i * (kThreads / 2) + tid / 2, of = samples / 8;
      const float4 w = __ldg(xv + (int)((int64_t)g * groups / of) + tid % 2);
      s[4 * i] = key_of(w.x);
      s[4 * i + 1] = key_of(w.y);
      s[4 * i + 2] = key_of(w.z);
      s[4 * i + 3] = key_of(w.w);
    }
    uint32_t smin = kFull, smax = 0, live = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      smax = max(smax, s[i]);
      smin = min(smin, s[i] ? s[i] : kFull);
      live += s[i] != 0;
    }
    smax = __reduce_max_sync(kFull, smax);
    smin = __reduce_min_sync(kFull, smin);
    live = __reduce_add_sync(kFull, live);
    if (lane == 0) {
      atomicMax(&sh.hi, smax);
      atomicMin(&sh.lo, smin);
      atomicAdd(&sh.live, live);
    }
    __syncthreads();
    smax = sh.hi;
    smin = sh.lo;
    const float p = (float)a.k / (float)n;
    uint32_t want = (uint32_t)(p * samples + 4.0f * sqrtf(p * (1.0f - p) * samples)) + 4u;
    if (want < sh.live) {  // else all: fewer samples can be selected than wanted
      uint32_t in = kFull;
      // by value, in equal steps: keys crowd into few bins, and lanes that
      // meet in a bin take turns
      const float lo = float_of(smin), step = (float_of(smax) - lo) * (1.0f / kBins);
      if (step > 0.0f && step < INFINITY) {
        const float inv = __frcp_rn(step);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (s[i])
            atomicAdd(&sh.bins[min((uint32_t)((float_of(s[i]) - lo) * inv), kBins - 1u)], 1u);
        __syncthreads();
        find_bin(want, sh);
        in = sh.found[2];
        thr = fmaf((float)sh.found[0], step, lo);  // near the bin's lower end: near is enough
        __syncthreads();
      }
      if (in > 64) {  // the values lie too far apart for equal steps
        narrow(
            [&](const auto& f) {
#pragma unroll
              for (int i = 0; i < 8; ++i) f(s[i]);
            },
            smin, smax, want, in, 2, sh);
        thr = float_of(smin);
      }
    }
  }
  __syncthreads();
  // ---- what reaches it, with its place
  if constexpr (kClustered) {
    const int slice = ((n + kCluster - 1) / kCluster + 3) / 4 * 4;
    const int from = min((int)rank * slice, n);
    filter(x, from, min(slice, n - from), thr, cidx, &sh.count, (uint32_t)a.cap);
    __syncthreads();
    const uint32_t own = sh.count;
    cluster_sync();  // every CTA has its count, and no other's is added to it yet
    if (rank != 0) {  // behind the first CTA's own
      if (tid == 0) {
        uint32_t at;
        asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                     : "=r"(at)
                     : "r"(in_first(&sh.count)), "r"(own)
                     : "memory");
        sh.found[0] = at;
      }
      __syncthreads();
      const uint32_t at = sh.found[0];
      const uint32_t i0 = in_first(cidx);
      for (uint32_t e = tid; e < min(own, (uint32_t)a.cap); e += kThreads)
        if (at + e < (uint32_t)a.cap)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(i0 + (at + e) * 4), "r"(cidx[e])
                       : "memory");
    }
    cluster_sync();  // the first CTA has them all
    if (rank != 0) return;
  } else {
    filter(x, 0, n, thr, cidx, &sh.count, (uint32_t)a.cap);
    __syncthreads();
  }
  const uint32_t total = sh.count;
  // below k: the threshold was too high, unless it was none at all
  if (total > (uint32_t)a.cap || (total < (uint32_t)a.k && thr != -FLT_MAX))
    return select_general(a, x, n, out, row, sh);

  // ---- the k-th largest: keys above `hi` are selected, and `want` of those
  // in [low, hi]
  uint32_t want = (uint32_t)a.k, in = total, low = 1, hi = 0;
  const bool all = total <= (uint32_t)a.k;
  if (!all) {
    low = key_of(thr);
    for (uint32_t e = tid; e < total; e += kThreads) {
      const uint32_t key = key_of(__ldg(x + cidx[e]));
      ckey[e] = key;
      hi = max(hi, key);
    }
    hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) atomicMax(&sh.hi, hi);
    __syncthreads();
    hi = sh.hi;
    narrow(
        [&](const auto& f) {
          for (uint32_t e = tid; e < total; e += kThreads) f(ckey[e]);
        },
        low, hi, want, in, 4, sh);
  }
  const bool limited = !all && in != want;  // then low == hi: equal keys
  // their bit map takes the histograms' place, where that is large enough
  uint32_t* const tie = a.map_words <= kBins ? sh.bins : map + a.map_words;
  if (limited) {
    for (int w = tid; w < words; w += kThreads) tie[w] = 0;
    __syncthreads();
  }
  for (uint32_t e = tid; e < total; e += kThreads) {
    if (!all && ckey[e] < low) continue;
    uint32_t* const m = limited && ckey[e] <= hi ? tie : map;
    atomicOr(m + cidx[e] / 32, 1u << (cidx[e] % 32));
  }
  __syncthreads();
  // ---- the bit map in order; thread t owns words [w0, w1)
  const int each = (words + kThreads - 1) / kThreads;
  const int w0 = min(tid * each, words), w1 = min(w0 + each, words);
  if (limited) {
    uint32_t own = 0, ignore;
    for (int w = w0; w < w1; ++w) own += __popc(tie[w]);
    uint32_t before = block_scan(own, sh.part, ignore);
    for (int w = w0; w < w1; ++w) {
      uint32_t m = tie[w], take = 0;
      for (; m != 0 && before < want; m &= m - 1, ++before) take |= m & (0u - m);
      map[w] |= take;
    }
  }
  uint32_t own = 0, count;
  for (int w = w0; w < w1; ++w) own += __popc(map[w]);
  uint32_t at = block_scan(own, sh.part, count);
  for (int w = w0; w < w1; ++w)
    for (uint32_t m = map[w]; m != 0; m &= m - 1) out[at++] = w * 32 + __ffs((int)m) - 1;
  for (int i = (int)count + tid; i < a.k; i += kThreads) out[i] = -1;
  if (tid == 0 && a.counts) a.counts[row] = (int32_t)count;
}

}  // namespace
}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" fp4idx_status fp4idx_topk_tokens(const float* logits, int64_t logits_stride,
                                            const int32_t* row_lens, int32_t* indices,
                                            int64_t indices_stride, int32_t* counts,
                                            int64_t num_rows, int64_t num_cols, int64_t k,
                                            void* stream) {
  if (num_rows < 0 || num_cols < 0) return FP4IDX_ERR_SHAPE;
  if (num_rows == 0) return FP4IDX_OK;
  if ((!logits && num_cols > 0) || !indices) return FP4IDX_ERR_NULL;
  if (num_rows >= (1ll << 31) || num_cols >= (1 << 30) || k < 1 || k > 4096 ||
      indices_stride < k || (num_rows > 1 && logits_stride < num_cols))
    return FP4IDX_ERR_SHAPE;
  if (!aligned(logits, 4) || !aligned(row_lens, 4) || !aligned(indices, 4) || !aligned(counts, 4))
    return FP4IDX_ERR_ALIGN;
  TopkArgs a = {logits, logits_stride, row_lens, indices, indices_stride, counts,
                (int32_t)num_cols, (int32_t)k, 0, 0};
  a.cap = cap_of(a.k, a.cols);
  size_t bytes = 0;
  bool clustered = false;
  if (num_cols <= kMaxMapCols) {
    a.map_words = (int32_t)((num_cols + 31) / 32);
    if (a.map_words == 0) a.map_words = 1;
    bytes = (2 * (size_t)a.cap + (a.map_words <= kBins ? 1 : 2) * a.map_words) * 4;
    constexpr int most = (2 * kMaxCap + 2 * kMaxMapCols / 32) * 4;
    static SmemOnce once, once_clustered;
    if (!once.set(topk_kernel<false>, most) || !once_clustered.set(topk_kernel<true>, most))
      return FP4IDX_ERR_CUDA;
    // a cluster per row where the rows leave most SMs idle and are long
    // enough for an eighth to be worth its own CTA
    clustered = num_rows * kCluster <= kMaxGrid && num_cols >= 16384;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clustered ? num_rows * kCluster : num_rows));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {kCluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = clustered ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, clustered ? topk_kernel<true> : topk_kernel<false>, a) ==
                 cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}
