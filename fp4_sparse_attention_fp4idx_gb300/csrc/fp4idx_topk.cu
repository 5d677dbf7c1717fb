// fp4idx_topk.cu -- the selection of the k largest logits of each row
// (fp4idx_topk_tokens, defined in include/fp4idx_attention.h): the step
// between the index scorer's logits and attention over the selected tokens.
//
// A logit becomes an unsigned key that orders like the float (0 for what can
// never be selected).  One CTA per row, bound by reading the row once:
//   1. 2,048 samples of the row give a threshold that about k + 4 sigma of
//      its entries reach;
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

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 12;                      // candidates a thread holds
constexpr int kCap = kThreads * kPer;         // 6144 candidates
constexpr int kSamples = 4 * kThreads;
constexpr int kBins = 2048;                   // 11 bits
constexpr int kMaxMapCols = 1 << 18;          // two bit maps of 32 KB

struct TopkArgs {
  const float* logits;
  int64_t stride;
  const int32_t* lens;
  int32_t* indices;
  int64_t istride;
  int32_t* counts;
  int32_t cols, k;
  int32_t map_words;  // words of a bit map; 0: columns beyond kMaxMapCols
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
  uint32_t bins[kBins];
  uint32_t part[kWarps];
  uint32_t part2[kWarps];
  uint32_t found[4];
  uint32_t count;
};

// Exclusive prefix sum over the block, and the sum of all.
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
  uint32_t base = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += part[w];
    all += part[w];
  }
  __syncthreads();
  return base + incl - v;
}

// Narrows [lo, hi] to where the want-th largest key lies, by at most `passes`
// histograms; keys outside [lo, hi] do not count.  On return the keys > hi
// are all selected and `want` of those in [lo, hi] are; `in` is their number.
template <int N>
__device__ __forceinline__ void narrow(const uint32_t (&key)[N], uint32_t& lo, uint32_t& hi,
                                       uint32_t& want, uint32_t& in, int passes, Shared& sh) {
  const int tid = threadIdx.x;
  for (int p = 0; p < passes && lo < hi && in != want; ++p) {
    const int bits = 32 - __clz((int)(hi - lo));
    const int shift = bits > 11 ? bits - 11 : 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) sh.bins[tid + i * kThreads] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] >= lo && key[i] <= hi) atomicAdd(&sh.bins[(key[i] - lo) >> shift], 1u);
    __syncthreads();
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
    const uint32_t bin = sh.found[0];
    want -= sh.found[1];
    in = sh.found[2];
    lo += bin << shift;
    const uint32_t top = lo + ((1u << shift) - 1u);
    hi = top < hi && top >= lo ? top : hi;
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

__global__ __launch_bounds__(kThreads, 3) void topk_kernel(const TopkArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint32_t* const ckey = reinterpret_cast<uint32_t*>(smem);  // candidates
  uint32_t* const cidx = ckey + kCap;
  uint32_t* const map = cidx + kCap;  // selected places
  uint32_t* const tie = map + a.map_words;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t row = blockIdx.x;
  const float* x = a.logits + row * a.stride;
  int32_t* out = a.indices + row * a.istride;
  int n = a.lens ? a.lens[row] : a.cols;
  n = n < 0 ? 0 : n > a.cols ? a.cols : n;
  if (a.map_words == 0) return select_general(a, x, n, out, row, sh);
  const int words = (n + 31) / 32;
  for (int i = tid; i < words; i += kThreads) map[i] = tie[i] = 0;

  uint32_t key[kPer];
  uint32_t top = 0, low = 1, total;
  const bool direct = n <= kCap;
  if (direct) {  // every entry is a candidate, in place
    uint32_t valid = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThreads;
      key[i] = e < n ? key_of(__ldg(x + e)) : 0u;
      valid += key[i] != 0;
      top = max(top, key[i]);
    }
    valid = __reduce_add_sync(kFull, valid);
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) {
      sh.part[warp] = valid;
      sh.part2[warp] = top;
    }
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      total += sh.part[w];
      top = max(top, sh.part2[w]);
    }
    __syncthreads();
  } else {
    // ---- the threshold: the sample of rank k/n * samples + 4 sigma
    float thr = -INFINITY;
    {
      uint32_t s[4];
      uint32_t smin = kFull, smax = 0;
      const int64_t g = (int64_t)(tid / 2) * (n - 8) / (kThreads / 2 - 1) + (tid % 2) * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = key_of(__ldg(x + g + i));
        smax = max(smax, s[i]);
        smin = min(smin, s[i] ? s[i] : kFull);
      }
      smax = __reduce_max_sync(kFull, smax);
      smin = __reduce_min_sync(kFull, smin);
      if (lane == 0) {
        sh.part[warp] = smax;
        sh.part2[warp] = smin;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        smax = max(smax, sh.part[w]);
        smin = min(smin, sh.part2[w]);
      }
      if (tid == 0) sh.count = 0;
      __syncthreads();
      const float p = (float)a.k / (float)n;
      uint32_t want = (uint32_t)(p * kSamples + 4.0f * sqrtf(p * (1.0f - p) * kSamples)) + 4u;
      // more samples wanted than there are (k near n, or few that count): all
      if (p < 1.0f && want < kSamples && smax != 0) {
        uint32_t in = kFull;
        narrow(s, smin, smax, want, in, 2, sh);
        if (smin != 0) thr = float_of(smin);
      }
    }
    // ---- what reaches it, with its place
    const auto keep = [&](float v, int e) {
      const bool hit = v >= thr && v > -INFINITY;
      const uint32_t m = __ballot_sync(kFull, hit);
      if (m == 0) return;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&sh.count, (uint32_t)__popc(m));
      at = __shfl_sync(kFull, at, 0) + __popc(m & ((1u << lane) - 1u));
      if (hit && at < kCap) {
        ckey[at] = key_of(v);
        cidx[at] = (uint32_t)e;
      }
    };
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) / 4 % 4);
    const int nv = (n - head) / 4;
    const float4* xv = reinterpret_cast<const float4*>(x + head);
    constexpr int kLoads = 4;
    for (int base = 0; base < nv; base += kThreads * kLoads) {
      float4 v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int e = base + i * kThreads + tid;
        v[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < nv) v[i] = __ldg(xv + e);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int e = head + (base + i * kThreads + tid) * 4;
        const bool h0 = v[i].x >= thr && v[i].x > -INFINITY;
        const bool h1 = v[i].y >= thr && v[i].y > -INFINITY;
        const bool h2 = v[i].z >= thr && v[i].z > -INFINITY;
        const bool h3 = v[i].w >= thr && v[i].w > -INFINITY;
        const uint32_t m0 = __ballot_sync(kFull, h0), m1 = __ballot_sync(kFull, h1);
        const uint32_t m2 = __ballot_sync(kFull, h2), m3 = __ballot_sync(kFull, h3);
        const uint32_t c0 = __popc(m0), c1 = __popc(m1), c2 = __popc(m2), c3 = __popc(m3);
        const uint32_t c = c0 + c1 + c2 + c3;
        if (c == 0) continue;
        uint32_t at = 0;
        if (lane == 0) at = atomicAdd(&sh.count, c);
        at = __shfl_sync(kFull, at, 0);
        const uint32_t below = (1u << lane) - 1u;
        const auto put = [&](bool h, uint32_t m, uint32_t first, float f, int place) {
          const uint32_t slot = first + __popc(m & below);
          if (h && slot < kCap) {
            ckey[slot] = key_of(f);
            cidx[slot] = (uint32_t)place;
          }
        };
        put(h0, m0, at, v[i].x, e);
        put(h1, m1, at + c0, v[i].y, e + 1);
        put(h2, m2, at + c0 + c1, v[i].z, e + 2);
        put(h3, m3, at + c0 + c1 + c2, v[i].w, e + 3);
      }
    }
    if (warp == 0) {  // the row's ends, not on 16-byte words: at most 3 + 3
      const int rest = head + nv * 4;
      const int e = lane < head ? lane : rest + lane - head;
      const bool on = lane < head || (lane >= head && e < n);
      keep(on ? __ldg(x + e) : -INFINITY, e);
    }
    __syncthreads();
    total = sh.count;
    // below k: the threshold was too high, unless it was none at all
    if (total > kCap || (total < (uint32_t)a.k && thr != -INFINITY))
      return select_general(a, x, n, out, row, sh);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t e = tid + i * kThreads;
      key[i] = e < total ? ckey[e] : 0u;
      top = max(top, key[i]);
    }
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) sh.part[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, sh.part[w]);
    __syncthreads();
    if (thr != -INFINITY) low = key_of(thr);
  }

  // ---- the k-th largest: keys above `hi` are selected, and `want` of those
  // in [low, hi]
  uint32_t want = (uint32_t)a.k, in = total, hi = top;
  const bool all = total <= (uint32_t)a.k;
  if (!all) narrow(key, low, hi, want, in, 4, sh);
  const bool limited = !all && in != want;  // then low == hi: equal keys
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (key[i] == 0 || (!all && key[i] < low)) continue;
    const uint32_t e = direct ? tid + i * kThreads : cidx[tid + i * kThreads];
    uint32_t* const m = limited && key[i] <= hi ? tie : map;
    atomicOr(m + e / 32, 1u << (e % 32));
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
                (int32_t)num_cols, (int32_t)k, 0};
  size_t bytes = 0;
  if (num_cols <= kMaxMapCols) {
    a.map_words = (int32_t)((num_cols + 31) / 32);
    if (a.map_words == 0) a.map_words = 1;
    bytes = 2 * (kCap + (size_t)a.map_words) * 4;
    static SmemOnce once;
    if (!once.set(topk_kernel, 2 * (kCap + kMaxMapCols / 32) * 4)) return FP4IDX_ERR_CUDA;
  }
  return launch_kernel(topk_kernel, (unsigned)num_rows, kThreads, bytes,
                       static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}
