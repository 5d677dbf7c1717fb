// fp4idx_topk.cu -- the selection of the k largest logits of each row
// (fp4idx_topk_tokens, defined in include/fp4idx_attention.h): the step
// between the index scorer's logits and attention over the selected tokens.
//
// A logit becomes an unsigned key that orders like the float (0 for what can
// never be selected).  The k-th largest key is found digit by digit from the
// top, eight bits a pass: a histogram of the digit over the keys that share
// the digits found so far.  A last pass walks the row in order and writes the
// indices whose key is larger, and of the equal ones the first that are still
// wanted, so the result is ascending and ties go to the lowest index.

#include "fp4idx_attention_common.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct TopkArgs {
  const float* logits;
  int64_t stride;
  const int32_t* lens;
  int32_t* indices;
  int64_t istride;
  int32_t* counts;
  int32_t cols, k;
};

// Orders like x; 0 for -inf and NaN; -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ __launch_bounds__(kThreads) void topk_kernel(TopkArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[3];  // digit, keys above it, keys in it
  __shared__ uint32_t sums[2][kWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t row = blockIdx.x;
  const float* x = a.logits + row * a.stride;
  int n = a.lens ? a.lens[row] : a.cols;
  n = n < 0 ? 0 : n > a.cols ? a.cols : n;

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
  int32_t* out = a.indices + row * a.istride;
  uint32_t done = 0, ties = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const uint32_t key = i < n ? key_of(__ldg(x + i)) : 0u;
    const uint32_t meq = __ballot_sync(kFull, key == prefix && key != 0);
    const uint32_t mgt = __ballot_sync(kFull, key > prefix);
    if (lane == 0) {
      sums[0][warp] = __popc(mgt);
      sums[1][warp] = __popc(meq);
    }
    __syncthreads();
    uint32_t gt = 0, eq = 0, gt_all = 0, eq_all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        gt += sums[0][w];
        eq += sums[1][w];
      }
      gt_all += sums[0][w];
      eq_all += sums[1][w];
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
                (int32_t)num_cols, (int32_t)k};
  return launch_kernel(topk_kernel, (unsigned)num_rows, kThreads, 0,
                       static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}
