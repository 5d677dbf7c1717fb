// fp4idx_kvcache.cu -- the 8-bit key/value cache: quantised as it is written
// (fp4idx_kv_store_fp8) and read back (fp4idx_kv_load_fp8).  The operations
// are defined in include/fp4idx_attention.h.
//
// Both are bound by memory: a store reads 2 bytes and writes 1 per element, a
// load the reverse.  A block's scale needs the maximum over its rows before
// the first code can be written, so a group of threads holds a whole run (at
// most 64 rows of one head) in registers: one read of the input, one
// reduction, one write.  Measured, 8 heads of 128: 40,007 tokens stored in 41
// us (88% of the copy bandwidth; without the early prefetch of the rows 45, then
// 512 threads a block 78, 8 blocks an SM 61), 256 appended in 6.8; 65,536 loaded in 66 us (90%; keys and values by threads
// of their own 70).

#include "fp4idx_attention_common.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kStoreThreads = 256;
constexpr int kPage = FP4IDX_KV_BLOCK;

struct StoreSide {  // keys or values
  const uint16_t* x;
  int64_t tstride, hstride;
  uint8_t* codes;
  float* scale;
};

struct StoreArgs {
  StoreSide k, v;
  int64_t num_blocks, code_stride, scale_stride;
  const int64_t* slots;
  int64_t T;
  uint32_t* err;
};

// One run of `len` rows (tokens t0 .., page rows off ..) of one head, by a
// group of kGroup threads (a warp, or the block).  A row takes D/8 lanes of
// 16 bytes each; kPasses passes hold kRows = kPasses * kGroup * 8 / D rows.
template <int D, bool kHalf, int kGroup, int kPasses>
__device__ __forceinline__ void store_run(const StoreArgs& a, const StoreSide& x, int head,
                                          int64_t t0, int64_t slot, int len, int tid, float* red) {
  constexpr int kLanes = D / 8;
  constexpr int kStep = kGroup / kLanes;  // rows per pass
  const int64_t page = slot / kPage;
  const int off = (int)(slot % kPage);
  const int r0 = tid / kLanes, c = tid % kLanes;
  const uint16_t* src = x.x + t0 * x.tstride + head * x.hstride + c * 8;
  uint4 w[kPasses];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kStep;
    w[i] = make_uint4(0, 0, 0, 0);
    if (r < len) w[i] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)r * x.tstride));
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16<kHalf>(u[j]);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  }
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  float* scale = x.scale + page * a.scale_stride + head;
  uint32_t before = 0;
  if (off > 0) before = __float_as_uint(__ldcg(scale)) >> 23 & 0xffu;
  if (kGroup > 32) {
    if (tid % 32 == 0) red[tid / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroup / 32; ++i) amax = fmaxf(amax, red[i]);
  } else {
    __syncwarp();
  }
  // every thread has read the old scale by here
  before = before > 254u ? 254u : before;
  uint32_t e = block_scale_exp(amax);
  if (off > 0 && before > e) e = before;
  if (tid == 0) __stcg(scale, __uint_as_float(e << 23));
  uint8_t* dst = x.codes + page * a.code_stride + (int64_t)head * kPage * D;
  const float inv = inv_scale(e);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kStep;
    if (r < len) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t out[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 f = unpack16<kHalf>(u[2 * j]), g = unpack16<kHalf>(u[2 * j + 1]);
        out[j] = e4m3x4(__fmul_rn(f.x, inv), __fmul_rn(f.y, inv), __fmul_rn(g.x, inv),
                        __fmul_rn(g.y, inv));
      }
      *reinterpret_cast<uint2*>(dst + (off + r) * D + c * 8) = make_uint2(out[0], out[1]);
    }
  }
  // the page's rows before the run, if its scale grew: code * old / new.  The
  // old scale may be as small as a biased exponent of 0 (an unwritten page).
  if (off > 0 && before < e) {
    const uint32_t d = e - before;
    const float shrink = d > 126u ? 0.0f : __uint_as_float((127u - d) << 23);
    constexpr int kOldLanes = D / 16;
    for (int r = tid / kOldLanes; r < off; r += kGroup / kOldLanes) {
      uint4* p = reinterpret_cast<uint4*>(dst + r * D + (tid % kOldLanes) * 16);
      uint4 o = *p;
      uint32_t* u = &o.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(u[j], lo, hi);
        const float2 f = unpack16<true>(lo), g = unpack16<true>(hi);
        u[j] = e4m3x4(__fmul_rn(f.x, shrink), __fmul_rn(f.y, shrink), __fmul_rn(g.x, shrink),
                      __fmul_rn(g.y, shrink));
      }
      *p = o;
    }
  }
}

// grid (ceil(T / chunk), kv_heads, keys / values).  A block owns the runs that
// begin among its chunk's tokens, wherever they end: at most 63 tokens behind
// the chunk, so the slots of chunk + 63 tokens decide.
template <int D, bool kHalf>
__global__ __launch_bounds__(kStoreThreads) void kv_store_kernel(StoreArgs a, int chunk) {
  __shared__ int64_t slots[2 * kPage];
  __shared__ uint32_t breaks[4];  // bit t: token t does not continue token t-1's run
  __shared__ uint32_t begins[2];  // bit t: a run begins at token t of the chunk
  __shared__ float red[kStoreThreads / 32];
  const int tid = threadIdx.x, warp = tid / 32;
  const int64_t base = (int64_t)blockIdx.x * chunk;
  const int head = blockIdx.y;
  const StoreSide side = blockIdx.z ? a.v : a.k;
  // the chunk's rows start on their way while the slots are looked at
  constexpr int kLines = D / 64;
  if (tid < chunk * kLines && base + tid / kLines < a.T)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(side.x + (base + tid / kLines) * side.tstride +
                                                  head * side.hstride + tid % kLines * 64));
  if (tid < 2 * kPage) {
    int64_t s = -1, prev = -1;
    if (base + tid < a.T) {
      s = __ldg(a.slots + base + tid);
      if (base + tid > 0) prev = __ldg(a.slots + base + tid - 1);
    }
    const int64_t limit = a.num_blocks * kPage;
    if (s >= limit) {
      if (tid < chunk && head == 0 && blockIdx.z == 0) flag_error(a.err, FP4IDX_ERRFLAG_SLOT);
      s = -1;
    }
    slots[tid] = s;
    // prev >= limit cannot be followed by a valid s = prev + 1
    const bool brk = s < 0 || s % kPage == 0 || prev < 0 || s != prev + 1;
    const uint32_t m = __ballot_sync(kFull, brk);
    const uint32_t b = __ballot_sync(kFull, brk && s >= 0 && tid < chunk);
    if (tid % 32 == 0) {
      breaks[warp] = m;
      if (warp < 2) begins[warp] = b;
    }
  }
  __syncthreads();
  const uint64_t starts = begins[0] | (uint64_t)begins[1] << 32;
  int n = 0;
  for (uint64_t left = starts; left != 0; left &= left - 1) {
    const int t = __ffsll((long long)left) - 1;
    // the next break behind t, at most 64 tokens on
    int end = t + 1;
    {
      const int w0 = end / 32;
      uint32_t m = breaks[w0] & (kFull << (end % 32));
      int w = w0;
      while (m == 0 && w < 3) m = breaks[++w];
      end = m != 0 ? w * 32 + __ffs((int)m) - 1 : 2 * kPage;
    }
    const int len = min(end - t, kPage);
    const int64_t slot = slots[t];
    if (len > 8) {  // the whole block
      store_run<D, kHalf, kStoreThreads, 64 * (D / 8) / kStoreThreads>(a, side, head, base + t,
                                                                       slot, len, tid, red);
      __syncthreads();  // red is used again
    } else {  // a short run: the next warp in turn
      if (n % (kStoreThreads / 32) == warp)
        store_run<D, kHalf, 32, 8 * (D / 8) / 32>(a, side, head, base + t, slot, len, tid % 32,
                                                  red);
      ++n;
    }
  }
}

struct LoadSide {
  const uint8_t* codes;
  const float* scale;
  uint16_t* out;
};

struct LoadArgs {
  LoadSide k, v;
  int64_t num_blocks, code_stride, scale_stride;
  const int64_t* slots;
  int64_t T;
  int32_t heads;
  uint32_t* err;
};

// A thread per 16 codes of a (token, head) row, keys and values: D/16 lanes a
// row, each code read as one 16-byte word and written as two.
template <int D, bool kHalf>
__global__ __launch_bounds__(256) void kv_load_kernel(LoadArgs a) {
  constexpr int kLanes = D / 16;
  const int64_t rows = a.T * a.heads;
  const int c = threadIdx.x % kLanes;
  for (int64_t r = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes; r < rows;
       r += (int64_t)gridDim.x * (256 / kLanes)) {
    const int64_t t = rows < (1ll << 32) ? (uint32_t)r / (uint32_t)a.heads : r / a.heads;
    const int h = (int)(r - t * a.heads);
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0) continue;
    if (slot >= a.num_blocks * kPage) {
      if (h == 0 && c == 0) flag_error(a.err, FP4IDX_ERRFLAG_SLOT);
      continue;
    }
    const int64_t page = slot / kPage;
    const int off = (int)(slot % kPage);
    const int64_t at = page * a.code_stride + ((int64_t)h * kPage + off) * D + c * 16;
    const int64_t sc = page * a.scale_stride + h;
    uint4 w[2];
    float s[2];
    w[0] = *reinterpret_cast<const uint4*>(a.k.codes + at);
    w[1] = *reinterpret_cast<const uint4*>(a.v.codes + at);
    s[0] = a.k.scale[sc];
    s[1] = a.v.scale[sc];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(u[j], lo, hi);
        const float2 f = unpack16<true>(lo), g = unpack16<true>(hi);
        o[2 * j] = pack16<kHalf>(__fmul_rn(f.x, s[e]), __fmul_rn(f.y, s[e]));
        o[2 * j + 1] = pack16<kHalf>(__fmul_rn(g.x, s[e]), __fmul_rn(g.y, s[e]));
      }
      uint4* dst = reinterpret_cast<uint4*>((e ? a.v.out : a.k.out) + r * D + c * 16);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <typename Args, typename... More>
cudaError_t launch3(void (*kern)(Args, More...), dim3 grid, unsigned block, void* stream,
                    const Args& a, More... more) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kern, a, more...);
}

}  // namespace
}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" fp4idx_status fp4idx_kv_store_fp8(
    const void* k, const void* v, int64_t k_token_stride, int64_t k_head_stride,
    int64_t v_token_stride, int64_t v_head_stride, int dtype, const int64_t* slot_mapping,
    const fp4idx_kv_cache* cache, int64_t num_tokens, uint32_t* err_flags, void* stream) {
  if (num_tokens < 0) return FP4IDX_ERR_SHAPE;
  if (num_tokens == 0) return FP4IDX_OK;
  const fp4idx_status cs = check_cache(cache);
  if (cs == FP4IDX_ERR_NULL || !k || !v || !slot_mapping) return FP4IDX_ERR_NULL;
  if (cs == FP4IDX_ERR_SHAPE || num_tokens >= (1ll << 31)) return FP4IDX_ERR_SHAPE;
  if (!dtype_ok(dtype)) return FP4IDX_ERR_ARG;
  if (cs != FP4IDX_OK || !aligned(k, 16) || !aligned(v, 16) || k_token_stride % 8 ||
      k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8 || !aligned(slot_mapping, 8) ||
      !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  StoreArgs a = {};
  a.k = {static_cast<const uint16_t*>(k), k_token_stride, k_head_stride, cache->k_codes,
         cache->k_scale};
  a.v = {static_cast<const uint16_t*>(v), v_token_stride, v_head_stride, cache->v_codes,
         cache->v_scale};
  a.num_blocks = cache->num_blocks;
  a.code_stride = cache->code_block_stride;
  a.scale_stride = cache->scale_block_stride;
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.err = err_flags;
  // Few tokens: 8 to a block, so that a decode batch (a run per token) fills
  // the GPU with one warp per run; many: 64, about one run of a prompt each.
  const int chunk = num_tokens * cache->kv_heads >= 64 * 512 ? 64 : 8;
  const dim3 grid((unsigned)((num_tokens + chunk - 1) / chunk), (unsigned)cache->kv_heads, 2);
  const bool half = dtype == FP4IDX_FP16;
  auto* kern = cache->head_dim == 128
                   ? (half ? kv_store_kernel<128, true> : kv_store_kernel<128, false>)
                   : (half ? kv_store_kernel<64, true> : kv_store_kernel<64, false>);
  return launch3(kern, grid, kStoreThreads, stream, a, chunk) == cudaSuccess ? FP4IDX_OK
                                                                            : FP4IDX_ERR_CUDA;
}

extern "C" fp4idx_status fp4idx_kv_load_fp8(const fp4idx_kv_cache* cache,
                                            const int64_t* slot_mapping, void* k_out, void* v_out,
                                            int dtype, int64_t num_tokens, uint32_t* err_flags,
                                            void* stream) {
  if (num_tokens < 0) return FP4IDX_ERR_SHAPE;
  if (num_tokens == 0) return FP4IDX_OK;
  const fp4idx_status cs = check_cache(cache);
  if (cs == FP4IDX_ERR_NULL || !slot_mapping || !k_out || !v_out) return FP4IDX_ERR_NULL;
  if (cs == FP4IDX_ERR_SHAPE || num_tokens >= (1ll << 31)) return FP4IDX_ERR_SHAPE;
  if (!dtype_ok(dtype)) return FP4IDX_ERR_ARG;
  if (cs != FP4IDX_OK || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slot_mapping, 8) ||
      !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  LoadArgs a = {};
  a.k = {cache->k_codes, cache->k_scale, static_cast<uint16_t*>(k_out)};
  a.v = {cache->v_codes, cache->v_scale, static_cast<uint16_t*>(v_out)};
  a.num_blocks = cache->num_blocks;
  a.code_stride = cache->code_block_stride;
  a.scale_stride = cache->scale_block_stride;
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.heads = cache->kv_heads;
  a.err = err_flags;
  const int rows_per_block = 256 * 16 / cache->head_dim;
  const int64_t want = (num_tokens * a.heads + rows_per_block - 1) / rows_per_block;
  const unsigned grid = (unsigned)(want < (1 << 30) ? want : (1 << 30));
  const bool half = dtype == FP4IDX_FP16;
  auto* kern = cache->head_dim == 128
                   ? (half ? kv_load_kernel<128, true> : kv_load_kernel<128, false>)
                   : (half ? kv_load_kernel<64, true> : kv_load_kernel<64, false>);
  return launch3(kern, dim3(grid), 256, stream, a) == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA;
}
