// fp4idx_attn.cuh -- what the entry points of the attention operators
// (fp4idx_attn.cu) and their kernels share.
#pragma once

#include <atomic>

#include "fp4idx_attention_common.cuh"

namespace fp4idx_impl {

constexpr int kMaxGrid = 152;  // persistent CTAs: one per SM

// The arguments of the attention kernels.  Dense: `batch` sequences.  Sparse:
// `batch` query tokens, each an item list of its own.
struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  int32_t half;  // fp16 elements (else bf16)
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  int64_t num_blocks, cstride, sstride;
  const int32_t* table;
  int64_t tstride;
  // dense
  const int32_t* ctx;
  const int32_t* starts;
  int32_t max_q, max_context, window, sinks;
  // sparse
  const int32_t* seq_ids;
  const int32_t* indices;
  int64_t idx_stride;
  int32_t nsel, table_pages, num_seqs, per_seq;

  int32_t batch, T, Hq, Hkv, G;
  int32_t R;       // query rows of an item
  int32_t rc_max;  // row chunks of a sequence, at most
  int32_t split;   // items may be cut at tiles (partial outputs in the workspace)
  int32_t withhold;  // testing: tile or stage of CTA 0 that is never ready (-1: none)
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_out;  // [slot][R][D] normalised partial outputs
  float* part_lse;  // [slot][R], log2
  // [kMaxGrid]: the item that begins in a CTA's share and ends in another's:
  // sequence, row chunk, key head, CTAs * 2 + the first one's slot (0: none)
  int4* cuts;
  uint32_t* err;
};

// Launches the kernel for few rows per item (fp4idx_attn_rows.cu).
fp4idx_status launch_rows(const AttnArgs& a, int head_dim, bool sparse, int grid,
                          cudaStream_t stream);

// Launches the kernel for many rows per item (fp4idx_attn_tiles.cu).
fp4idx_status launch_tiles(const AttnArgs& a, int head_dim, int grid, cudaStream_t stream);

// Raises a kernel's dynamic shared-memory limit, once per device.
class SmemOnce {
 public:
  template <typename Kernel>
  bool set(Kernel* kern, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done_.load(std::memory_order_acquire) >> dev & 1u) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
      return false;
    done_.fetch_or(1ull << dev, std::memory_order_release);
    return true;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// Whether `items` of `total` tiles, the longest of `most`, are cut where the
// CTAs' equal shares end, and joined, or each is one CTA's.  Cutting saves what
// the fullest CTA has more than the mean (a sequence's items follow one another
// and are as long).  It costs each CTA another item's start and end, the more
// the more rows, and the join.  Measured, cut against whole, us: 8 items of 32
// tiles 10.7 / 16.4, 240 of up to 32 tiles 37 / 30, of up to 94 tiles 65 / 70,
// 160 of up to 63 tiles 40 / 43; 80 of 32 rows and up to 32 tiles 62 / 39, 1024
// of 16 rows and up to 128 tiles 338 / 380.  Selected tokens cost twice as much
// a tile.
__host__ __device__ inline bool worth_cutting(int64_t items, int64_t total, int64_t most,
                                              int64_t rows, int64_t ctas, bool sparse) {
  const int64_t rounds = (items + ctas - 1) / ctas;
  const int64_t saved = rounds * ctas * most - total;  // tiles x CTAs
  return saved * (sparse ? 2 : 1) > (14 + rows) * rounds * ctas;
}

// Launches kern behind the stream's last kernel, allowed to start early: it
// waits for that kernel's results itself (griddepcontrol.wait).
template <typename Args>
inline cudaError_t launch_after(void (*kern)(Args), unsigned grid, unsigned block,
                                cudaStream_t stream, const Args& a) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace fp4idx_impl
