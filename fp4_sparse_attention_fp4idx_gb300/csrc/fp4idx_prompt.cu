// fp4idx_prompt.cu -- attention of packed sequences over their own keys and
// values in 16 bits (fp4idx_prompt_attention, defined in include/fp4idx_step.h),
// on the tensor cores through tcgen05.mma kind::f16.
//
// What bounds it.  4 D operations per query row and key against 4 D bytes per
// key for a whole item of 256 rows: the tensor cores and, next to them, one
// exponential per score; for single tokens over long keys the keys' bytes.
// Measured: 8,192 tokens, 64 heads of 128 over 8 key heads, 660 to 670 us at 1.92 GHz,
// 1,640 to 1,660 TFLOP/s, tensor pipe busy 74%, and 712 us (1.83 GHz) call after call;
// 16,384 tokens 2,480 us (1.9 GHz) to 2,810 us (1.72 GHz) by how far the power limit
// holds the clock down, 1,560 to 1,770 TFLOP/s (a library product of large matrices
// 1,719 sustained, 1,930 in a burst).  A tile of 128 keys takes a CTA 2,570 cycles, its
// MMAs 2,048: each half's scores, softmax (1,430) and product follow one another.  32
// single tokens over up to 20,000 keys: 140 us, 5.97 TB/s, 88% of the copy rate.
//
// Mathematics.  With x = softmax_scale * log2(e) * q k a row keeps M, the
// reference of its sums, l = sum 2^(x - M) and O = sum 2^(x - M) v; out = O / l.
// M is kShift below an x that was the row's largest, and follows the largest only
// when that has grown by more than kSlack, so the sums in TMEM are seldom rescaled.
// Probabilities 2^(x - M) are rounded to the elements' type for the product with the
// values (the tensor core wants both operands of one type); l is summed from the
// unrounded ones.  bf16 has fp32's range: one may grow to 2^8, all are shifted down
// by 2^6, so that O is in range where sum 2^(x - top) |v| < 2^125, top the row's
// largest x, and that none above 2^-120 of the largest vanishes.  (A slack of 2^4,
// which needs less of a shift, takes up to 10% more time: 8,192 tokens, 32 heads of
// 128 over 8, scores of standard deviation 2, 344 -> 378 us.)  In fp16 they are shifted
// up by 2^10 and may grow by 2^4 more, and the smallest that does not vanish is 2^-35
// of the largest.
//
// Roles (one CTA per SM).  An item is 256 rows (token i, head g of a key head's
// group: row i * G + g) of a sequence, as two M = 128 halves A and B that share
// every key tile of 128 keys.
//   warp 0          issues the MMAs: S = Q K^T, then O += P V with P from TMEM
//                   and V as it lies in memory (the transposed operand form).
//                   While half A's softmax runs, half B's products do.
//   warp 1          walks the CTA's list of work, describes its segments and
//                   loads their key and value tiles by TMA, 128-byte swizzled,
//                   into a ring that keys and values share
//   warps 2, 3      queries of half A, of half B, into shared memory; and rows
//                   of a value tile that no query of the item sees are set to
//                   zero (a probability of 0 times what may lie there is NaN)
//   warps 4-7, 8-11 softmax of half A, of half B: a row per thread, its 128
//                   scores read from TMEM into registers, its probabilities
//                   written back over the first half of them, 64 keys handed to
//                   the issuer while the other 64 are made; and the outputs, which
//                   leave through shared memory by TMA.  (Two threads a row made a
//                   tile 7% slower: the exponentials take as long, and each tile
//                   has a barrier more.  A third score buffer in TMEM, which D =
//                   64 has room for, changed nothing.)
// TMEM: scores A and B at columns 0 and 128 (P over the first 64), O at 256 and
// 256 + D.
// The items and their tiles form one list, cut into equal shares, one per CTA,
// from the lengths alone; an item cut by a share's end leaves normalised
// partial outputs, joined by a second kernel in a fixed order.  Where no item has
// more than kWhole tiles, an item belongs to the share that holds its first tile
// instead, and there is no second kernel.
// Every wait is bounded (1 s) and a shared abort flag stops every role; copies
// and MMAs in flight are waited for before the CTA ends.

#include <cuda.h>

#include "fp4idx_attn.cuh"
#include "fp4idx_step.h"
#include "fp4idx_tc.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kTile = 128;  // keys of a tile
constexpr int kHalfRows = 128, kWarpRows = 32;
constexpr int kItemRows = 2 * kHalfRows;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kSideWarp = 2, kSoftWarp = 4;
constexpr int kThreads = 12 * 32;
constexpr int kSegUsers = 11;  // warps that read a segment: the issuer, the sides, the softmax
constexpr int kSegRing = 2;
constexpr int kCleanRing = 4;
// Registers of a thread, by warpgroup, within the launch's 168.
constexpr int kLaunchRegs = 168, kSoftRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * kLaunchRegs, "the launch's registers");
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t q_bytes(int D) { return kItemRows * D * 2; }
__host__ __device__ constexpr uint32_t kv_bytes(int D) { return kTile * D * 2; }
// Tiles of keys and values in shared memory.
__host__ __device__ constexpr int ring_of(int D) { return D == 128 ? 4 : 8; }
// A value tile's clean barrier is used again 4 tiles on, its own slot 4 at most.
static_assert(ring_of(64) <= 2 * kCleanRing && ring_of(128) <= 2 * kCleanRing, "clean ring");
// Keys and values take turns, so that values have the odd slots to themselves.
static_assert(ring_of(64) % 2 == 0 && ring_of(128) % 2 == 0, "a slot holds keys or values");
// Where a softmax warp turns its rows of 64 output elements.
constexpr uint32_t kStageBytes = 32 * 128;
__host__ __device__ constexpr uint32_t smem_bytes(int D) {
  return q_bytes(D) + ring_of(D) * kv_bytes(D) + 8 * kStageBytes + 1024;
}

struct PromptArgs {
  CUtensorMap kmap, vmap, qmap, omap;
  int32_t kx, kz, vx, vz;  // a head's step in the maps' first and last coordinate
  const uint16_t* q;
  int64_t q_ts, q_hs;
  int32_t q_tma;  // queries are loaded by TMA: whole tokens fill a half
  int32_t o_tma;  // outputs are stored by TMA: whole tokens fill a warp's rows
  const int32_t* q_starts;
  const int32_t* k_starts;
  int32_t max_q, max_k, window, sinks;
  int32_t batch, Tq, Tk, Hq, Hkv, G;
  FastDiv by_g;
  int32_t rc_max;    // row chunks of a sequence, at most
  int32_t whole;     // items are not cut
  int32_t withhold;  // testing: tile of CTA 0 that is never loaded (-1: none)
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_out;  // normalised partial outputs, by part_at
  float* part_lse;  // [slot][kItemRows], log2
  // [grid]: the item that begins in a CTA's share and ends in another's:
  // sequence, row chunk, key head, CTAs * 2 + the first one's slot (0: none)
  int4* cuts;
  uint32_t* err;
};

// One item: up to 256 consecutive rows of a sequence and key head.
struct Item {
  int row0, rows;
  int q0, k0;     // first query token and first key of the sequence
  int first;      // position of its first query token
  int lo, hi;     // keys that any row sees: [lo, hi) and [0, sinks)
  int ts, tl;     // tiles: 0 .. ts-1, then tl ..
  int nt;         // tiles in all, at least one
};

// The rows' chunk rc of sequence b; false: it has no rows, nor has any behind it.
__device__ __forceinline__ bool item_of(const PromptArgs& a, int b, int rc, Item& m) {
  m.q0 = min(max(__ldg(a.q_starts + b), 0), a.Tq);
  const int n = min(max(__ldg(a.q_starts + b + 1), m.q0), a.Tq) - m.q0;
  m.k0 = min(max(__ldg(a.k_starts + b), 0), a.Tk);
  const int c = min(max(__ldg(a.k_starts + b + 1), m.k0), a.Tk) - m.k0;
  m.first = c - n;
  m.row0 = rc * kItemRows;
  m.rows = min(min(n, a.max_q) * a.G - m.row0, kItemRows);
  if (m.rows <= 0) return false;
  const int last = m.first + (int)a.by_g.div(m.row0 + m.rows - 1);
  m.hi = max(min(min(c, a.max_k), last + 1), 0);
  m.lo = a.window > 0
             ? min(max(m.first + (int)a.by_g.div(m.row0) - a.window + 1, 0), m.hi)
             : 0;
  m.tl = m.lo / kTile;
  m.ts = a.window > 0 ? min((a.sinks + kTile - 1) / kTile, m.tl) : 0;
  m.nt = max(m.ts + (m.hi + kTile - 1) / kTile - m.tl, 1);
  return true;
}

// The first key of the item's tile t.
__device__ __forceinline__ int key_of_tile(const Item& m, int t) {
  return (t < m.ts ? t : m.tl + (t - m.ts)) * kTile;
}

// What an item costs beside its tiles, in tiles: its first scores, its last product
// and its output wait for one another.  Measured (fitted to 1 to 4 items a CTA of 2 to
// 32 tiles) 5,400 cycles against 2,570 a tile for D = 128, 4,200 against 2,240 for D =
// 64.  Shares of equal tiles left the CTA with the shortest items 1.5 times the
// others' time.
constexpr int kStart = 2;
// Tiles up to which items are not cut.  Measured, cut against whole, us: items of up
// to 2 tiles, one prompt of 256 tokens (32 heads over 8) 17.3 / 13.4, forty 50 / 45;
// of 4, one of 500 19.0 / 15.8, sixty-four 138 / 133, 30 single tokens over 500 keys
// 22.0 / 19.7; of 8, one of 1,024 25.2 / 22.0, but 4 single tokens over 1,000 keys
// 16.5 / 23.4; of 16, one of 2,000 (8 heads over 1) 22.5 / 29.4.
constexpr int kWhole = 4;

// Where element d (a multiple of 4, and up to 3 more) of an item's row lies in
// partial output `place`: the rows of four elements together, so that a warp
// writes 512 bytes on end.
template <int D>
__device__ __forceinline__ int64_t part_at(int64_t place, int d, int row) {
  return ((place * (D / 4) + d / 4) * kItemRows + row) * 4 + d % 4;
}

// The list of work: for each sequence, row chunk and key head kStart units and
// the item's tiles, a unit each.  It is cut into equal shares, one per CTA.
struct Share {
  int64_t s0, s1, total;
  int b, rc, head;       // the item of unit s0
  int off, units;        // that unit in it; its units
  int grid;              // CTAs with a share
};

// A segment of the share: an item's tiles [t0, t1).
struct Seg {
  Item m;
  int head, t0, t1;
  int whole;  // the item as a whole
  int part;   // else the slot of its partial outputs
  int more;   // segments follow
};

// This CTA's share, by the whole CTA.
__device__ __forceinline__ void locate_share(const PromptArgs& a, Share& sh) {
  __shared__ int64_t part[kThreads / 32];
  __shared__ int count[kThreads / 32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t pairs = (int64_t)a.batch * a.rc_max;
  const int64_t each = (pairs + kThreads - 1) / kThreads;
  const int64_t p0 = min(tid * each, pairs), p1 = min(p0 + each, pairs);
  const int b0 = (int)(p0 / a.rc_max), rc0 = (int)(p0 - (int64_t)b0 * a.rc_max);
  int64_t own = 0;
  int items = 0;
  Item m;
  for (int64_t p = p0, b = b0, rc = rc0; p < p1;) {
    if (item_of(a, (int)b, (int)rc, m)) {
      own += m.nt + kStart;
      ++items;
      ++p;
      ++rc;
    } else {  // (a call may have thousands of sequences, few as long as the longest)
      p += a.rc_max - rc;
      rc = a.rc_max;
    }
    if (rc == a.rc_max) {
      rc = 0;
      ++b;
    }
  }
  own *= a.Hkv;
  int64_t incl = own;
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  items = __reduce_add_sync(kFull, items);
  if (lane == 31) {
    part[warp] = incl;
    count[warp] = items;
  }
  __syncthreads();
  int64_t base = 0, total = 0, n = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += part[w];
    total += part[w];
    n += count[w];
  }
  // shares of at least four tiles, but every item may have a CTA of its own
  const int64_t most = gridDim.x;
  const int64_t each_own = min(n * a.Hkv, most);
  const int64_t grid = a.whole ? each_own : max(min(total / 4, most), each_own);
  const int64_t s0 = blockIdx.x < grid ? total * blockIdx.x / grid : 0;
  const int64_t s1 = blockIdx.x < grid ? total * (blockIdx.x + 1) / grid : 0;
  const int64_t from = base + incl - own;
  if (tid == 0) {
    sh.s0 = s0;
    sh.s1 = s1;
    sh.total = total;
    sh.grid = (int)grid;
  }
  if (s0 < s1 && from <= s0 && s0 < from + own) {
    int64_t at = from;
    for (int b = b0, rc = rc0;;) {
      if (item_of(a, b, rc, m)) {
        const int units = m.nt + kStart;
        const int64_t u = (int64_t)units * a.Hkv;
        if (s0 < at + u) {
          sh.b = b;
          sh.rc = rc;
          sh.head = (int)((s0 - at) / units);
          sh.off = (int)((s0 - at) % units);
          sh.units = units;
          break;
        }
        at += u;
        ++rc;
      } else {
        rc = a.rc_max;
      }
      if (rc == a.rc_max) {
        rc = 0;
        ++b;
      }
    }
  }
  __syncthreads();
}

// The CTA whose share holds unit x.
__device__ __forceinline__ int cta_of(int64_t x, const Share& sh) {
  return (int)(((x + 1) * sh.grid - 1) / sh.total);
}

// An operand whose rows run along K, 64 elements of M or N in each of 128 bytes,
// 128-byte swizzled: 8-row groups 1024 bytes apart, 64-element blocks of M or N
// `block` bytes apart.
__device__ __forceinline__ uint64_t sw128_rows_desc(uint32_t addr, uint32_t block) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// kind::f16: A and B bf16 or fp16, A K-major, B K-major or (rows) along N; fp32
// D, M = 128.
__host__ __device__ constexpr uint32_t idesc16(int N, bool half, bool rows) {
  return (1u << 4) | (half ? 0u : (1u << 7) | (1u << 10)) | (rows ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kHalfRows >> 4) << 24);
}

// A box of 64 elements x 128 rows at (x, row, z), completing on `bar`.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row,
                                        int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(row), "r"(z)
      : "memory");
}

// A box of 64 elements from shared memory to (x, y, z), in a group of its own.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z,
                                          uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// This thread's stores have read shared memory; have ended.
__device__ __forceinline__ void bulk_read_wait() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// What a TMEM load has filled is not looked at before its wait.
__device__ __forceinline__ void settle(float* s) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+f"(s[i]), "+f"(s[i + 1]), "+f"(s[i + 2]), "+f"(s[i + 3]), "+f"(s[i + 4]),
                   "+f"(s[i + 5]), "+f"(s[i + 6]), "+f"(s[i + 7]));
}

// A warp's wait for a phase; false when another role has given up or after 1 s.
// (Short, as it stands in many places, whose code short items fetch anew: 64 prompts
// up to 500 tokens 136 -> 131 us.  The clock is read seldom.)
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t k = 1; !__all_sync(kFull, mbar_try_wait(bar, parity)); ++k) {
    if (k % 256 != 0) continue;
    const unsigned long long now = global_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(kFull, *abort != 0 || now - t0 > kWaitLimitNs)) {
      *abort = 1u;
      return false;
    }
  }
  return true;
}

// A place in the ring of tiles and the phase of its barriers.
template <int kRing>
struct Place {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// 64 scores of a row -> their probabilities 2^(c s - ref), written to TMEM in the
// elements' type; the unrounded ones are added to `sum`.
template <bool kHalf>
__device__ __forceinline__ void probabilities(const float* s, float c, float ref, uint32_t to,
                                              float& sum) {
  float b0 = sum, b1 = 0.0f, b2 = 0.0f, b3 = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float* v = s + w * 32;
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float y0, y1, y2, y3;
      fma2s(y0, y1, v[e], v[e + 1], c, -ref);
      fma2s(y2, y3, v[e + 2], v[e + 3], c, -ref);
      y0 = exp2_approx(y0);
      y1 = exp2_approx(y1);
      y2 = exp2_approx(y2);
      y3 = exp2_approx(y3);
      sum2(b0, b1, b0, b1, y0, y1);
      sum2(b2, b3, b2, b3, y2, y3);
      p[e / 2] = pack16<kHalf>(y0, y1);
      p[e / 2 + 1] = pack16<kHalf>(y2, y3);
    }
    tmem_st16(to + w * 16, p);
  }
  sum = (b0 + b1) + (b2 + b3);
}

// Barriers.
template <int D>
struct Bars {
  enum {
    kFullAt = 0,                      // a tile of the ring is loaded
    kEmpty = kFullAt + ring_of(D),    // and used
    kClean = kEmpty + ring_of(D),     // a value tile holds nothing that is not seen
    kSFull = kClean + kCleanRing,     // per half: its scores are in TMEM
    kPHalf = kSFull + 2,              // per half: 64 keys' probabilities are, O rescaled
    kPFull = kPHalf + 2,              // per half: and the others'
    kODone = kPFull + 2,              // per half: a segment's last product is done
    kQFull = kODone + 2,              // per half: its queries are in shared memory
    kQEmpty = kQFull + 2,             // per half: and used
    kSegFull = kQEmpty + 2,           // a segment is described
    kSegEmpty = kSegFull + kSegRing,  // and read by all
    kEnd = kSegEmpty + kSegRing,      // everything in flight is done
    kCount
  };
  // The arrivals that complete a barrier's phase.
  static __device__ __forceinline__ int arrivals(int i) {
    if (i >= kSegEmpty && i < kEnd) return kSegUsers;
    if (i >= kPHalf && i < kODone) return 4;
    if (i >= kClean && i < kSFull) return 2;
    return 1;
  }
};

template <int D>
struct Ctl {
  uint64_t bars[Bars<D>::kCount];
  Share share;
  Seg segs[kSegRing];
  uint32_t tmem;
  uint32_t abort;
};

template <int D, bool kHalf>
__global__ __launch_bounds__(kThreads, 1) void prompt_kernel(const __grid_constant__ PromptArgs a) {
  using B = Bars<D>;
  constexpr int kBlocks = D / 64;               // 64-element column blocks of a row
  constexpr uint32_t kBlock = kTile * 128;      // bytes of one, of 128 rows
  constexpr int kRing = ring_of(D);
  constexpr float kShift = kHalf ? 10.0f : -6.0f, kSlack = kHalf ? 4.0f : 8.0f;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl<D> ctl;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, skv = base + q_bytes(D);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  volatile uint32_t* abort = &ctl.abort;
  const auto bar = [&](int i) { return smem_addr(&ctl.bars[i]); };
  const auto slot_at = [&](uint32_t u) { return skv + u % kRing * kv_bytes(D); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // joins as CTAs end
  locate_share(a, ctl.share);
  const Share& share = ctl.share;
  // (a share may be empty, or end before the first tile of its first item)
  const int64_t begin = share.s0 - share.off;  // of that
  const bool theirs = a.whole && share.off > kStart;
  if (share.s0 >= share.s1 || begin + (theirs ? share.units : 0) + kStart >= share.s1) {
    if (tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < B::kCount; ++i) mbar_init(bar(i), B::arrivals(i));
    fence_mbar_init();
    ctl.abort = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&ctl.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ctl.tmem, 0);
  const uint32_t bars = bar(0);
  const auto wait = [&](int i, uint32_t parity) {
    const uint32_t b = bars + i * 8;
    return wait_on(b, parity, abort);
  };
  uint32_t loaded = 0, skipped = 0xffffffffu;  // warp 1: tiles asked for, one withheld
  uint32_t fills = 0;  // warps 2, 3: times that queries were asked for

  if (warp >= kSoftWarp) {
    // ------------------------------------------------------------- softmax
    set_regs_up<kSoftRegs>();
    const int half = (warp - kSoftWarp) / 4, rl = tid % kHalfRows;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + lanes + half * 128;
    const uint32_t to = tmem + lanes + 256 + half * D;
    // a factor of zero would make a masked score NaN
    const float c = fmaxf(a.scale_log2, 0x1p-100f);
    uint32_t n = 0, all = 0;  // tiles so far: of this half, of the CTA
    uint32_t done = 0;        // segments of this half so far
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = wait(B::kSegFull + i % kSegRing, i / kSegRing & 1u);
      if (!ok) break;
      const Seg& seg = ctl.segs[i % kSegRing];
      const Item& m = seg.m;
      const int nt = seg.t1 - seg.t0, t0 = seg.t0, ts_tiles = m.ts, tl = m.tl;
      const bool more = seg.more != 0;
      const bool both = m.rows > kHalfRows;
      if (half == 1 && !both) {  // no rows in this half
        all += nt;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::kSegEmpty + i % kSegRing));
        if (!more) break;
        continue;
      }
      const bool whole = seg.whole != 0;
      const int part = seg.part;
      const int w0 = half * kHalfRows + warp % 4 * 32;  // the warp's first row
      const int r = m.row0 + half * kHalfRows + rl;     // row of the sequence
      const bool live = half * kHalfRows + rl < m.rows;
      const int tok = (int)a.by_g.div(r);
      // (rows of the output stay below 2^31)
      const int orow = (m.q0 + tok) * a.Hq + seg.head * a.G + (r - tok * a.G);
      // the last key that the row sees, and for the warp's first and last row
      const int pos = live ? min(m.first + tok, m.hi - 1) : -1;
      const int pos_lo = min(m.first + (int)a.by_g.div(m.row0 + w0), m.hi - 1);
      const int pos_hi = m.first + (int)a.by_g.div(m.row0 + min(w0 + 31, m.rows - 1));
      const int lo_key = a.window > 0 ? m.first + tok - a.window + 1 : -(1 << 30);
      const bool idle = w0 >= m.rows;  // no row: keep the barriers going
      // one thread says when tiles and queries are used: what the tensor core has
      // been asked for before scores that are there is done
      const bool says = lane == 0 && warp % 4 == 0, says_all = says && half == (both ? 1 : 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kSegEmpty + i % kSegRing));
      float M = -INFINITY, l = 0.0f;
      for (int t = 0; t < nt; ++t, ++n, ++all) {
        const int kt = t0 + t;
        const int kb = (kt < ts_tiles ? kt : tl + (kt - ts_tiles)) * kTile;
        const bool full = kb + kTile <= pos_lo + 1 &&
                          (a.window <= 0 || kb > pos_hi - a.window || kb + kTile <= a.sinks);
        ok = wait(B::kSFull + half, n & 1u);
        if (!ok) break;
        fence_after();
        if (says_all) {
          if (t > 0) mbar_arrive(bar(B::kEmpty + (2 * all - 1) % kRing));
          mbar_arrive(bar(B::kEmpty + 2 * all % kRing));
        }
        if (says && t + 1 == nt) mbar_arrive(bar(B::kQEmpty + half));
        if (!idle) {
          float s[kTile];
#pragma unroll
          for (int w = 0; w < 4; ++w) tmem_ld32(ts + w * 32, s + w * 32);
          tmem_wait_ld();
#pragma unroll
          for (int w = 0; w < 4; ++w) settle(s + w * 32);
          if (__builtin_expect(!full, 0)) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int from = kb + w * 32;
              const uint32_t on = sees(pos - from, lo_key - from, a.sinks - from);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(on >> e & 1u)) s[w * 32 + e] = -INFINITY;
            }
          }
          const auto top = [&]() {
            return c * fmaxf(fmaxf(top32(s), top32(s + 32)), fmaxf(top32(s + 64), top32(s + 96)));
          };
          const float x = top();
          // ---- the sums' reference, moved seldom
          const bool move = x > M + (kShift + kSlack) || (M == -INFINITY && x != -INFINITY);
          if (__builtin_expect(__any_sync(kFull, move), 0)) {
            const float al = move ? exp2_approx(M - (x - kShift)) : 1.0f;
            if (move) M = x - kShift;
            l *= al;
            if (t > 0) {
              // few columns at a time: s stays in registers
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                float o[16];
                tmem_ld16(to + d, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  asm volatile("" : "+f"(o[j]));
                  o[j] *= al;
                }
                tmem_st16(to + d, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          float sum = 0.0f;
          probabilities<kHalf>(s, c, or_zero(M), ts, sum);
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::kPHalf + half));
          probabilities<kHalf>(s + 64, c, or_zero(M), ts + 32, sum);
          l += sum;
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(bar(B::kPHalf + half));
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::kPFull + half));
      }
      // ---- the output row
      if (ok) ok = wait(B::kODone + half, done++ & 1u);
      if (says_all) mbar_arrive(bar(B::kEmpty + (2 * all - 1) % kRing));
      if (ok && !idle) {
        fence_after();
        // (scores that are all NaN move no reference)
        const bool some = M != -INFINITY || l != l;
        const float inv = some ? __frcp_rn(l) : 0.0f;
        const float lse2 = some ? M + __log2f(l) : -INFINITY;
        const uint32_t stage = skv + kRing * kv_bytes(D) + (warp - kSoftWarp) * kStageBytes;
        const uint32_t lives = __ballot_sync(kFull, live);
#pragma unroll 1
        for (int d = 0; d < D; d += 64) {
          float o[64];
          __syncwarp();
          tmem_ld32(to + d, o);
          tmem_ld32(to + d + 32, o + 32);
          tmem_wait_ld();
          settle(o);
          settle(o + 32);
#pragma unroll
          for (int j = 0; j < 64; j += 2) mul2(o[j], o[j + 1], o[j], o[j + 1], inv, inv);
          if (!some)  // (0 times what an infinite value has left there)
#pragma unroll
            for (int j = 0; j < 64; ++j) o[j] = 0.0f;
          if (!whole) {
            if (live)
#pragma unroll
              for (int j = 0; j < 64; j += 4)
                *reinterpret_cast<float4*>(a.part_out +
                                           part_at<D>(part, d + j, half * kHalfRows + rl)) =
                    make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          } else {
            // A row a lane into shared memory.  Where all of the warp's rows are there
            // they leave by one asynchronous copy (the stores of an item's 64 KB took
            // 2,700 cycles), else 128 bytes of a row by 8 lanes.
            if (lane == 0) bulk_read_wait();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* v = o + 8 * j;
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                               stage + lane * 128 + ((j ^ lane) & 7) * 16),
                           "r"(pack16<kHalf>(v[0], v[1])), "r"(pack16<kHalf>(v[2], v[3])),
                           "r"(pack16<kHalf>(v[4], v[5])), "r"(pack16<kHalf>(v[6], v[7]))
                           : "memory");
            }
            if (a.o_tma && lives == kFull) {
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) {
                const int token = orow / a.Hq;
                tma_store(&a.omap, d, orow - token * a.Hq, token, stage);
              }
            } else {
              __syncwarp();
              const int c = lane % 8;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int row = j * 4 + lane / 8;
                const int at = __shfl_sync(kFull, orow, row);
                uint32_t u[4];
                lds128(stage + row * 128 + ((c ^ row) & 7) * 16, u);
                if (lives >> row & 1u)
                  *reinterpret_cast<uint4*>(a.out + (int64_t)at * D + d + c * 8) =
                      make_uint4(u[0], u[1], u[2], u[3]);
              }
            }
          }
        }
        const int64_t prow = (int64_t)part * kItemRows + half * kHalfRows + rl;
        if (live) {
          if (!whole)
            a.part_lse[prow] = lse2;
          else if (a.lse)
            a.lse[orow] = lse2 * kLn2;
        }
      }
      if (!more) break;
    }
    if (lane == 0) bulk_wait();
  } else {
    set_regs_down<kOtherRegs>();
  }
  if (warp >= kSideWarp && warp < kSoftWarp) {
    // ------------------------------------------- queries, unseen value rows
    const int half = warp - kSideWarp;
    uint32_t n = 0;  // tiles so far
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = wait(B::kSegFull + i % kSegRing, i / kSegRing & 1u);
      if (!ok) break;
      const Seg seg = ctl.segs[i % kSegRing];
      const Item& m = seg.m;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kSegEmpty + i % kSegRing));
      if (m.rows > half * kHalfRows) {
        if (fills > 0) ok = wait(B::kQEmpty + half, (fills - 1) & 1u);
        if (!ok) break;
        ++fills;
        const uint32_t to = sq + half * kBlocks * kBlock;
        if (a.q_tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B::kQFull + half), kHalfRows * D * 2);
            const int tok = m.q0 + (int)a.by_g.div(m.row0 + half * kHalfRows);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
              tma_box(to + k * kBlock, &a.qmap, k * 64, seg.head * a.G, tok, bar(B::kQFull + half));
          }
        } else {
#pragma unroll 1
          for (int row = lane; row < kHalfRows; row += 32) {  // a row a lane
            const int rr = half * kHalfRows + row, r = m.row0 + rr;
            const int tok = (int)a.by_g.div(r);
            const bool real = rr < m.rows;
            const uint16_t* src = a.q;
            if (real)
              src += (m.q0 + tok) * a.q_ts + (int64_t)(seg.head * a.G + r - tok * a.G) * a.q_hs;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               to + c / 8 * kBlock + row * 128 + ((c ^ row) & 7) * 16),
                           "l"(src + c * 8), "r"(real ? 16 : 0)
                           : "memory");
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::kQFull + half));
        }
      }
      for (int t = seg.t0; t < seg.t1 && ok; ++t, ++n) {
        // (the value tile alone, whose slot is not filled again before this warp's
        // arrival: a key tile's slot is given back without it, so that its barrier
        // could complete twice unseen)
        const uint32_t u = 2 * n + 1;
        ok = wait(B::kFullAt + u % kRing, u / kRing & 1u);
        if (!ok) break;
        const int kb = key_of_tile(m, t);
        // this warp's 64 rows of the tile
        bool touched = false;
#pragma unroll 1
        for (int w = 2 * half; w < 2 * half + 2; ++w) {
          const int from = kb + 32 * w;
          const uint32_t on = sees(m.hi - 1 - from, m.lo - from, a.sinks - from);
          if (on == kFull) continue;
          touched = true;
          const uint32_t at = slot_at(u) + (w * 32 + lane / 8) * 128 + lane % 8 * 16;
#pragma unroll 1
          for (int e = 0; e < 32; e += 4)
            if (!(on >> (e + lane / 8) & 1u))
#pragma unroll
              for (int k = 0; k < kBlocks; ++k)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + e * 128 +
                                                                           k * kBlock),
                             "r"(0)
                             : "memory");
        }
        if (touched) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::kClean + n % kCleanRing));
      }
      if (!seg.more) break;
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t kQkDesc = idesc16(kTile, kHalf, false), kPvDesc = idesc16(D, kHalf, true);
    // a descriptor's address field moves by (bytes >> 4)
    const uint64_t dq = sw128_desc(sq), dk = sw128_desc(skv);
    const uint64_t dv = sw128_rows_desc(skv, D == 128 ? kBlock : 1024);
    const uint32_t elected = elect_one();
    const auto issue_s = [&](int half, uint32_t slot) {
      const uint64_t qa = dq + half * (kBlocks * kBlock >> 4);
      const uint64_t kb = dk + slot * (kv_bytes(D) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(elected, tmem + half * 128, qa + (k / 4 * (kBlock >> 4) + k % 4 * 2),
               kb + (k / 4 * (kBlock >> 4) + k % 4 * 2), kQkDesc, k > 0);
      mma_commit(elected, bar(B::kSFull + half));
    };
    // the product with 64 keys' values
    const auto issue_o = [&](int half, uint32_t slot, int keys, bool first) {
      const uint64_t vb = dv + slot * (kv_bytes(D) >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ts(elected, tmem + 256 + half * D, tmem + half * 128 + keys / 2 + k * 8,
               vb + (keys / 16 + k) * (2048 >> 4), kPvDesc, !first || k > 0);
    };
    bool ok = true;
    uint32_t n = 0, n_b = 0;    // tiles so far: of the CTA (and half A), of half B
    uint32_t q_a = 0, q_b = 0;  // segments so far, of each half
    Place<kRing> at;            // the next tile
    for (uint32_t i = 0; ok; ++i) {
      ok = wait(B::kSegFull + i % kSegRing, i / kSegRing & 1u);
      if (!ok) break;
      const Seg& seg = ctl.segs[i % kSegRing];
      const int nt = seg.t1 - seg.t0;
      const int halves = seg.m.rows > kHalfRows ? 2 : 1;
      const bool more = seg.more != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kSegEmpty + i % kSegRing));
      ok = wait(B::kFullAt + at.slot, at.phase);
      for (int h = 0; h < halves && ok; ++h) {
        ok = wait(B::kQFull + h, (h ? q_b : q_a) & 1u);
        if (!ok) break;
        fence_after();
        issue_s(h, at.slot);
      }
      ++q_a;
      q_b += halves - 1;
      at.next();
      for (int t = 0; t < nt && ok; ++t, ++n) {
        const uint32_t v = at.slot;  // keys' and values' tiles take turns
        const bool last = t + 1 == nt;
        at.next();
        // (a clean tile has been loaded)
        ok = wait(B::kClean + n % kCleanRing, n / kCleanRing & 1u) &&
             (last || wait(B::kFullAt + at.slot, at.phase));
        for (int h = 0; h < halves && ok; ++h) {
          const uint32_t parity = (h ? n_b : n) & 1u;
          ok = wait(B::kPHalf + h, parity);
          if (!ok) break;
          fence_after();
          issue_o(h, v, 0, t == 0);
          ok = wait(B::kPFull + h, parity);
          if (!ok) break;
          fence_after();
          issue_o(h, v, 64, false);
          if (last)
            mma_commit(elected, bar(B::kODone + h));
          else
            issue_s(h, at.slot);
        }
        if (!ok) break;
        n_b += halves - 1;
        if (!last) at.next();
      }
      if (!more) break;
    }
  } else if (warp == kLoadWarp) {
    // -------------------------------------------------- work list and tiles
    int b = share.b, rc = share.rc, head = share.head;
    int64_t at = begin;  // the item's first unit
    int4 cut = make_int4(0, 0, 0, 0);
    bool more = true;
    const auto next_item = [&]() {
      if (++head < a.Hkv) return;
      head = 0;
      Item it;
      if (++rc < a.rc_max && item_of(a, b, rc, it)) return;
      // the next sequence with rows, 32 looked at at once: the other warps' waits for
      // the next segment run out after a second
      rc = 0;
      for (++b;; b += 32) {
        const uint32_t has =
            __ballot_sync(kFull, lane < a.batch - b && item_of(a, b + lane, 0, it));
        if (has != 0) b += __ffs(has) - 1;
        if (has != 0 || a.batch - b <= 32) break;
      }
    };
    if (theirs) {
      at += share.units;
      next_item();
    }
    // (testing hook, see fp4idx_test_withhold_next: a tile that is not loaded)
    const uint32_t held = blockIdx.x == 0 && a.withhold >= 0 ? 2u * a.withhold : 0xffffffffu;
    bool ok = true;
    for (uint32_t i = 0; more && ok; ++i) {
      if (i >= kSegRing) ok = wait(B::kSegEmpty + i % kSegRing, (i / kSegRing + 1) & 1u);
      if (!ok) break;
      Seg sg;
      item_of(a, b, rc, sg.m);
      sg.head = head;
      const int units = sg.m.nt + kStart;
      const int64_t tiles = at + kStart;  // the unit of the first one
      sg.t0 = a.whole ? 0 : (int)max(share.s0 - tiles, (int64_t)0);
      sg.t1 = a.whole ? sg.m.nt : (int)min(share.s1 - tiles, (int64_t)sg.m.nt);
      sg.whole = sg.t0 == 0 && sg.t1 == sg.m.nt;
      sg.part = 2 * blockIdx.x + (sg.t0 == 0 && i > 0 ? 1 : 0);
      if (!sg.whole && sg.t0 == 0)  // the first fragment of a cut item
        cut = make_int4(b, rc, head,
                        (cta_of(at + units - 1, share) - (int)blockIdx.x + 1) * 2 + (sg.part & 1));
      at += units;
      more = at + kStart < share.s1;  // the next item's first tile
      sg.more = more;
      if (lane == 0) {
        ctl.segs[i % kSegRing] = sg;
        mbar_arrive(bar(B::kSegFull + i % kSegRing));
      }
      for (int t = sg.t0; t < sg.t1 && ok; ++t) {
        const int row = sg.m.k0 + key_of_tile(sg.m, t);
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t u = loaded;
          if (u >= (uint32_t)kRing) ok = wait(B::kEmpty + u % kRing, (u / kRing + 1) & 1u);
          if (!ok) break;
          ++loaded;
          if (u == held) {
            skipped = u;
            continue;
          }
          if (lane == 0) {
            const uint32_t full = bar(B::kFullAt + u % kRing);
            mbar_arrive_expect_tx(full, kv_bytes(D));
            const CUtensorMap* map = kv ? &a.vmap : &a.kmap;
            const int x = head * (kv ? a.vx : a.kx), z = head * (kv ? a.vz : a.kz);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
              tma_box(slot_at(u) + k * kBlock, map, x + k * 64, row, z, full);
          }
          __syncwarp();
        }
      }
      if (more) next_item();
    }
    if (lane == 0) a.cuts[blockIdx.x] = cut;
  }

  __syncwarp();
  fence_before();
  __syncthreads();
  if (*abort) {
    // Copies and MMAs in flight land before shared memory and TMEM are
    // released.  A commit stands for its own lane's MMAs: the lane that was
    // elected to issue them.
    if (warp == kLoadWarp)
      for (uint32_t u = loaded > (uint32_t)kRing ? loaded - kRing : 0; u < loaded; ++u)
        if (u != skipped) mbar_wait_bounded(bar(B::kFullAt + u % kRing), u / kRing & 1u);
    if (a.q_tma && warp >= kSideWarp && warp < kSoftWarp && fills > 0)
      mbar_wait_bounded(bar(B::kQFull + warp - kSideWarp), (fills - 1) & 1u);
    if (warp == kMmaWarp && elect_one()) {
      flag_error(a.err, FP4IDX_ERRFLAG_TIMEOUT);
      const uint32_t b = bar(B::kEnd);
      mma_commit(1, b);
      mbar_wait_bounded(b, 0);
    }
    __syncthreads();
  }
  __syncwarp();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the partial outputs of the items that a share's end cut: weights
// 2^(lse - max), applied in two halves (a part of weight 2^-126 counts where its
// values are as much larger), in the order of the CTAs.  A warp takes 32 rows, a row a lane, and
// 16 elements of each: it reads partial outputs in runs of 512 bytes and writes 32
// bytes a row.  Blocks (CTA whose share begins the item, 4,096 of
// its elements).
template <int D, bool kHalf>
__global__ __launch_bounds__(256) void join_prompt_kernel(const __grid_constant__ PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kParts = D / 16, kRowsOf = 8 / kParts * 32;  // warps of a row; rows of a block
  const int cta = blockIdx.x / (kItemRows / kRowsOf);
  const int4 cut = a.cuts[cta];
  const int n = cut.w / 2;
  if (n < 2) return;
  Item m;
  item_of(a, cut.x, cut.y, m);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int row = blockIdx.x % (kItemRows / kRowsOf) * kRowsOf + warp / kParts * 32 + lane;
  const int d = warp % kParts * 16;
  if (row >= m.rows) return;
  const auto slot = [&](int f) { return (int64_t)2 * (cta + f) + (f == 0 ? cut.w & 1 : 0); };
  float top = -INFINITY;
  bool nan = false;
#pragma unroll 4
  for (int f = 0; f < n; ++f) {
    const float x = a.part_lse[slot(f) * kItemRows + row];
    nan = nan || x != x;
    top = fmaxf(top, x);
  }
  // (parts that are all NaN have no largest)
  const bool some = top != -INFINITY || nan;
  const float ref = or_zero(top);
  float den = 0.0f, o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.0f;
#pragma unroll 4
  for (int f = 0; f < n; ++f) {
    const int64_t place = slot(f);
    const float w = exp2_approx(0.5f * (a.part_lse[place * kItemRows + row] - ref));
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const float4*>(a.part_out + part_at<D>(place, d + 4 * j, row));
    den = fmaf(w, w, den);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[4 * j] = fmaf(v[j].x * w, w, o[4 * j]);
      o[4 * j + 1] = fmaf(v[j].y * w, w, o[4 * j + 1]);
      o[4 * j + 2] = fmaf(v[j].z * w, w, o[4 * j + 2]);
      o[4 * j + 3] = fmaf(v[j].w * w, w, o[4 * j + 3]);
    }
  }
  const float inv = some ? __frcp_rn(den) : 0.0f;
  const int r = m.row0 + row, tok = (int)a.by_g.div(r);
  const int64_t orow = (int64_t)(m.q0 + tok) * a.Hq + cut.z * a.G + (r - tok * a.G);
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = pack16<kHalf>(o[2 * j] * inv, o[2 * j + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + d);
  dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
  dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
  if (a.lse && d == 0) a.lse[orow] = some ? (top + __log2f(den)) * kLn2 : -INFINITY;
}

template <int D, bool kHalf>
fp4idx_status launch_prompt(const PromptArgs& a, int grid, cudaStream_t stream) {
  static SmemOnce once;
  if (!once.set(prompt_kernel<D, kHalf>, smem_bytes(D))) return FP4IDX_ERR_CUDA;
  if (launch_kernel(prompt_kernel<D, kHalf>, (unsigned)grid, kThreads, smem_bytes(D), stream, a) !=
      cudaSuccess)
    return FP4IDX_ERR_CUDA;
  if (a.whole) return FP4IDX_OK;
  return launch_after(join_prompt_kernel<D, kHalf>, (unsigned)(grid * (D / 16)), 256, stream,
                      a) == cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}

struct Workspace {
  int64_t part_lse, cuts, total;  // offsets in bytes; partial outputs at 0
};

// Two partial outputs per CTA (an item cut at its share's start and one at
// its end), and the cut items.
Workspace workspace_of(int64_t head_dim) {
  Workspace w;
  w.part_lse = 2 * kMaxGrid * kItemRows * head_dim * 4;
  w.cuts = w.part_lse + 2 * kMaxGrid * kItemRows * 4;
  w.total = w.cuts + (kMaxGrid * 16 + 255) / 256 * 256;
  return w;
}

bool workspace_args_ok(int64_t batch, int64_t max_q, int64_t num_heads, int64_t kv_heads,
                       int64_t head_dim) {
  return batch >= 0 && max_q >= 1 && kv_heads >= 1 && kv_heads <= 65535 &&
         num_heads >= kv_heads && num_heads % kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && batch < (1ll << 31) && num_heads < (1ll << 20) &&
         max_q < (1ll << 31) / num_heads;
}

// CTAs of a call: one per SM, or as many as its items can have tiles, where a key head
// has `rows` rows in all.
constexpr int grid_of(int64_t rows, int64_t batch, int64_t kv_heads, int64_t max_k) {
  const int64_t chunks = (rows + kItemRows - 1) / kItemRows + batch;
  if (chunks >= kMaxGrid) return kMaxGrid;
  const int64_t tiles = chunks * kv_heads * (max_k / kTile + 1);  // below 2^47
  return tiles < kMaxGrid ? (int)tiles : (int)kMaxGrid;
}
static_assert(grid_of(1, 1, 1, 0) == 2 && grid_of(256, 1, 2, 1000) == 32, "tiles of a small call");
// (the largest sizes that a call may have: the product of all does not fit 64 bits)
static_assert(grid_of((1ll << 31) - 1, (1ll << 31) - 1, 65535, (1 << 30) - 1) == kMaxGrid &&
                  grid_of(1, 1, 65535, (1 << 30) - 1) == kMaxGrid &&
                  grid_of(1, kMaxGrid - 2, 65535, (1 << 30) - 1) == kMaxGrid,
              "tiles of the largest calls");

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's call that describes a tensor to the TMA unit.
EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> found{nullptr};
  EncodeTiled f = found.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult got;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &got) != cudaSuccess ||
      got != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiled>(p);
  found.store(f, std::memory_order_release);
  return f;
}

// How the rows of k or v lie: a token's heads within its stride (the map's first
// axis spans them), or a head's tokens within its stride (its last axis).
struct Rows {
  uint64_t dim[3], stride[2];  // strides of the second and third axis, in bytes
  int32_t x, z;                // a head's step in the first and last coordinate
  bool shape_ok, align_ok;
};

Rows rows_of(int64_t tokens, int64_t heads, int64_t head_dim, int64_t ts, int64_t hs) {
  Rows r = {};
  if (heads == 1) hs = 0;
  if (tokens == 1) ts = (heads - 1) * hs + head_dim;
  if (ts < 0 || hs < 0 || ts >= (1ll << 38) || hs >= (1ll << 38)) return r;
  const int64_t span = (heads - 1) * hs + head_dim;
  r.align_ok = ts % 8 == 0 && hs % 8 == 0;
  if (ts >= span) {
    r.shape_ok = span < (1ll << 31) && ts <= (1ll << 38) / (tokens > 0 ? tokens : 1);
    r.dim[0] = span;
    r.dim[1] = tokens;
    r.dim[2] = 1;
    r.stride[0] = ts * 2;
    r.stride[1] = r.shape_ok ? ts * 2 * tokens : 0;
    r.x = (int32_t)hs;
  } else if (ts >= head_dim && hs >= ts && (tokens - 1) <= (hs - head_dim) / ts) {
    r.shape_ok = hs % ts == 0 && hs <= (1ll << 38) / heads;
    r.dim[0] = head_dim;
    r.dim[1] = tokens;
    r.dim[2] = heads;
    r.stride[0] = ts * 2;
    r.stride[1] = hs * 2;
    r.z = 1;
  }
  return r;
}

// The same of q, heads before tokens, if a half's rows are whole tokens and a
// token's heads lie within its stride.
bool query_rows(Rows& r, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t ts,
                int64_t hs) {
  if (kHalfRows % group) return false;
  if (heads == 1) hs = head_dim;
  if (tokens == 1) ts = heads * hs;
  if (hs < head_dim || ts < heads * hs || ts % hs || ts > (1ll << 38) / tokens) return false;
  r = {};
  r.dim[0] = head_dim;
  r.dim[1] = heads;
  r.dim[2] = tokens;
  r.stride[0] = hs * 2;
  r.stride[1] = ts * 2;
  return true;
}

// A map of boxes of 64 elements x box1 x box2.
bool encode(CUtensorMap* map, const void* base, const Rows& r, bool half, uint32_t box1 = kTile,
            uint32_t box2 = 1) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dim[3] = {r.dim[0], r.dim[1], r.dim[2]}, stride[2] = {r.stride[0], r.stride[1]};
  const cuuint32_t box[3] = {64, box1, box2}, step[3] = {1, 1, 1};
  return f(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
           const_cast<void*>(base), dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Testing hook: the tile that the next launch withholds (-1: none), taken once.
std::atomic<int64_t> g_prompt_withhold{-1};

}  // namespace

void prompt_withhold_next(int64_t index) { g_prompt_withhold.store(index); }

}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" size_t fp4idx_prompt_workspace_bytes(int64_t batch, int64_t max_q, int64_t num_heads,
                                                int64_t kv_heads, int64_t head_dim) {
  if (!workspace_args_ok(batch, max_q, num_heads, kv_heads, head_dim)) return 0;
  return (size_t)workspace_of(head_dim).total;
}

extern "C" fp4idx_status fp4idx_prompt_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
    int64_t v_head_stride, int dtype, const int32_t* q_starts, const int32_t* k_starts,
    int64_t max_q, int64_t max_k, int64_t window, int64_t sinks, float softmax_scale, void* out,
    float* lse, int64_t batch, int64_t q_tokens, int64_t k_tokens, int64_t num_heads,
    int64_t kv_heads, int64_t head_dim, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream) {
  if (batch < 0 || q_tokens < 0 || k_tokens < 0) return FP4IDX_ERR_SHAPE;
  if (batch == 0 || q_tokens == 0) return FP4IDX_OK;
  if (!q || !q_starts || !out || !workspace || (k_tokens > 0 && (!k || !v)))
    return FP4IDX_ERR_NULL;
  if (!workspace_args_ok(batch, max_q, num_heads, kv_heads, head_dim) || max_k < 0 ||
      q_tokens >= (1ll << 31) / num_heads || q_tokens >= (1 << 30) || k_tokens >= (1 << 30) ||
      max_q >= (1 << 30) || max_k >= (1 << 30))
    return FP4IDX_ERR_SHAPE;
  const Rows kr = rows_of(k_tokens, kv_heads, head_dim, k_token_stride, k_head_stride);
  const Rows vr = rows_of(k_tokens, kv_heads, head_dim, v_token_stride, v_head_stride);
  if (k_tokens > 0 && (!kr.shape_ok || !vr.shape_ok)) return FP4IDX_ERR_SHAPE;
  const Workspace w = workspace_of(head_dim);
  if (workspace_bytes < (size_t)w.total) return FP4IDX_ERR_SCRATCH;
  if (!dtype_ok(dtype) || !isfinite(softmax_scale) || softmax_scale < 0.0f || window < 0 ||
      sinks < 0 || out == q || (k_tokens > 0 && (out == k || out == v)))
    return FP4IDX_ERR_ARG;
  if (!aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 || !aligned(k, 16) ||
      !aligned(v, 16) || (k_tokens > 0 && (!kr.align_ok || !vr.align_ok)) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(q_starts, 4) ||
      !aligned(k_starts, 4) || !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  PromptArgs a = {};
  const bool half = dtype == FP4IDX_FP16;
  a.q = static_cast<const uint16_t*>(q);
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.q_starts = q_starts;
  a.k_starts = k_starts ? k_starts : q_starts;
  a.max_q = (int32_t)max_q;
  a.max_k = (int32_t)max_k;
  // a window that holds every key is no window (a sequence may have more than max_k:
  // its window still ends at the query)
  a.window = window < k_tokens ? (int32_t)window : 0;
  a.sinks = (int32_t)(sinks < max_k ? sinks : max_k);
  a.batch = (int32_t)batch;
  a.Tq = (int32_t)q_tokens;
  a.Tk = (int32_t)k_tokens;
  a.Hq = (int32_t)num_heads;
  a.Hkv = (int32_t)kv_heads;
  a.G = (int32_t)(num_heads / kv_heads);
  a.by_g = make_fastdiv((uint32_t)a.G);
  const int64_t most_q = max_q < q_tokens ? max_q : q_tokens;
  a.rc_max = (int32_t)((most_q * a.G + kItemRows - 1) / kItemRows);
  // tiles of an item, at most
  int64_t tiles = (max_k + kTile - 1) / kTile;
  if (a.window > 0) {
    const int64_t seen = (a.window + kItemRows / a.G + 2 * kTile) / kTile +
                         (a.sinks + kTile - 1) / kTile;
    if (seen < tiles) tiles = seen;
  }
  a.whole = tiles <= kWhole;
  a.withhold = -1;
  a.scale_log2 = softmax_scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  a.part_out = reinterpret_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.cuts = reinterpret_cast<int4*>(ws + w.cuts);
  a.err = err_flags;
  if (k_tokens > 0) {
    a.kx = kr.x;
    a.kz = kr.z;
    a.vx = vr.x;
    a.vz = vr.z;
    if (!encode(&a.kmap, k, kr, half) || !encode(&a.vmap, v, vr, half)) return FP4IDX_ERR_CUDA;
  } else {  // no key: one row of the workspace, which no query sees
    const Rows none = rows_of(1, 1, head_dim, head_dim, head_dim);
    if (!encode(&a.kmap, workspace, none, half)) return FP4IDX_ERR_CUDA;
    a.vmap = a.kmap;
  }
  Rows qr;
  a.q_tma = query_rows(qr, q_tokens, num_heads, a.G, head_dim, q_token_stride, q_head_stride);
  if (a.q_tma && !encode(&a.qmap, q, qr, half, a.G, kHalfRows / a.G)) return FP4IDX_ERR_CUDA;
  Rows orows;
  a.o_tma = kWarpRows % a.G == 0 &&
            query_rows(orows, q_tokens, num_heads, a.G, head_dim, num_heads * head_dim, head_dim);
  if (a.o_tma && !encode(&a.omap, out, orows, half, a.G, kWarpRows / a.G)) return FP4IDX_ERR_CUDA;
  if (g_prompt_withhold.load(std::memory_order_relaxed) >= 0) {
    const int64_t held = g_prompt_withhold.exchange(-1);
    if (held < (1 << 28)) a.withhold = (int32_t)held;
  }
  const int grid = grid_of(q_tokens * a.G, batch, kv_heads, max_k);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (head_dim == 128)
    return half ? launch_prompt<128, true>(a, grid, s) : launch_prompt<128, false>(a, grid, s);
  return half ? launch_prompt<64, true>(a, grid, s) : launch_prompt<64, false>(a, grid, s);
}
