// fp4idx_attn_tiles.cu -- attention over the 8-bit cache for many query rows
// per key head: prompts in whole or in chunks (fp4idx_paged_attention_fp8,
// defined in include/fp4idx_attention.h), on the tensor cores through
// tcgen05.mma kind::f16.
//
// What bounds it.  4 D operations per query row and key against 2 D bytes per
// key for a whole item of 256 rows: the tensor cores, then the exponentials.
// Measured: 4 chunks of up to 1,500 tokens, 32 heads of 128 over 8 key heads,
// contexts up to 16,384, 486 us, 55% of the bf16 rate.  That is 4,800 cycles for
// each of a CTA's 210 tiles at 2,070 MHz, segments' starts and ends among them;
// the MMAs of a tile alone take 2,051, a half's softmax 1,222 to 1,706.  (Where
// the rest goes is not measured; the tensor pipe is busy 45% of the time.)
//
// Mathematics.  As in fp4idx_attn_rows.cu: E4M3 codes are exact in fp16 and a
// query row is scaled by a power of two into fp16's range (with the sign of
// softmax_scale, so that the factor c of a page, ks * scale * log2(e) times
// the row's power, is not negative).  A row keeps m = max s, l = sum 2^(s-m)
// and M, the reference of its output sums: p = 2^(s + log2 vs - M + 10), in
// fp16.  M follows max (s + log2 vs) only when that has grown by more than 4,
// so p <= 2^14 and the sums in TMEM are seldom rescaled; p is rounded to
// 2^-11 of itself, or 2^-35 of the largest contribution.  l is summed from
// the same exponentials, moved by the difference of the two references; a
// page whose values are 2^60 below M's takes exponentials of its own for l.
//
// Roles (one CTA per SM).  The item's rows are two M = 128 halves A and B that
// share every key tile of 128 keys (two pages).
//   warp 0          issues the MMAs: S = Q K^T, then O += P V with P from
//                   TMEM.  While half A's softmax runs, half B's products do.
//                   (One issuer for both keeps the halves out of step; with an
//                   issuer each they fell into step and 501 us became 643.)
//   warp 1          walks the CTA's list of work and describes its segments
//                   and, eight ahead, its tiles: pages, scales, visible rows
//   warps 4-7       converters: the codes from global memory through
//                   registers to fp16 tiles in shared memory, keys as
//                   [key][d], values transposed as [d][key], both K-major in
//                   128-byte swizzled rows, two stages each; the next tile's
//                   loads are in flight while this one is converted
//   warps 8-11, 12-15  softmax of half A, of half B: a row per thread, its
//                   scores read from TMEM a page at a time, its probabilities
//                   written back over them.  A register spilled here costs
//                   much: the shared memory leaves L1 too small to hold it
//                   (60 bytes of spills a thread: 770 us).
// TMEM: scores A and B at columns 0 and 128 (P over the first page's scores,
// once those are in registers), O at 256 and 256 + D.
// The items and their tiles form one list, cut into equal shares, one per CTA,
// from the lengths alone; an item cut by a share's end leaves normalised
// partial outputs, joined by a second kernel in a fixed order.
// Every wait is bounded (1 s) and a shared abort flag stops every role; MMAs
// in flight are waited for before TMEM is released.

#include <type_traits>

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kPage = FP4IDX_KV_BLOCK;
constexpr int kTile = 128;  // keys of a tile
constexpr int kHalfRows = 128;
constexpr int kItemRows = 2 * kHalfRows;
constexpr int kMmaWarp = 0, kSegWarp = 1, kConvWarp = 4, kSoftWarp = 8;
constexpr int kSegUsers = 9;       // warps that read a segment: the issuer and the softmax
constexpr int kThreads = 16 * 32;  // warps 2-3 only complete the warpgroup
// Registers of a thread, by warpgroup: the launch's 128, moved from the others
// to the softmax.
constexpr int kLaunchRegs = 128, kSoftRegs = 144, kConvRegs = 128, kMmaRegs = 96;
static_assert(2 * kSoftRegs + kConvRegs + kMmaRegs <= 4 * kLaunchRegs, "the launch's registers");
constexpr int kStages = 2;
constexpr int kTileRing = 8;
constexpr int kSegRing = 2;
constexpr float kShift = 10.0f, kSlack = 4.0f, kFar = 60.0f;
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t q_bytes(int D) { return kItemRows * D * 2; }
__host__ __device__ constexpr uint32_t kv_bytes(int D) { return kTile * D * 2; }
__host__ __device__ constexpr uint32_t smem_bytes(int D) {
  return q_bytes(D) + 2 * kStages * kv_bytes(D) + 1024;
}

// One item: 256 consecutive rows (token i, head g: row i * G + g) of a
// sequence and key head.
struct Item {
  int row0, rows;
  int q0, first;  // first query token of the sequence, its position
  int lo, hi;     // keys that any row sees: [lo, hi) and [0, sinks)
  int ts, tl;     // tiles: 0 .. ts-1, then tl ..
  int nt;         // tiles in all, at least one
};

// The rows' chunk rc of sequence b; false: it has no rows.
__device__ __forceinline__ bool item_of(const AttnArgs& a, int b, int rc, Item& m) {
  const int ctx = min(max(__ldg(a.ctx + b), 0), a.max_context);
  int full = a.max_q;
  m.q0 = b * a.max_q;
  if (a.starts) {
    m.q0 = __ldg(a.starts + b);
    full = max(__ldg(a.starts + b + 1) - m.q0, 0);
  }
  m.first = ctx - full;
  m.row0 = rc * kItemRows;
  m.rows = min(min(full, a.max_q) * a.G - m.row0, kItemRows);
  m.hi = max(min(ctx, m.first + (m.row0 + m.rows - 1) / a.G + 1), 0);
  m.lo = a.window > 0 ? min(max(m.first + m.row0 / a.G - a.window + 1, 0), m.hi) : 0;
  m.tl = m.lo / kTile;
  m.ts = a.window > 0 ? min((a.sinks + kTile - 1) / kTile, m.tl) : 0;
  m.nt = max(m.ts + (m.hi + kTile - 1) / kTile - m.tl, 1);
  return m.rows > 0;
}

// The first key of the item's tile t.
__device__ __forceinline__ int key_of_tile(const Item& m, int t) {
  return (t < m.ts ? t : m.tl + (t - m.ts)) * kTile;
}

// The list of work: for each sequence, row chunk and key head the item's
// tiles.  It is cut into equal shares, one per CTA.
struct Share {
  int64_t s0, s1, total;
  int b, rc, head, off;  // the item of unit s0, and the tile in it
  int grid;              // CTAs with a share
};

// A segment of the share: an item's tiles [t0, t1).
struct Seg {
  Item m;
  int b, head, t0, t1;
  int whole;  // the item as a whole
  int part;   // else the slot of its partial outputs
  int more;   // segments follow
};

// This CTA's share, by the whole CTA.
__device__ __forceinline__ void locate_share(const AttnArgs& a, Share& sh) {
  __shared__ int64_t part[kThreads / 32];
  __shared__ int count[kThreads / 32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t pairs = (int64_t)a.batch * a.rc_max;
  const int64_t each = (pairs + kThreads - 1) / kThreads;
  const int64_t p0 = min(tid * each, pairs), p1 = min(p0 + each, pairs);
  int64_t own = 0;
  int items = 0;
  Item m;
  for (int64_t p = p0; p < p1; ++p)
    if (item_of(a, (int)(p / a.rc_max), (int)(p % a.rc_max), m)) {
      own += m.nt;
      ++items;
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
  const int64_t grid = min(max(total / 4, min(n * a.Hkv, most)), most);
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
    for (int64_t p = p0;; ++p) {
      const int b = (int)(p / a.rc_max), rc = (int)(p % a.rc_max);
      if (!item_of(a, b, rc, m)) continue;
      const int64_t u = (int64_t)m.nt * a.Hkv;
      if (s0 < at + u) {
        sh.b = b;
        sh.rc = rc;
        sh.head = (int)((s0 - at) / m.nt);
        sh.off = (int)((s0 - at) % m.nt);
        break;
      }
      at += u;
    }
  }
  __syncthreads();
}

// The CTA whose share holds unit x.
__device__ __forceinline__ int cta_of(int64_t x, const Share& sh) {
  return (int)(((x + 1) * sh.grid - 1) / sh.total);
}

// Waits for a phase; false when another role has given up or after 1 s.  The
// clock is read seldom: a read of it costs more than most waits take.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  unsigned long long t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 256; ++k)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const unsigned long long now = global_ns();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > kWaitLimitNs) {
      *abort = 1u;
      return false;
    }
  }
}

// K-major operand in the 128-byte swizzled layout: rows of 128 bytes, 8-row
// groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// kind::f16: fp16 A and B, both K-major, fp32 D, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kHalfRows >> 4) << 24);
}

// The MMAs and commits take the elected lane as a predicate: the whole warp
// computes their operands, which then live in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(elected)
      : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 columns of the thread's lane, as fp32.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
        "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
        "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The largest of 32 values, two to an instruction in four chains.
__device__ __forceinline__ float top32(const float* s) {
  float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < 28; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = max3(x[j], s[i + 2 * j], s[i + 2 * j + 1]);
  return max3(max3(x[0], s[28], s[29]), max3(x[1], s[30], s[31]), fmaxf(x[2], x[3]));
}

// (a * b + c, a' * b + c) packed.
__device__ __forceinline__ void fma2s(float& r0, float& r1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rr;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %4};\n\t"
      "mov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rr, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rr;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

__device__ __forceinline__ float log2_scale(float s) {
  return (float)((int)(__float_as_uint(s) >> 23 & 0xffu) - 127);
}

__device__ __forceinline__ float or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// Bits i of a word with i <= last.
__device__ __forceinline__ uint32_t bits_to(int last) {
  return last >= 31 ? kFull : last < 0 ? 0u : (2u << last) - 1u;
}

// The keys that a row sees of 32 of a tile's: key i (from the first of the 32)
// with i <= hi and (i >= lo or i < sk).
__device__ __forceinline__ uint32_t sees(int hi, int lo, int sk) {
  return bits_to(hi) & (~bits_to(lo - 1) | bits_to(sk - 1));
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barriers.
enum {
  kKFull = 0,
  kKEmpty = kKFull + kStages,
  kVFull = kKEmpty + kStages,
  kVEmpty = kVFull + kStages,
  kSFull = kVEmpty + kStages,  // per half: its scores are in TMEM
  kPFull = kSFull + 2,         // per half: its probabilities are, O rescaled
  kODone = kPFull + 2,         // per half: the product with the values is done
  kQFull = kODone + 2,         // per half: its queries are in shared memory
  kSegFull = kQFull + 2,       // a segment is described
  kSegEmpty = kSegFull + kSegRing,
  kTileFull = kSegEmpty + kSegRing,  // a tile is described
  kTileFree = kTileFull + kTileRing,  // and nothing reads that any more
  kBars = kTileFree + kTileRing
};

// The arrivals that complete a barrier's phase.
__device__ __forceinline__ int arrivals(int i) {
  if (i >= kTileFull) return 1;
  if (i >= kSegEmpty) return kSegUsers;
  if (i >= kSegFull) return 1;
  const bool commit = (i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kPFull) ||
                      (i >= kODone && i < kQFull);
  return commit ? 1 : 4;
}

// A tile of the CTA's list, described ahead of its use.  A page that holds no
// visible key (below the window, behind the first tokens) is not looked up, and
// the rows that the item does not see are not loaded: zeros take their place,
// since a probability of 0 times a NaN code is NaN.  (Two words a page: with
// 64-bit masks the converters' tests took the prompts' 485 us to 496.)
struct alignas(16) TileInfo {
  float scale[4];       // ks of its two pages, vs of both (negative: page left out)
  int64_t off[2];       // bytes from the codes' start to each page's rows of the head
  uint32_t rows[2][2];  // rows of each page that hold visible keys, a bit each
  int key0;             // its first key
  int last;             // no tile follows
};

struct Ctl {
  uint64_t bars[kBars];
  TileInfo tiles[kTileRing];
  Share share;
  Seg segs[kSegRing];
  uint32_t tmem;
  uint32_t abort;
};

template <int D>
__global__ __launch_bounds__(kThreads, 1) void tiles_kernel(const AttnArgs a) {
  constexpr int kHalves = D / 64;                   // 64-element column blocks of a row
  constexpr uint32_t kQHalf = kHalfRows * 128;      // bytes of one column block of 128 rows
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = sq + q_bytes(D), sv = sk + kStages * kv_bytes(D);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  volatile uint32_t* abort = &ctl.abort;
  const auto bar = [&](int i) { return smem_addr(&ctl.bars[i]); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // joins as CTAs end
  locate_share(a, ctl.share);
  const Share& share = ctl.share;
  if (share.s0 >= share.s1) {
    if (tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), arrivals(i));
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

  if (warp >= kSoftWarp) {
    // ------------------------------------------------------------- softmax
    set_regs_up<kSoftRegs>();
    const int half = (warp - kSoftWarp) / 4, rl = tid % kHalfRows;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + lanes + half * 128;
    const uint32_t to = tmem + lanes + 256 + half * D;
    uint32_t n = 0, n_half = 0;  // tiles so far: of the CTA, of this half
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = __all_sync(kFull, wait_bar(bar(kSegFull + i % kSegRing), i / kSegRing & 1u, abort));
      if (!ok) break;
      const Seg& seg = ctl.segs[i % kSegRing];
      const Item& m = seg.m;
      const int nt = seg.t1 - seg.t0;
      const bool more = seg.more != 0;
      if (half == 1 && m.rows <= kHalfRows) {  // no rows in this half
        n += nt;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSegEmpty + i % kSegRing));
        if (!more) break;
        continue;
      }
      const bool whole = seg.whole != 0;
      const int part = seg.part;
      const int r = m.row0 + half * kHalfRows + rl;  // row of the sequence
      const bool live_row = r < m.row0 + m.rows;
      const int tok = m.q0 + r / a.G, h = seg.head * a.G + r % a.G;
      const bool live = live_row && tok >= 0 && tok < a.T;
      // ---- the warp's rows of Q into shared memory, kRowLanes lanes to a row,
      // and scaled there by powers of two.  (Loops that stay loops: what runs
      // once per item is cold code, and its fetch costs more than its steps.)
      float fac;
      {
        constexpr int kRowLanes = D / 8, kPer = 32 / kRowLanes;
        const int64_t own = live ? tok * a.q_ts + h * a.q_hs : -1;  // of the lane's row
        const int c = lane % kRowLanes, row = warp % 4 * 32 + lane / kRowLanes;
        const uint32_t dst = sq + half * kHalves * kQHalf + c / 8 * kQHalf + row * 128;
#pragma unroll 1
        for (int i = 0; i < kRowLanes; ++i) {
          const int64_t off = __shfl_sync(kFull, own, i * kPer + lane / kRowLanes);
          const uint32_t at = dst + i * kPer * 128 + ((c ^ (row + i * kPer)) & 7) * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at),
                       "l"(a.q + (off < 0 ? 0 : off + c * 8)), "r"(off < 0 ? 0 : 16)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        // the lane's own row; magnitudes compare as their bits do
        const uint32_t src = sq + half * kHalves * kQHalf + rl * 128;
        const auto chunk = [&](int k) {
          return src + k / 8 * kQHalf + ((k ^ rl) & 7) * 16;
        };
        uint32_t top = 0;
#pragma unroll 4
        for (int k = 0; k < kRowLanes; ++k) {
          uint32_t u[4];
          lds128(chunk(k), u);
#pragma unroll
          for (int j = 0; j < 4; ++j) top = __vmaxu2(top, u[j] & 0x7fff7fffu);
        }
        const float2 both = unpack16(a.half, top);
        // the largest * 2^(141 - b) lies in [2^14, 2^15) for its biased exponent b
        const uint32_t b = max(__float_as_uint(fmaxf(both.x, both.y)) >> 23, 15u);
        const float up = __uint_as_float((268u - b) << 23 | (uint32_t)(a.scale_log2 < 0.0f) << 31);
        fac = fabsf(a.scale_log2) * __uint_as_float((b - 14u) << 23);
#pragma unroll 4
        for (int k = 0; k < kRowLanes; ++k) {
          uint32_t u[4];
          lds128(chunk(k), u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16(a.half, u[j]);
            u[j] = pack16<true>(f.x * up, f.y * up);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(chunk(k)), "r"(u[0]),
                       "r"(u[1]), "r"(u[2]), "r"(u[3])
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQFull + half));
      }
      const int pos = live_row ? m.first + r / a.G : -1;
      // positions of the warp's first and last row
      const int w0 = m.row0 + half * kHalfRows + warp % 4 * 32;
      const int pos_lo = m.first + w0 / a.G;
      const int pos_hi = m.first + min(w0 + 31, m.row0 + m.rows - 1) / a.G;
      const bool idle = w0 >= m.row0 + m.rows;  // no row: keep the barriers going
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSegEmpty + i % kSegRing));
      float mm = -INFINITY, MM = -INFINITY, l = 0.0f;
      const int lo_key = a.window > 0 ? pos - a.window + 1 : -(1 << 30);
      for (int t = 0; t < nt; ++t, ++n, ++n_half) {
        ok = __all_sync(kFull, wait_bar(bar(kSFull + half), n_half & 1, abort));
        if (!ok) break;
        fence_after();
        if (!idle) {
          const TileInfo& info = ctl.tiles[n % kTileRing];
          const float4 sc = lds_f4(smem_addr(info.scale));
          int kb;
          asm volatile("ld.shared.s32 %0, [%1];" : "=r"(kb) : "r"(smem_addr(&info.key0)));
          const bool full = fminf(sc.z, sc.w) >= 0.0f && kb + kTile <= pos_lo + 1 &&
                            (a.window <= 0 || kb > pos_hi - a.window || kb + kTile <= a.sinks);
          // a factor of zero would make a masked score NaN
          const float c0 = fmaxf(fac * sc.x, 0x1p-100f), c1 = fmaxf(fac * sc.y, 0x1p-100f);
          const float e0 = log2_scale(sc.z), e1 = log2_scale(sc.w);
          float s[kPage];  // one page's scores at a time
          const auto load = [&](int page) {
            tmem_ld32(ts + page * kPage, s);
            tmem_ld32(ts + page * kPage + 32, s + 32);
            tmem_wait_ld();
            if (__builtin_expect(!full, 0)) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int from = kb + page * kPage + w * 32;
                uint32_t on = sees(pos - from, lo_key - from, a.sinks - from);
                if ((page ? sc.w : sc.z) < 0.0f) on = 0;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(on >> e & 1u)) s[w * 32 + e] = -INFINITY;
              }
            }
          };
          load(1);
          const float x1 = fmaxf(top32(s), top32(s + 32)) * c1;
          load(0);
          const float x0 = fmaxf(top32(s), top32(s + 32)) * c0;
          const float m1 = fmaxf(mm, fmaxf(x0, x1));
          const float M1 = fmaxf(x0 + e0, x1 + e1);
          // ---- O's reference, moved seldom
          const bool move = M1 > MM + kSlack || (MM == -INFINITY && M1 != -INFINITY);
          if (__builtin_expect(__any_sync(kFull, move), 0)) {
            const float al = move ? exp2_approx(MM - M1) : 1.0f;
            if (move) MM = M1;
            if (t > 0) {
              ok = __all_sync(kFull, wait_bar(bar(kODone + half), (n_half - 1) & 1, abort));
              if (!ok) break;
              fence_after();
              // few columns at a time: s stays in registers
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= al;
                tmem_st16(to + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          const float mz = or_zero(m1), Mz = or_zero(MM);
          l *= exp2_approx(mm - mz);
          mm = m1;
#pragma unroll
          for (int page = 0; page < 2; ++page) {
            const float c = page ? c1 : c0;
            const float ref = Mz - (page ? e1 : e0) - kShift;
            if (page) load(1);
            const bool far = ref + kShift - mz > kFar;
            const bool any_far = __any_sync(kFull, far);
            float own = 0.0f, b0 = 0.0f, b1 = 0.0f, b2 = 0.0f, b3 = 0.0f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float* v = s + w * 32;
              if (__builtin_expect(any_far, 0)) {
#pragma unroll
                for (int q = 0; q < 32; ++q) own += exp2_approx(fmaf(v[q], c, -mz));
              }
              uint32_t p[16];
#pragma unroll
              for (int q = 0; q < 32; q += 4) {
                float y0, y1, y2, y3;
                fma2s(y0, y1, v[q], v[q + 1], c, -ref);
                fma2s(y2, y3, v[q + 2], v[q + 3], c, -ref);
                y0 = exp2_approx(y0);
                y1 = exp2_approx(y1);
                y2 = exp2_approx(y2);
                y3 = exp2_approx(y3);
                sum2(b0, b1, b0, b1, y0, y1);
                sum2(b2, b3, b2, b3, y2, y3);
                p[q / 2] = pack16<true>(y0, y1);
                p[q / 2 + 1] = pack16<true>(y2, y3);
              }
              tmem_st16(ts + page * 32 + w * 16, p);
            }
            const float moved = (b0 + b1 + (b2 + b3)) * exp2_approx(ref - mz);
            l += far ? own : moved;
          }
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + half));
      }
      // ---- the output row
      if (ok) ok = __all_sync(kFull, wait_bar(bar(kODone + half), (n_half - 1) & 1, abort));
      if (ok && !idle) {
        fence_after();
        const bool some = mm != -INFINITY;
        const float inv = some ? __frcp_rn(l) : 0.0f;
        // 2^(M-m-10) in two halves: with values near 2^-126 it is 0 itself
        const float f = some ? exp2_approx(0.5f * (MM - mm - kShift)) : 0.0f;
        const float lse2 = some ? mm + __log2f(l) : -INFINITY;
        const int64_t orow = (int64_t)tok * a.Hq + h;
        const int64_t prow = (int64_t)part * kItemRows + half * kHalfRows + rl;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tmem_ld32(to + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = some ? o[i] * (inv * f) * f : 0.0f;
          if (!live) {
          } else if (!whole) {
            float4* dst = reinterpret_cast<float4*>(a.part_out + prow * D + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack16(a.half, o[8 * i], o[8 * i + 1]),
                                  pack16(a.half, o[8 * i + 2], o[8 * i + 3]),
                                  pack16(a.half, o[8 * i + 4], o[8 * i + 5]),
                                  pack16(a.half, o[8 * i + 6], o[8 * i + 7]));
          }
        }
        if (live) {
          if (!whole)
            a.part_lse[prow] = lse2;
          else if (a.lse)
            a.lse[orow] = lse2 * kLn2;
        }
      }
      if (!more) break;
    }
  } else if (warp >= kConvWarp) {
    // ---------------------------------------------------------- converters
    set_regs_down<kConvRegs>();
    const int cw = warp - kConvWarp;
    // the tile whose codes are loaded next
    int64_t off[2];
    uint32_t rows[2][2];
    bool last = false;
    const auto look = [&](uint32_t n) {
      const bool ok = 0 != __all_sync(kFull, wait_bar(bar(kTileFull + n % kTileRing),
                                                      n / kTileRing & 1u, abort));
      const TileInfo& info = ctl.tiles[n % kTileRing];
      last = info.last != 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        off[k] = info.off[k];
        rows[k][0] = ok ? info.rows[k][0] : 0u;
        rows[k][1] = ok ? info.rows[k][1] : 0u;
      }
      return ok;
    };
    // Keys: a row of codes is kRowLanes lanes of 16 bytes; load i of a lane is
    // row key + 4 * kRows * i.
    constexpr int kRowLanes = D / 16, kRows = 32 / kRowLanes, kLoads = kTile / (4 * kRows);
    const int key = cw * kRows + lane / kRowLanes;
    const int c = lane % kRowLanes;  // d 16c .. 16c + 15
    uint4 kreg[kLoads];
    const auto load_k = [&]() {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = i / (kLoads / 2), step = i % (kLoads / 2) * (4 * kRows);
        kreg[i] = make_uint4(0, 0, 0, 0);
        if (rows[k][step / 32] & 1u << (key + step % 32))
          kreg[i] = ld_stream(a.kc + off[k] + (key + step) * D + c * 16);
      }
    };
    // the lanes of the second column block store their upper half first: the
    // two blocks lie on the same banks
    const int flip = c / 4;
    const uint32_t atk = sk + c / 4 * (kTile * 128) + key * 128;
    const uint32_t at0 = atk + ((c % 4 * 2 + flip) ^ (key & 7)) * 16;
    const uint32_t at1 = atk + ((c % 4 * 2 + 1 - flip) ^ (key & 7)) * 16;
    // Values: a step covers a page's 64 keys (16 lanes x 4 rows) and 32 d (2
    // lanes x 16).
    constexpr int kSteps = D / 64;
    const int d0 = (D == 128 ? cw : cw % 2) * 32 + lane / 16 * 16;
    const int q = lane % 16;  // keys 4q .. 4q + 3: 8 bytes of a row of d
    uint4 vreg[kSteps][4];
    const auto page_of = [&](int i) { return D == 128 ? i : cw / 2; };
    const auto load_v = [&]() {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint8_t* src = a.vc + (page_of(i) ? off[1] : off[0]) + q * 4 * D + d0;
        const uint32_t on0 = page_of(i) ? rows[1][0] : rows[0][0];
        const uint32_t on1 = page_of(i) ? rows[1][1] : rows[0][1];
        const uint32_t on = (q < 8 ? on0 : on1) >> (q % 8 * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          vreg[i][j] = make_uint4(0, 0, 0, 0);
          if (on >> j & 1u) vreg[i][j] = ld_stream(src + j * D);
        }
      }
    };
    const uint32_t atv = sv + d0 * 128 + q / 2 * 16 + q % 2 * 8;

    bool ok = look(0);
    load_k();
    for (uint32_t n = 0; ok; ++n) {
      const int stage = n % kStages;
      const bool done = last;
      load_v();
      if (n >= kStages)
        ok = __all_sync(kFull, wait_bar(bar(kKEmpty + stage), (n / kStages + 1) & 1u, abort));
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t u[4] = {kreg[i].x, kreg[i].y, kreg[i].z, kreg[i].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) e4m3x4_to_f16x2(u[j], o[2 * j], o[2 * j + 1]);
        const uint32_t to = stage * kv_bytes(D) + i * (4 * kRows * 128);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at0 + to),
                     "r"(flip ? o[4] : o[0]), "r"(flip ? o[5] : o[1]), "r"(flip ? o[6] : o[2]),
                     "r"(flip ? o[7] : o[3])
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at1 + to),
                     "r"(flip ? o[0] : o[4]), "r"(flip ? o[1] : o[5]), "r"(flip ? o[2] : o[6]),
                     "r"(flip ? o[3] : o[7])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull + stage));
      if (!done) {
        ok = look(n + 1);
        load_k();
      }
      if (ok && n >= kStages)
        ok = __all_sync(kFull, wait_bar(bar(kVEmpty + stage), (n / kStages + 1) & 1u, abort));
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t blk = atv + stage * kv_bytes(D) + page_of(i) * (D * 128);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // d0 + 4e ..
          const uint32_t r0 = (&vreg[i][0].x)[e], r1 = (&vreg[i][1].x)[e];
          const uint32_t r2 = (&vreg[i][2].x)[e], r3 = (&vreg[i][3].x)[e];
          // byte pairs (key 0, key 1) and (2, 3) of four d
          uint32_t lo[4], hi[4];
          e4m3x4_to_f16x2(prmt(r0, r1, 0x5140u), lo[0], lo[1]);
          e4m3x4_to_f16x2(prmt(r0, r1, 0x7362u), lo[2], lo[3]);
          e4m3x4_to_f16x2(prmt(r2, r3, 0x5140u), hi[0], hi[1]);
          e4m3x4_to_f16x2(prmt(r2, r3, 0x7362u), hi[2], hi[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 4 * e + j;  // of the swizzle: d0 is a multiple of 16
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"((blk ^ (d % 8 * 16)) + d * 128),
                         "r"(lo[j]), "r"(hi[j])
                         : "memory");
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kVFull + stage));
      if (done) break;
    }
  } else {
    set_regs_down<kMmaRegs>();
  }
  if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t kQkDesc = f16_idesc(kTile), kPvDesc = f16_idesc(D);
    // a descriptor's address field moves by (bytes >> 4)
    const uint64_t dq = sw128_desc(sq), dk = sw128_desc(sk), dv = sw128_desc(sv);
    const uint32_t elected = elect_one();
    const auto issue_s = [&](int half, int stage) {
      const uint64_t qa = dq + half * (kHalves * kQHalf >> 4), kb = dk + stage * (kv_bytes(D) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(elected, tmem + half * 128, qa + (k / 4 * (kQHalf >> 4) + k % 4 * 2),
               kb + (k / 4 * (kTile * 128 >> 4) + k % 4 * 2), kQkDesc, k > 0);
      mma_commit(elected, bar(kSFull + half));
    };
    const auto issue_o = [&](int half, int stage, bool first) {
      const uint64_t vb = dv + stage * (kv_bytes(D) >> 4);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(elected, tmem + 256 + half * D, tmem + half * 128 + k * 8,
               vb + (k / 4 * (D * 128 >> 4) + k % 4 * 2), kPvDesc, !first || k > 0);
      mma_commit(elected, bar(kODone + half));
    };
    const auto release = [&](int i) { mma_commit(elected, bar(i)); };
    const auto wait = [&](int i, uint32_t parity) {
      return __all_sync(kFull, wait_bar(bar(i), parity, abort)) != 0;
    };
    bool ok = true;
    uint32_t n = 0, n_a = 0, n_b = 0;  // tiles so far: of the CTA, of each half
    uint32_t q_a = 0, q_b = 0;         // segments so far, of each half
    for (uint32_t i = 0; ok; ++i) {
      ok = wait(kSegFull + i % kSegRing, i / kSegRing & 1u);
      if (!ok) break;
      const Seg& seg = ctl.segs[i % kSegRing];
      const int nt = seg.t1 - seg.t0;
      const int halves = seg.m.rows > kHalfRows ? 2 : 1;
      const bool more = seg.more != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSegEmpty + i % kSegRing));
      ok = wait(kKFull + n % kStages, n / kStages & 1u);
      for (int h = 0; h < halves && ok; ++h) {
        ok = wait(kQFull + h, (h ? q_b : q_a) & 1u);
        if (!ok) break;
        fence_after();
        issue_s(h, n % kStages);
      }
      ++q_a;
      q_b += halves - 1;
      if (ok) release(kKEmpty + n % kStages);
      for (int t = 0; t < nt && ok; ++t, ++n) {
        const int stage = n % kStages, next = (n + 1) % kStages;
        ok = wait(kVFull + stage, n / kStages & 1u);
        for (int h = 0; h < halves && ok; ++h) {
          ok = wait(kPFull + h, (h ? n_b : n_a) & 1u);
          if (!ok) break;
          fence_after();
          issue_o(h, stage, t == 0);
          if (t + 1 < nt) {
            if (h == 0) ok = wait(kKFull + next, (n + 1) / kStages & 1u);
            if (!ok) break;
            issue_s(h, next);
          }
        }
        if (!ok) break;
        // both halves have their probabilities, and V is converted
        if (lane == 0) mbar_arrive(bar(kTileFree + n % kTileRing));
        ++n_a;
        n_b += halves - 1;
        release(kVEmpty + stage);
        if (t + 1 < nt) release(kKEmpty + next);
      }
      if (!more) break;
    }
  } else if (warp == kSegWarp) {
    // ------------------------------------------------------ work list
    int b = share.b, rc = share.rc, head = share.head, t0 = share.off;
    int64_t at = share.s0;
    int4 cut = make_int4(0, 0, 0, 0);
    uint32_t n = 0;  // tiles described
    // (testing hook, see fp4idx_test_withhold_next: a tile that is not)
    const int held = blockIdx.x == 0 ? a.withhold : -1;
    for (uint32_t i = 0; at < share.s1; ++i) {
      if (i >= kSegRing &&
          !__all_sync(kFull, wait_bar(bar(kSegEmpty + i % kSegRing), (i / kSegRing + 1) & 1u,
                                      abort)))
        break;
      Seg sg;
      item_of(a, b, rc, sg.m);
      sg.b = b;
      sg.head = head;
      sg.t0 = t0;
      sg.t1 = (int)min((int64_t)sg.m.nt, t0 + (share.s1 - at));
      sg.whole = t0 == 0 && sg.t1 == sg.m.nt;
      sg.part = 2 * blockIdx.x + (t0 == 0 && i > 0 ? 1 : 0);
      if (!sg.whole && t0 == 0)  // the first fragment of a cut item
        cut = make_int4(b, rc, head,
                        (cta_of(at + sg.m.nt - 1, share) - (int)blockIdx.x + 1) * 2 +
                            (sg.part & 1));
      at += sg.t1 - t0;
      sg.more = at < share.s1;
      if (lane == 0) {
        ctl.segs[i % kSegRing] = sg;
        mbar_arrive(bar(kSegFull + i % kSegRing));
      }
      // its tiles, four at a time, a lane each
      bool ok = true;
      for (int t = sg.t0; t < sg.t1 && ok; t += 4) {
        const int k = min(sg.t1 - t, 4);
        TileInfo info;
        if (lane < k) {
          info.key0 = key_of_tile(sg.m, t + lane);
          info.last = !sg.more && t + lane + 1 == sg.t1;
          const int32_t* row = a.table + b * a.tstride + info.key0 / kPage;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int from = info.key0 + e * kPage;
#pragma unroll
            for (int w = 0; w < 2; ++w)
              info.rows[e][w] = sees(sg.m.hi - 1 - from - 32 * w, sg.m.lo - from - 32 * w,
                                     a.sinks - from - 32 * w);
            const bool seen = (info.rows[e][0] | info.rows[e][1]) != 0;
            int page = seen ? __ldg(row + e) : -1;
            info.scale[e] = 1.0f;
            info.scale[2 + e] = -1.0f;
            if (page >= 0 && page < a.num_blocks) {
              info.scale[e] = a.ks[page * a.sstride + head];
              info.scale[2 + e] = fabsf(a.vs[page * a.sstride + head]);
            } else {
              if (seen) flag_error(a.err, FP4IDX_ERRFLAG_PAGE);
              info.rows[e][0] = info.rows[e][1] = page = 0;
            }
            info.off[e] = page * a.cstride + (int64_t)head * kPage * D;
          }
        }
        for (int e = 0; e < k && ok; ++e, ++n) {
          if (n >= kTileRing)
            ok = __all_sync(kFull, wait_bar(bar(kTileFree + n % kTileRing),
                                            (n / kTileRing + 1) & 1u, abort));
          if (ok && lane == e && (int)n != held) {
            ctl.tiles[n % kTileRing] = info;
            mbar_arrive(bar(kTileFull + n % kTileRing));
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      t0 = 0;
      if (++head == a.Hkv && sg.more) {
        head = 0;
        Item it;
        do {
          if (++rc == a.rc_max) {
            rc = 0;
            ++b;
          }
        } while (!item_of(a, b, rc, it));
      }
    }
    if (lane == 0) a.cuts[blockIdx.x] = cut;
  }

  __syncwarp();
  fence_before();
  __syncthreads();
  if (*abort) {
    // MMAs in flight land before TMEM and shared memory are released.  A commit
    // stands for its own lane's MMAs: the lane that was elected to issue them.
    if (warp == kMmaWarp && elect_one()) {
      flag_error(a.err, FP4IDX_ERRFLAG_TIMEOUT);
      const uint32_t b = bar(kQFull);  // re-used: one arrival by the commit
      asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(b) : "memory");
      mbar_init(b, 1);
      fence_mbar_init();
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
// 2^(lse - max), in the order of the CTAs, applied in two halves (a part of weight
// 2^-126 counts where its values are as much larger).  Blocks (CTA whose share
// begins the item, 32 of its rows), four rows a warp.
template <int D>
__global__ __launch_bounds__(256) void join_tiles_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kBlocks = kItemRows / 32;
  const int cta = blockIdx.x / kBlocks;
  const int4 cut = a.cuts[cta];
  const int n = cut.w / 2;
  if (n < 2) return;
  Item m;
  item_of(a, cut.x, cut.y, m);
  const int lane = threadIdx.x % 32;
  const auto slot = [&](int f) { return (int64_t)2 * (cta + f) + (f == 0 ? cut.w & 1 : 0); };
  constexpr int kV = D / 32, kRows = 4;
  const int r0 = blockIdx.x % kBlocks * 32 + threadIdx.x / 32 * kRows;
  if (r0 >= m.rows) return;
  float top[kRows], den[kRows], o[kRows][kV];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    top[k] = -INFINITY;
    den[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) o[k][j] = 0.0f;
  }
#pragma unroll 2
  for (int f = 0; f < n; ++f)
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (r0 + k < m.rows) top[k] = fmaxf(top[k], a.part_lse[slot(f) * kItemRows + r0 + k]);
#pragma unroll 2
  for (int f = 0; f < n; ++f)
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (r0 + k >= m.rows || top[k] == -INFINITY) continue;
      const int64_t row = slot(f) * kItemRows + r0 + k;
      const float half = exp2_approx(0.5f * (a.part_lse[row] - top[k]));
      den[k] = fmaf(half, half, den[k]);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        o[k][j] = fmaf(a.part_out[row * D + lane * kV + j] * half, half, o[k][j]);
    }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = m.row0 + r0 + k;
    const int tok = m.q0 + r / a.G;
    if (r0 + k >= m.rows || tok < 0 || tok >= a.T) continue;
    const bool some = top[k] != -INFINITY;
    const float inv = some ? __frcp_rn(den[k]) : 0.0f;
    const int64_t orow = (int64_t)tok * a.Hq + cut.z * a.G + r % a.G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + lane * kV);
#pragma unroll
    for (int j = 0; j < kV; j += 2)
      dst[j / 2] = pack16(a.half, o[k][j] * inv, o[k][j + 1] * inv);
    if (a.lse && lane == 0)
      a.lse[orow] = some ? (top[k] + __log2f(den[k])) * kLn2 : -INFINITY;
  }
}

template <int D>
fp4idx_status launch_d(const AttnArgs& a, int grid, cudaStream_t stream) {
  static SmemOnce once;
  if (!once.set(tiles_kernel<D>, smem_bytes(D))) return FP4IDX_ERR_CUDA;
  if (launch_kernel(tiles_kernel<D>, (unsigned)grid, kThreads, smem_bytes(D), stream, a) !=
      cudaSuccess)
    return FP4IDX_ERR_CUDA;
  return launch_after(join_tiles_kernel<D>, (unsigned)(grid * (kItemRows / 32)), 256, stream, a) ==
                 cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}

}  // namespace

fp4idx_status launch_tiles(const AttnArgs& a, int head_dim, int grid, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128>(a, grid, stream) : launch_d<64>(a, grid, stream);
}

}  // namespace fp4idx_impl
