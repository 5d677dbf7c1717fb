// fp4idx_attn_rows.cu -- attention over the 8-bit cache for few query rows per
// key head: single tokens, a handful of drafted tokens, and selected tokens
// (fp4idx_sparse_attention_fp8).  The operations are defined in
// include/fp4idx_attention.h.
//
// What bounds it.  Every visible key and value byte is read once and used for
// the R = 8, 16 or 32 query rows of an item, so the bound is the memory's
// bandwidth; below it lies the latency of a warp's chain (fragments, products,
// softmax, products).  Eight warps compute, each alone on 32-key pieces of the
// cache with its own running softmax and output sums in registers; they meet
// only at the end of an item.  Eight others each fill the ring of one of them
// with asynchronous copies: the walk over pages or selected entries and the
// copies' issue took a computing warp 950 to 1,900 cycles a piece, next to
// 1,450 to 2,500 of arithmetic.  Measured: 64 single tokens, 8 key heads of
// 128, contexts up to 32,768, 428 to 448 us box to box (87 to 91% of the copy
// bandwidth); 32 rows, 192 items of 65 tiles, heads of 64, 76 us (a piece takes
// a warp 3,800 cycles); 64 tokens of 2,048 selected keys each 69 us, 1,021 over
// one key head 134.
//
// Mathematics.  Codes are E4M3, exact in fp16; a query row is scaled by a
// power of two, its largest element into [2^14, 2^15).  That is exact for bf16
// elements down to 2^-31 of the largest and for fp16 ones down to 2^-28 (8 and 11
// bits above fp16's least step of 2^-24); smaller ones are rounded by 2^-39 of
// the largest at most.  The products of the score are exact and their sum is
// fp32.  With the page's scales ks and vs (powers of two), in units of
// log2:  s = sum(q k) * ks * scale * log2(e).  The running softmax has two
// references: m, of the sum l = sum 2^(s-m), and M, of the output sums,
//   p = 2^(s + log2 vs - M + 10) in fp16,   O = sum p * code,
// near the largest s and the largest contribution s + log2 vs.  M follows only
// when a contribution exceeds it by more than 4, m when a score exceeds it by
// 60: then p <= 2^14, and most pieces need no exchange between lanes and no
// rescaling.  p is rounded to 2^-11 of itself, or 2^-35 of the largest
// contribution, however far the pages' scales lie apart.  l is summed from the
// same exponentials, moved by the references' difference, as long as that and
// the spread of a piece's scales are small; else it takes its own.
//   out = O * 2^(M - m - 10) / l,   lse = m + log2 l.
//
// Layout.  The scores are computed transposed, S^T = K Q^T, by
// mma.m16n8k16 with 16 keys and 8 query rows: the keys fill the M side
// whatever the number of rows.  Keys are read from shared memory with
// ldmatrix and converted in registers; which byte of a row meets which k slot
// is free as long as the queries use the same order.  V^T is read with
// ldmatrix.trans as pairs of bytes, whose halves belong to neighbouring d:
// they go to the rows g and g + 8 of the fragment.  P^T as the second
// product's operand is the transpose of the scores' fragment: movmatrix.
//
// Work split.  The items (sequence, key head, R rows) and their 64-key tiles
// form one list, cut into equal shares, one per CTA, from the lengths alone.
// An item cut by a share's end leaves normalised partial outputs with their
// lse, joined by a second kernel in a fixed order.

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kWarps = 8;  // that compute; as many copy
constexpr int kThreads = 2 * kWarps * 32;
// Registers of a thread that computes; one that copies has 256 less those (the
// launch's 128 each, moved).  The least that spill nothing, or next to it: what
// is spilled goes past the little L1 that the rings leave.
__host__ __device__ constexpr int compute_regs(int D, int NT, bool sparse) {
  if (D == 64) return NT == 4 ? 200 : 152;
  return NT == 1 ? 152 : sparse ? 184 : 192;
}
constexpr int kPage = FP4IDX_KV_BLOCK;
constexpr int kSub = 32;  // keys of a piece: half a page
constexpr float kShift = 10.0f, kSlack = 4.0f, kFar = 60.0f, kSpread = 40.0f;

__host__ __device__ constexpr int stages(int D) { return D == 128 ? 3 : 6; }
// keys, values, 2 x 32 scales, the mask of visible keys
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * kSub * D + 256 + 16; }
__host__ __device__ constexpr int q_row_bytes(int D) { return 2 * D + 32; }

// Where the queries' fragments would not fit the registers.
__host__ __device__ constexpr bool q_in_smem(int D, int NT) { return D * NT > 128; }

__host__ __device__ constexpr int smem_bytes(int D, int NT) {
  return kWarps * stages(D) * stage_bytes(D) + kWarps * 8 * NT * 3 * 4 +
         (q_in_smem(D, NT) ? 8 * NT * q_row_bytes(D) : 0) + kWarps * stages(D) * 16;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Arrives at bar once this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Waits for a phase; false when a warp has given up, or after 1 s.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  unsigned long long t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
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

__device__ __forceinline__ void compute_sync() {  // the warps that compute
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float max_g(float v) {  // over the lanes of one column pair
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 16));
}

__device__ __forceinline__ float sum_g(float v) {
  v += __shfl_xor_sync(kFull, v, 4);
  v += __shfl_xor_sync(kFull, v, 8);
  return v + __shfl_xor_sync(kFull, v, 16);
}

__device__ __forceinline__ float or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// One sequence (dense) or query token (sparse): its rows, its keys' tiles.
struct Seq {
  int q0;      // first query token
  int n;       // query tokens
  int first;   // position of the first (dense)
  int lo, hi;  // keys that any of them sees: [lo, hi) and [0, sinks)
  int ts, tl;  // tiles: 0 .. ts-1, then tl ..
  int nt;      // tiles in all, at least one
  int rcs;     // row chunks
  int items;   // key heads x row chunks
};

template <bool kSparse>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq m;
  if constexpr (kSparse) {
    m.q0 = b;
    m.n = 1;
    m.first = m.lo = m.ts = m.tl = 0;
    m.hi = a.nsel;
    m.nt = (a.nsel + kPage - 1) / kPage;
  } else {
    const int ctx = min(max(__ldg(a.ctx + b), 0), a.max_context);
    int full = a.max_q;
    m.q0 = b * a.max_q;
    if (a.starts) {
      m.q0 = __ldg(a.starts + b);
      full = max(__ldg(a.starts + b + 1) - m.q0, 0);
    }
    m.n = min(full, a.max_q);
    m.first = ctx - full;
    m.hi = max(min(ctx, m.first + m.n), 0);
    m.lo = a.window > 0 ? min(max(m.first - a.window + 1, 0), m.hi) : 0;
    m.tl = m.lo / kPage;
    m.ts = a.window > 0 ? min((a.sinks + kPage - 1) / kPage, m.tl) : 0;
    m.nt = m.ts + (m.hi + kPage - 1) / kPage - m.tl;
  }
  m.nt = max(m.nt, 1);
  m.rcs = (m.n * a.G + a.R - 1) / a.R;
  m.items = a.Hkv * m.rcs;
  return m;
}

// A place in the list of items.
template <bool kSparse>
struct Cursor {
  int b, it;
  int64_t begin;  // the item's first unit
  bool cut;       // units are tiles, or items as a whole (dense)
  Seq m;

  __device__ __forceinline__ bool cuts(const AttnArgs& a) const {
    return kSparse ? a.split != 0 : cut;
  }
  __device__ __forceinline__ int units(const AttnArgs& a) const { return cuts(a) ? m.nt : 1; }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    begin += units(a);
    if (++it == m.items) {
      it = 0;
      do {
        if (++b >= a.batch) return;
        m = seq_of<kSparse>(a, b);
      } while (m.items == 0);
    }
  }
};

// The units of the whole list, this CTA's share [s0, s1) of them and the
// cursor at s0.  Dense: a prefix sum over the sequences, by the whole CTA, and
// the lengths decide whether items are cut after all, where the caller's bound
// on them let it seem worth it (a.split).
template <bool kSparse>
__device__ __forceinline__ int64_t locate_share(const AttnArgs& a, Cursor<kSparse>& cur,
                                                int64_t& s0, int64_t& s1) {
  cur.cut = a.split != 0;
  const int cta = blockIdx.x;
  int64_t total = 0;
  // no CTA's share is empty but those behind the last unit's
  const auto share = [&]() {
    const int64_t grid = min((int64_t)gridDim.x, total);
    s0 = cta < grid ? total * cta / grid : 0;
    s1 = cta < grid ? total * (cta + 1) / grid : 0;
  };
  if constexpr (kSparse) {
    cur.m = seq_of<true>(a, 0);
    const int64_t per = (int64_t)cur.m.items * cur.units(a);
    total = per * a.batch;
    share();
    if (s0 >= s1) return total;
    cur.b = (int)(s0 / per);
    cur.begin = cur.b * per;
    cur.m = seq_of<true>(a, cur.b);
  } else {
    __shared__ int64_t part[kThreads / 32];
    __shared__ int2 part_items[kThreads / 32];  // items; the longest one's tiles
    __shared__ int64_t found_begin;
    __shared__ int found_b;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int each = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * each, a.batch), b1 = min(b0 + each, a.batch);
    int64_t own = 0;
    int own_items = 0, most = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq m = seq_of<false>(a, b);
      own += (int64_t)m.items * m.nt;
      own_items += m.items;
      if (m.items > 0) most = max(most, m.nt);
    }
    if (a.split) {
      most = __reduce_max_sync(kFull, most);
      const int items = __reduce_add_sync(kFull, own_items);
      int64_t sum = own;
      for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(kFull, sum, d);
      if (lane == 0) {
        part[warp] = sum;
        part_items[warp] = make_int2(items, most);
      }
      __syncthreads();
      int n = 0;
      int64_t tiles = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        tiles += part[w];
        n += part_items[w].x;
        most = max(most, part_items[w].y);
      }
      cur.cut = worth_cutting(n, tiles, most, a.R, gridDim.x, false);
      __syncthreads();
    }
    if (!cur.cut) own = own_items;
    int64_t incl = own;
    for (int d = 1; d < 32; d *= 2) {
      const int64_t o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += part[w];
      total += part[w];
    }
    share();
    const int64_t from = base + incl - own;
    if (s0 < s1 && from <= s0 && s0 < from + own) {
      int64_t at = from;
      int b = b0;
      for (;; ++b) {
        const Seq m = seq_of<false>(a, b);
        const int64_t u = (int64_t)m.items * (cur.cut ? m.nt : 1);
        if (s0 < at + u) break;
        at += u;
      }
      found_b = b;
      found_begin = at;
    }
    __syncthreads();
    if (s0 >= s1) return total;
    cur.b = found_b;
    cur.begin = found_begin;
    cur.m = seq_of<false>(a, cur.b);
  }
  const int u = cur.units(a);
  cur.it = (int)((s0 - cur.begin) / u);
  cur.begin += (int64_t)cur.it * u;
  return total;
}

// The CTA whose share holds unit x: the last c with total * c / grid <= x.
__device__ __forceinline__ int cta_of(int64_t x, int64_t total) {
  const int64_t grid = min((int64_t)gridDim.x, total);
  return (int)(((x + 1) * grid - 1) / total);
}

// The copies into one ring: a cursor ahead of the arithmetic.  Dense: a
// piece's page is looked up one piece before its copies.  Sparse: its entries
// two pieces before, their pages one.
template <int D, bool kSparse>
struct Producer {
  Cursor<kSparse> pc;
  int64_t at;      // end of the open segment's units
  int t0, xb, xe;  // the segment's first tile; its pieces [xb, xe) of the CTA's list
  int x;           // this warp's next piece
  // the next piece to copy
  bool have, ok;
  int key0, page, head, lo, hi, pos;
  // sparse: the one after it
  bool f_have;
  int f_idx, f_b, f_head;

  __device__ __forceinline__ void open(const AttnArgs& a, int64_t s1) {
    const int u = pc.units(a);
    const int64_t end = min(s1, pc.begin + u);
    t0 = pc.cuts(a) ? (int)(at - pc.begin) : 0;
    xe = xb + 2 * (pc.cuts(a) ? (int)(end - at) : pc.m.nt);
    at = end;
  }
  __device__ __forceinline__ bool seek(const AttnArgs& a, int64_t s1) {
    while (x >= xe) {
      if (at >= s1) return false;
      pc.next(a);
      xb = xe;
      open(a, s1);
    }
    return true;
  }
  __device__ __forceinline__ void fetch(const AttnArgs& a, int64_t s1, int lane) {
    f_have = seek(a, s1);
    f_idx = -1;
    if (!f_have) return;
    const int k = (t0 * 2 + (x - xb)) * kSub + lane;
    f_b = pc.b;
    f_head = pc.it / pc.m.rcs;
    if (k < a.nsel) f_idx = __ldg(a.indices + (int64_t)f_b * a.idx_stride + k);
    x += kWarps;
  }
  __device__ __forceinline__ void locate(const AttnArgs& a, int64_t s1, int lane) {
    page = -1;
    if constexpr (kSparse) {
      have = f_have;
      head = f_head;
      pos = f_idx;
      ok = false;
      if (have) {
        const int seq = a.seq_ids ? __ldg(a.seq_ids + f_b) : f_b / a.per_seq;
        if (pos >= 0) {
          ok = pos / kPage < a.table_pages && seq >= 0 && seq < a.num_seqs;
          if (ok)
            page = __ldg(a.table + seq * a.tstride + pos / kPage);
          else
            flag_error(a.err, FP4IDX_ERRFLAG_PAGE);
        }
        fetch(a, s1, lane);
      }
    } else {
      have = seek(a, s1);
      if (!have) return;
      const int j = t0 + (x - xb) / 2;
      const int tile = j < pc.m.ts ? j : pc.m.tl + (j - pc.m.ts);
      key0 = tile * kPage + ((x - xb) & 1) * kSub;
      head = pc.it / pc.m.rcs;
      lo = pc.m.lo;
      hi = pc.m.hi;
      ok = key0 < hi;
      if (ok) page = __ldg(a.table + pc.b * a.tstride + tile);
      x += kWarps;
    }
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const Cursor<kSparse>& cur, int64_t s0,
                                        int64_t s1, int warp, int lane) {
    pc = cur;
    at = s0;
    xb = 0;
    x = warp;
    open(a, s1);
    if constexpr (kSparse) fetch(a, s1, lane);
    locate(a, s1, lane);
  }
  // Copies the next piece into the stage at `st` and moves on.  Rows of keys
  // that no query of the item sees are zero-filled.
  __device__ __forceinline__ void issue(const AttnArgs& a, int64_t s1, uint32_t st, uint32_t full,
                                        int lane) {
    constexpr int kChunks = D / 16;
    {
      const bool page_ok = page >= 0 && page < a.num_blocks;
      bool vis = ok;
      int64_t row_off = 0, sc_off = 0;  // this lane's (sparse) or the piece's (dense) codes
      if constexpr (!kSparse) {
        const int key = key0 + lane;
        vis = key < hi && (key >= lo || key < a.sinks);
      }
      if (vis && !page_ok) {
        flag_error(a.err, FP4IDX_ERRFLAG_PAGE);
        vis = false;
      }
      if (page_ok) {
        row_off = page * a.cstride +
                  ((int64_t)head * kPage + (kSparse ? pos : key0) % kPage) * D;
        sc_off = page * a.sstride + head;
      }
      const uint32_t mask = __ballot_sync(kFull, vis);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int q = j * 32 + lane;
        const int row = q / kChunks, c = q % kChunks;
        const int sw = D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
        const int bytes = (mask >> row & 1u) ? 16 : 0;
        const int64_t off =
            kSparse ? __shfl_sync(kFull, row_off, row) + c * 16 : row_off + q * 16;
        cp_async16(st + row * D + sw * 16, a.kc + off, bytes);
        cp_async16(st + kSub * D + row * D + sw * 16, a.vc + off, bytes);
      }
      const uint32_t sc = st + 2 * kSub * D;
      if (kSparse || lane == 0) {
        const int bytes = (kSparse ? vis : page_ok) ? 4 : 0;
        cp_async4(sc + lane * 4, a.ks + sc_off, bytes);
        cp_async4(sc + 128 + lane * 4, a.vs + sc_off, bytes);
      }
      if (lane == 0) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(sc + 256), "r"(mask) : "memory");
        mbar_arrive(full);
      }
      cp_arrive(full);
      locate(a, s1, lane);
    }
  }
};

// log2 of a power of two, from its exponent bits.
__device__ __forceinline__ float log2_scale(uint32_t bits) {
  return (float)((int)(bits >> 23 & 0xffu) - 127);
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int D, int NT, bool kSparse>
__global__ __launch_bounds__(kThreads, 1) void rows_kernel(const AttnArgs a) {
  constexpr int S = stages(D);
  constexpr int kStage = stage_bytes(D);
  constexpr int R = 8 * NT;
  constexpr int kChunks = D / 16;  // 16-byte chunks of a row of codes
  constexpr bool kQSmem = q_in_smem(D, NT);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t abort_flag;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, t = lane % 4;
  const int w8 = warp % kWarps;  // the ring
  const uint32_t ring = smem_addr(smem) + w8 * S * kStage;
  float* const st_m = reinterpret_cast<float*>(smem + kWarps * S * kStage);  // [warp][row]
  float* const st_M = st_m + kWarps * R;
  float* const st_l = st_M + kWarps * R;
  const uint32_t qs = smem_addr(st_l + kWarps * R);
  const uint32_t bars = qs + (kQSmem ? R * q_row_bytes(D) : 0);
  const auto full = [&](int i) { return bars + (w8 * S + i) * 16; };  // stage i is filled
  const auto empty = [&](int i) { return full(i) + 8; };              // and read
  volatile uint32_t* const abort = &abort_flag;

  if (tid < kWarps * S) {  // 32 lanes' copies and the mask; the computing warp
    // (testing hook, see fp4idx_test_withhold_next: a stage that never fills)
    mbar_init(bars + tid * 16, blockIdx.x == 0 && tid == a.withhold ? 34 : 33);
    mbar_init(bars + tid * 16 + 8, 1);
    fence_mbar_init();
  }
  if (tid == 0) abort_flag = 0;
  int64_t s0, s1;
  Cursor<kSparse> cur;
  const int64_t total = locate_share<kSparse>(a, cur, s0, s1);
  if (s0 >= s1) {
    if (a.split && tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  __syncthreads();

  if (warp >= kWarps) {
    // ---------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(
        256 - compute_regs(D, NT, kSparse)));
    Producer<D, kSparse> prod;
    prod.start(a, cur, s0, s1, w8, lane);
    int slot = 0;
    uint32_t parity = 1;  // of the stage's last release
    for (int i = 0; prod.have; ++i) {
      if (i >= S && !__all_sync(kFull, wait_bar(empty(slot), parity, abort))) break;
      prod.issue(a, s1, ring + slot * kStage, full(slot), lane);
      if (++slot == S) {
        slot = 0;
        parity ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(
      compute_regs(D, NT, kSparse)));

  int4 cut = make_int4(0, 0, 0, 0);
  int slot = 0;         // of the warp's next piece
  uint32_t parity = 0;  // of its fill
  bool held = false;    // the slot before it is not released yet
  int xb = 0, x = warp;
  for (int64_t at = s0; at < s1;) {
    const int u = cur.units(a);
    const int64_t end = min(s1, cur.begin + u);
    const int t0 = cur.cuts(a) ? (int)(at - cur.begin) : 0;
    const int xe = xb + 2 * (cur.cuts(a) ? (int)(end - at) : cur.m.nt);
    const int head = cur.it / cur.m.rcs;
    const int row0 = (cur.it - head * cur.m.rcs) * R;  // first row of the sequence's n * G
    const int rows = min(cur.m.n * a.G - row0, R);

    // ---- the queries, scaled into fp16's range, as the product's operand
    uint32_t qf[kQSmem ? 1 : NT][kChunks][2];
    float fac[NT][2];  // of columns 8i + 2t, + 1: score = sum * ks * fac
    int last[NT][2];   // position of the column's query
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = 8 * i + g;
      const int tok = cur.m.q0 + (row0 + r) / a.G;
      const int h = head * a.G + (row0 + r) % a.G;
      const bool live = r < rows && tok >= 0 && tok < a.T;
      const uint16_t* src = a.q + (live ? tok * a.q_ts + h * a.q_hs : 0) + 4 * t;
      uint2 w[kChunks];
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        w[c] = make_uint2(0, 0);
        if (live) w[c] = __ldg(reinterpret_cast<const uint2*>(src + 16 * c));
        const float2 e = unpack16(a.half, w[c].x), f = unpack16(a.half, w[c].y);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(e.x), fabsf(e.y)), fmaxf(fabsf(f.x), fabsf(f.y))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      // amax * 2^(141 - b) lies in [2^14, 2^15) for its biased exponent b
      const uint32_t b = max(__float_as_uint(amax) >> 23, 15u);
      const float up = __uint_as_float((268u - b) << 23 | (uint32_t)(a.scale_log2 < 0.0f) << 31);
      const float f = fabsf(a.scale_log2) * __uint_as_float((b - 14u) << 23);
      fac[i][0] = __shfl_sync(kFull, f, 8 * t);
      fac[i][1] = __shfl_sync(kFull, f, 8 * t + 4);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float2 e = unpack16(a.half, w[c].x), h2 = unpack16(a.half, w[c].y);
        const uint32_t b0 = pack16<true>(e.x * up, e.y * up);
        const uint32_t b1 = pack16<true>(h2.x * up, h2.y * up);
        if constexpr (kQSmem) {
          if (warp == 0)
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(qs + r * q_row_bytes(D) + 32 * c +
                                                                 8 * t),
                         "r"(b0), "r"(b1)
                         : "memory");
        } else {
          qf[i][c][0] = b0;
          qf[i][c][1] = b1;
        }
      }
      if constexpr (!kSparse) {
        last[i][0] = cur.m.first + (row0 + 8 * i + 2 * t) / a.G;
        last[i][1] = cur.m.first + (row0 + 8 * i + 2 * t + 1) / a.G;
      }
    }
    if constexpr (kQSmem) compute_sync();
    // a piece within [full_lo, full_hi) or the first tokens is seen by every row
    const int full_hi = cur.m.first + row0 / a.G + 1;
    const int full_lo =
        a.window > 0 ? cur.m.first + (row0 + rows - 1) / a.G - a.window + 1 : -(1 << 30);

    float acc[kChunks][NT][4];
    float m[NT][2], M[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[i][j] = M[i][j] = -INFINITY;
        l[i][j] = 0.0f;
      }
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][i][j] = 0.0f;

    for (; x < xe; x += kWarps) {
      __syncwarp();
      if (held && lane == 0) mbar_arrive(empty(slot == 0 ? S - 1 : slot - 1));
      held = true;
      const bool landed = __all_sync(kFull, wait_bar(full(slot), parity, abort));
      const uint32_t st = ring + slot * kStage;
      const uint32_t sc = st + 2 * kSub * D;
      if (++slot == S) {
        slot = 0;
        parity ^= 1;
      }
      if (!landed) continue;
      const uint32_t mask = lds32(sc + 256);
      if (mask == 0) continue;

      // ---- scores of 2 x 16 keys
      float s[2][NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[k][i][j] = 0.0f;
      const int lr = (lane & 7) + (lane >> 3 & 1) * 8;  // ldmatrix row of this lane
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t qb[NT][2][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (kQSmem) {
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                           : "=r"(qb[i][e][0]), "=r"(qb[i][e][1])
                           : "r"(qs + (8 * i + g) * q_row_bytes(D) + 32 * (c + e) + 8 * t));
            } else {
              qb[i][e][0] = qf[i][c + e][0];
              qb[i][e][1] = qf[i][c + e][1];
            }
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = 16 * k + lr;
          const int ch = c + (lane >> 4);
          const int sw = D == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
          uint32_t w[4];
          ldsm4(st + row * D + sw * 16, w);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t f[4];
            e4m3x4_to_f16x2(w[2 * e], f[0], f[2]);
            e4m3x4_to_f16x2(w[2 * e + 1], f[1], f[3]);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma16816(s[k][i], f, qb[i][e][0], qb[i][e][1]);
          }
        }
      }
      // ---- scales and masks
      float ks[2][2], ev[2][2];  // keys 16k + g, 16k + g + 8
      if constexpr (kSparse) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[k][e] = __uint_as_float(lds32(sc + 4 * (16 * k + 8 * e + g)));
            ev[k][e] = log2_scale(lds32(sc + 128 + 4 * (16 * k + 8 * e + g)));
          }
      } else {
        ks[0][0] = __uint_as_float(lds32(sc));
        ev[0][0] = log2_scale(lds32(sc + 128));
      }
      bool full = mask == kFull;
      int key0 = 0;
      if constexpr (!kSparse) {
        const int j = t0 + (x - xb) / 2;
        const int tile = j < cur.m.ts ? j : cur.m.tl + (j - cur.m.ts);
        key0 = tile * kPage + ((x - xb) & 1) * kSub;
        full = full && key0 + kSub <= full_hi && (key0 >= full_lo || key0 + kSub <= a.sinks);
      }
      // a piece of one page: the factor is not negative, so the largest sum
      // gives the largest score, and the products join the exponents' fma.  (A
      // factor of zero would make a masked score NaN.)
      float cf[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          cf[i][j] = kSparse ? 1.0f : fmaxf(ks[0][0] * fac[i][j], 0x1p-100f);
          if constexpr (kSparse) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) s[k][i][2 * e + j] *= ks[k][e] * fac[i][j];
          }
        }
      if (!full) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kl = 16 * k + 8 * e + g;
            const bool on = mask >> kl & 1u;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                bool see = on;
                if constexpr (!kSparse) {
                  const int key = key0 + kl;
                  see = see && key <= last[i][j] &&
                        (a.window <= 0 || key > last[i][j] - a.window || key < a.sinks);
                }
                if (!see) s[k][i][2 * e + j] = -INFINITY;
              }
          }
      }
      // ---- running softmax
      // contributions: the scores with their values' scale.  e0: of the piece
      // (dense), of its first visible key (sparse); kf = 2^(e0 - ev) of a key
      float e0 = ev[0][0], kf[2][2];
      bool spread = false;
      if constexpr (kSparse) {
        e0 = log2_scale(lds32(sc + 128 + 4 * (__ffs((int)mask) - 1)));
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = e0 - ev[k][e];
            spread = spread || ((mask >> (16 * k + 8 * e + g) & 1u) && fabsf(d) > kSpread);
            kf[k][e] = __int_as_float((127 + (int)fminf(fmaxf(d, -kSpread), kSpread)) << 23);
          }
      }
      bool move = false;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float a0 = s[0][i][j], a1 = s[0][i][2 + j], a2 = s[1][i][j], a3 = s[1][i][2 + j];
          const float top = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * cf[i][j];
          const float topv = kSparse ? fmaxf(fmaxf(a0 + ev[0][0], a1 + ev[0][1]),
                                             fmaxf(a2 + ev[1][0], a3 + ev[1][1]))
                                     : top + e0;
          move = move || topv > M[i][j] + kSlack || top > m[i][j] + kFar;
        }
      if (__any_sync(kFull, move)) {  // the references follow the maxima
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float al[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float a0 = s[0][i][j], a1 = s[0][i][2 + j], a2 = s[1][i][j],
                        a3 = s[1][i][2 + j];
            const float top = max_g(fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * cf[i][j]);
            float topv = top + e0;
            if constexpr (kSparse)
              topv = max_g(fmaxf(fmaxf(a0 + ev[0][0], a1 + ev[0][1]),
                                 fmaxf(a2 + ev[1][0], a3 + ev[1][1])));
            const float m1 = fmaxf(m[i][j], top), M1 = fmaxf(M[i][j], topv);
            l[i][j] *= exp2_approx(m[i][j] - or_zero(m1));
            al[j] = exp2_approx(M[i][j] - or_zero(M1));
            m[i][j] = m1;
            M[i][j] = M1;
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            acc[c][i][0] *= al[0];
            acc[c][i][1] *= al[1];
            acc[c][i][2] *= al[0];
            acc[c][i][3] *= al[1];
          }
        }
      }
      // far: the piece's contributions lie so far below M that l loses them
      bool far = spread;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) far = far || or_zero(M[i][j]) - e0 - or_zero(m[i][j]) > kFar;
      const bool any_far = __any_sync(kFull, far);
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mz = or_zero(m[i][j]), Mz = or_zero(M[i][j]);
          float sum = 0.0f;
          if (any_far) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) sum += exp2_approx(fmaf(s[k][i][2 * e + j], cf[i][j], -mz));
          }
          float w = 0.0f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = s[k][i][2 * e + j];
              v = exp2_approx(fmaf(v, cf[i][j], (kSparse ? ev[k][e] : e0) - Mz + kShift));
              w = kSparse ? fmaf(v, kf[k][e], w) : w + v;
            }
          l[i][j] += any_far ? sum : w * exp2_approx(Mz - e0 - kShift - mz);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          pb[k][i][0] = transpose8(pack16<true>(s[k][i][0], s[k][i][1]));
          pb[k][i][1] = transpose8(pack16<true>(s[k][i][2], s[k][i][3]));
        }
      }
      // ---- output sums: rows g and g + 8 of the fragment are d = 16c + 2g, + 1
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int sw = D == 128 ? (c ^ (lane & 7)) : (c ^ ((lane >> 1) & 3));
        uint32_t w[4];
        ldsm4_trans(st + kSub * D + lane * D + sw * 16, w);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t f[4];
          e4m3x4_to_f16x2(prmt(w[2 * k], 0u, 0x3120u), f[0], f[1]);
          e4m3x4_to_f16x2(prmt(w[2 * k + 1], 0u, 0x3120u), f[2], f[3]);
#pragma unroll
          for (int i = 0; i < NT; ++i) mma16816(acc[c][i], f, pb[k][i][0], pb[k][i][1]);
        }
      }
    }

    // ---- the warps' sums joined, through each warp's slot that is not
    // released yet (a warp without one has no sums)
    const int free_slot = slot == 0 ? S - 1 : slot - 1;
    __shared__ int free_of[kWarps];
    __shared__ float join_f[kWarps][R];  // factor of a warp's sums
    __shared__ float join_s[3][R];       // of the row: the common factors; lse, log2
    if (lane == 0) free_of[warp] = free_slot;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = sum_g(l[i][j]);
        if (g == 0) {
          st_m[warp * R + 8 * i + 2 * t + j] = m[i][j];
          st_M[warp * R + 8 * i + 2 * t + j] = M[i][j];
          st_l[warp * R + 8 * i + 2 * t + j] = sum;
        }
      }
    const bool whole = at == cur.begin && end == cur.begin + u;
    const int part = blockIdx.x * 2 + (at == cur.begin && at != s0 ? 1 : 0);
    // a slot holds 16 rows; the columns of rows 2t, 2t + 1 are turned by 16 t
    // floats, so that the lanes of a store lie on different banks
#pragma unroll
    for (int i0 = 0; i0 < NT; i0 += 2) {
      constexpr int kPer = NT < 2 ? NT : 2;
      float* const own = reinterpret_cast<float*>(smem + (warp * S + free_slot) * kStage);
      if (held) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<float2*>(own + (8 * i + 2 * t + j) * D + ((16 * c) ^ (16 * t)) +
                                         2 * g) = make_float2(acc[c][i0 + i][j],
                                                              acc[c][i0 + i][2 + j]);
      }
      compute_sync();
      if (i0 == 0) {
        // lane (row, warp): the factors, once for all columns
        for (int e = tid; e < R * kWarps; e += kWarps * 32) {
          const int r = e / kWarps, w = e % kWarps;
          const float mw = st_m[w * R + r], Mw = st_M[w * R + r];
          float mg = mw, Mg = Mw;
#pragma unroll
          for (int d = 1; d < kWarps; d *= 2) {
            mg = fmaxf(mg, __shfl_xor_sync(kFull, mg, d));
            Mg = fmaxf(Mg, __shfl_xor_sync(kFull, Mg, d));
          }
          float L = mw == -INFINITY ? 0.0f : st_l[w * R + r] * exp2_approx(mw - mg);
#pragma unroll
          for (int d = 1; d < kWarps; d *= 2) L += __shfl_xor_sync(kFull, L, d);
          join_f[w][r] = mw == -INFINITY ? 0.0f : exp2_approx(Mw - Mg);
          if (w == 0) {
            // 2^(M-m-10) in two halves: with values near 2^-126 it is 0 itself
            const float half = mg == -INFINITY ? 0.0f : exp2_approx(0.5f * (Mg - mg - kShift));
            join_s[0][r] = mg == -INFINITY ? 0.0f : __frcp_rn(L) * half;
            join_s[1][r] = mg == -INFINITY ? -INFINITY : mg + __log2f(L);
            join_s[2][r] = half;
          }
        }
        compute_sync();
      }
      for (int e = tid; e < 8 * kPer * D / 4; e += kWarps * 32) {
        const int rl = e / (D / 4), d = e % (D / 4) * 4;
        const int r = 8 * i0 + rl;
        if (r >= rows) continue;
        const int at_d = rl * D + (d ^ (rl / 2 % 4 * 16));
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = join_f[w][r];
          if (f == 0.0f) continue;  // no sums there, or none that count
          const float4 v = *reinterpret_cast<const float4*>(
              smem + (w * S + free_of[w]) * kStage + at_d * 4);
          o.x = fmaf(v.x, f, o.x);
          o.y = fmaf(v.y, f, o.y);
          o.z = fmaf(v.z, f, o.z);
          o.w = fmaf(v.w, f, o.w);
        }
        const float f = join_s[0][r], lse2 = join_s[1][r], f2 = join_s[2][r];
        o.x = o.x * f * f2;
        o.y = o.y * f * f2;
        o.z = o.z * f * f2;
        o.w = o.w * f * f2;
        if (whole) {
          const int tok = cur.m.q0 + (row0 + r) / a.G;
          const int h = head * a.G + (row0 + r) % a.G;
          if (tok >= 0 && tok < a.T) {
            const int64_t orow = (int64_t)tok * a.Hq + h;
            *reinterpret_cast<uint2*>(a.out + orow * D + d) =
                make_uint2(pack16(a.half, o.x, o.y), pack16(a.half, o.z, o.w));
            if (a.lse && d == 0) a.lse[orow] = lse2 * kLn2;
          }
        } else {
          *reinterpret_cast<float4*>(a.part_out + ((int64_t)part * R + r) * D + d) = o;
          if (d == 0) a.part_lse[part * R + r] = lse2;
        }
      }
      compute_sync();
    }
    if (!whole && at == cur.begin)  // the first fragment of a cut item
      cut = make_int4(cur.b, cur.it - head * cur.m.rcs, head,
                      (cta_of(cur.begin + u - 1, total) - (int)blockIdx.x + 1) * 2 + (part & 1));
    xb = xe;
    at = end;
    if (at < s1) cur.next(a);
  }
  if (tid == 0) {
    if (a.split) a.cuts[blockIdx.x] = cut;
    if (*abort) flag_error(a.err, FP4IDX_ERRFLAG_TIMEOUT);
  }
}

// Joins the partial outputs of the items that a share's end cut: weights
// 2^(lse - max lse), in the order of the CTAs, applied in two halves (a part of
// weight 2^-126 counts where its values are as much larger).  One block per CTA
// whose share begins such an item, a warp per row.
template <int D, bool kSparse>
__global__ __launch_bounds__(128) void join_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x;
  const int4 cut = a.cuts[cta];
  const int n = cut.w / 2;
  if (n < 2) return;
  const Seq m = seq_of<kSparse>(a, cut.x);
  const int lane = threadIdx.x % 32;
  const int head = cut.z, row0 = cut.y * a.R;
  const int rows = min(m.n * a.G - row0, a.R);
  const int first = 2 * cta + (cut.w & 1);
  for (int r = threadIdx.x / 32; r < rows; r += 4) {
    float top = -INFINITY;
    for (int f = lane; f < n; f += 32)
      top = fmaxf(top, a.part_lse[(f == 0 ? first : 2 * (cta + f)) * a.R + r]);
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    constexpr int kV = D / 32;
    float o[kV], den = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) o[i] = 0.0f;
    if (top != -INFINITY) {
#pragma unroll 4
      for (int f = 0; f < n; ++f) {
        const int64_t slot = (int64_t)(f == 0 ? first : 2 * (cta + f)) * a.R + r;
        const float half = exp2_approx(0.5f * (a.part_lse[slot] - top));
        den = fmaf(half, half, den);
        const float* p = a.part_out + slot * D + lane * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i) o[i] = fmaf(p[i] * half, half, o[i]);
      }
      const float inv = __frcp_rn(den);
#pragma unroll
      for (int i = 0; i < kV; ++i) o[i] *= inv;
    }
    const int tok = m.q0 + (row0 + r) / a.G;
    const int h = head * a.G + (row0 + r) % a.G;
    if (tok < 0 || tok >= a.T) continue;
    const int64_t orow = (int64_t)tok * a.Hq + h;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + lane * kV);
#pragma unroll
    for (int i = 0; i < kV; i += 2) dst[i / 2] = pack16(a.half, o[i], o[i + 1]);
    if (a.lse && lane == 0)
      a.lse[orow] = top == -INFINITY ? -INFINITY : (top + __log2f(den)) * kLn2;
  }
}

template <int D, int NT, bool kSparse>
fp4idx_status launch_one(const AttnArgs& a, int grid, cudaStream_t stream) {
  auto* kern = rows_kernel<D, NT, kSparse>;
  constexpr int bytes = smem_bytes(D, NT);
  static_assert(bytes + 2048 <= 227 * 1024, "the rings fit the shared memory");
  static SmemOnce once;
  if (!once.set(kern, bytes)) return FP4IDX_ERR_CUDA;
  if (launch_kernel(kern, (unsigned)grid, kThreads, bytes, stream, a) != cudaSuccess)
    return FP4IDX_ERR_CUDA;
  if (!a.split) return FP4IDX_OK;
  return launch_after(join_kernel<D, kSparse>, (unsigned)grid, 128, stream, a) == cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}

template <int D, bool kSparse>
fp4idx_status launch_nt(const AttnArgs& a, int grid, cudaStream_t stream) {
  if (a.R == 8) return launch_one<D, 1, kSparse>(a, grid, stream);
  // 32 rows of 128 columns do not fit the registers
  if (D == 128 || a.R == 16) return launch_one<D, 2, kSparse>(a, grid, stream);
  return launch_one<D, D == 64 ? 4 : 2, kSparse>(a, grid, stream);
}

}  // namespace

fp4idx_status launch_rows(const AttnArgs& a, int head_dim, bool sparse, int grid,
                          cudaStream_t stream) {
  if (head_dim == 128)
    return sparse ? launch_nt<128, true>(a, grid, stream) : launch_nt<128, false>(a, grid, stream);
  return sparse ? launch_nt<64, true>(a, grid, stream) : launch_nt<64, false>(a, grid, stream);
}

}  // namespace fp4idx_impl
