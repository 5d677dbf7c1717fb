// fp4idx_attn_tiles.cu -- attention over the 8-bit cache for many query rows
// per key head: prompts in whole or in chunks (fp4idx_paged_attention_fp8,
// defined in include/fp4idx_attention.h), on the tensor cores through
// tcgen05.mma kind::f16.
//
// What bounds it.  4 D operations per query row and key against 2 D bytes per
// key for a whole item of 256 rows: the tensor cores, then the exponentials.
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
// Roles (13 warps, one CTA per SM).  The item's rows are two M = 128 halves A
// and B that share every key tile of 128 keys (two pages).
//   warps 0-3, 4-7  softmax of half A, of half B: a row per thread, its scores
//                   read from TMEM, its probabilities written back over them
//   warps 8-11      converters: the codes from global memory through
//                   registers to fp16 tiles in shared memory, keys as
//                   [key][d], values transposed as [d][key], both K-major in
//                   128-byte swizzled rows, two stages each; the next tile's
//                   loads are in flight while this one is converted
//   warp 12         issues the MMAs: S = Q K^T, then O += P V with P from
//                   TMEM.  While half A's softmax runs, half B's products do.
// TMEM: scores A and B at columns 0 and 128 (P over the upper half of its
// scores, once they are in registers), O at 256 and 256 + D.
// Every wait is bounded (1 s) and a shared abort flag stops every role; MMAs
// in flight are waited for before TMEM is released.

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kPage = FP4IDX_KV_BLOCK;
constexpr int kTile = 128;  // keys of a tile
constexpr int kHalfRows = 128;
constexpr int kItemRows = 2 * kHalfRows;
constexpr int kConvWarp = 8, kMmaWarp = 12;
constexpr int kThreads = 13 * 32;
constexpr int kStages = 2;
constexpr int kScaleRing = 4;
constexpr float kShift = 10.0f, kSlack = 4.0f, kFar = 60.0f;
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t q_bytes(int D) { return kItemRows * D * 2; }
__host__ __device__ constexpr uint32_t kv_bytes(int D) { return kTile * D * 2; }
__host__ __device__ constexpr uint32_t smem_bytes(int D) {
  return q_bytes(D) + 2 * kStages * kv_bytes(D) + 1024;
}

// One item: 256 consecutive rows (token i, head g: row i * G + g) of a
// sequence and key head, its keys' tiles [t0, t1) of the visible list.
struct Item {
  int b, head, row0, rows;
  int q0, first;  // first query token of the sequence, its position
  int hi;         // keys any row sees are below hi
  int ts, tl;     // tiles: 0 .. ts-1, then tl ..
  int t0, t1;
};

__device__ __forceinline__ bool item_of(const AttnArgs& a, Item& m) {
  // the last row chunks first: they see the most keys
  const int per = a.batch * a.Hkv;
  const int sp = blockIdx.x % a.splits;
  const int i = blockIdx.x / a.splits;
  const int rc = a.rc_max - 1 - i / per;
  m.b = i % per / a.Hkv;
  m.head = i % per % a.Hkv;
  const int ctx = min(max(__ldg(a.ctx + m.b), 0), a.max_context);
  int full = a.max_q;
  m.q0 = m.b * a.max_q;
  if (a.starts) {
    m.q0 = __ldg(a.starts + m.b);
    full = max(__ldg(a.starts + m.b + 1) - m.q0, 0);
  }
  const int n = min(full, a.max_q);
  m.first = ctx - full;
  m.row0 = rc * kItemRows;
  m.rows = min(n * a.G - m.row0, kItemRows);
  if (m.rows <= 0) return false;
  m.hi = max(min(ctx, m.first + (m.row0 + m.rows - 1) / a.G + 1), 0);
  int lo = a.window > 0 ? max(m.first + m.row0 / a.G - a.window + 1, 0) : 0;
  lo = min(lo, m.hi);
  m.tl = lo / kTile;
  m.ts = a.window > 0 ? min((a.sinks + kTile - 1) / kTile, m.tl) : 0;
  const int nt = m.ts + (m.hi + kTile - 1) / kTile - m.tl;
  m.t0 = (int)((int64_t)nt * sp / a.splits);
  m.t1 = (int)((int64_t)nt * (sp + 1) / a.splits);
  return true;
}

__device__ __forceinline__ int key_of_tile(const Item& m, int t) {
  return (t < m.ts ? t : m.tl + (t - m.ts)) * kTile;
}

// Waits for a phase; false when another role has given up or after 1 s.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    for (int k = 0; k < 16; ++k)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
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

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
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

// The visible keys of a row in a tile: key i (from the tile's first) with
// i <= hi and (i >= lo or i < sk).
struct Vis {
  int hi, lo, sk;
  __device__ __forceinline__ bool sees(int i) const { return i <= hi && (i >= lo || i < sk); }
};

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
  kBars = kQFull + 2
};

struct Ctl {
  uint64_t bars[kBars];
  float4 scales[kScaleRing];  // ks of the tile's two pages, vs of both (vs < 0: page left out)
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

  Item m;
  if (!item_of(a, m)) return;
  const int nt = m.t1 - m.t0;
  const int halves = m.rows > kHalfRows ? 2 : 1;

  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool commit = (i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kPFull) ||
                          (i >= kODone && i < kQFull);
      mbar_init(bar(i), commit ? 1 : 4);
    }
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
  const uint32_t tmem = ctl.tmem;

  if (warp < kConvWarp) {
    // ------------------------------------------------------------- softmax
    const int half = warp / 4;
    if (half < halves) {
      const int r = m.row0 + half * kHalfRows + tid % kHalfRows;  // row of the sequence
      const int rl = tid % kHalfRows;
      const bool live_row = r < m.row0 + m.rows;
      const int tok = m.q0 + r / a.G, h = m.head * a.G + r % a.G;
      const bool live = live_row && tok >= 0 && tok < a.T;
      const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
      const uint32_t ts = tmem + lanes + half * 128, tp = ts + 64;
      const uint32_t to = tmem + lanes + 256 + half * D;
      // ---- this row of Q, scaled by a power of two, into shared memory
      float fac;
      {
        const uint16_t* src = a.q + (live ? tok * a.q_ts + h * a.q_hs : 0);
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (live) w = __ldg(reinterpret_cast<const uint4*>(src) + c);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16(a.half, u[j]);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        const uint32_t b = max(__float_as_uint(amax) >> 23, 15u);
        float up = __uint_as_float((268u - b) << 23);
        fac = a.scale_log2 * __uint_as_float((b - 14u) << 23);
        if (fac < 0.0f) {
          fac = -fac;
          up = -up;
        }
        const uint32_t dst = sq + half * kHalves * kQHalf + rl * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (live) w = __ldg(reinterpret_cast<const uint4*>(src) + c);
          uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16(a.half, u[j]);
            u[j] = pack16<true>(f.x * up, f.y * up);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                           dst + c / 8 * kQHalf + ((c % 8) ^ (rl & 7)) * 16),
                       "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
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
      float mm = -INFINITY, MM = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int t = 0; t < nt; ++t) {
        ok = __all_sync(kFull, wait_bar(bar(kSFull + half), t & 1, abort));
        if (!ok) break;
        fence_after();
        if (!idle) {
          const float4 sc = ctl.scales[t % kScaleRing];
          const int kb = key_of_tile(m, m.t0 + t);
          const bool both = sc.z >= 0.0f && sc.w >= 0.0f;
          const bool full = both && kb + kTile <= pos_lo + 1 &&
                            (a.window <= 0 || kb > pos_hi - a.window || kb + kTile <= a.sinks);
          const Vis vis{pos - kb, a.window > 0 ? pos - kb - a.window + 1 : -(1 << 30),
                        a.sinks - kb};
          const float c0 = fac * sc.x, c1 = fac * sc.y;
          const float e0 = log2_scale(sc.z), e1 = log2_scale(sc.w);
          float s[64];
          const auto mask = [&](int from, bool page) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!page || !vis.sees(from + i)) s[i] = -INFINITY;
          };
          const auto top = [&]() {
            float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              x0 = fmaxf(x0, s[i]);
              x1 = fmaxf(x1, s[i + 1]);
              x2 = fmaxf(x2, s[i + 2]);
              x3 = fmaxf(x3, s[i + 3]);
            }
            return fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
          };
          // a masked maximum times a factor of zero stays masked
          const auto times = [](float x, float c) { return x == -INFINITY ? x : x * c; };
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          tmem_wait_ld();
          if (!full) mask(0, sc.z >= 0.0f);
          const float x0 = times(top(), c0);
          tmem_ld32(ts + 64, s);
          tmem_ld32(ts + 96, s + 32);
          tmem_wait_ld();
          if (!full) mask(64, sc.w >= 0.0f);
          const float x1 = times(top(), c1);
          const float m1 = fmaxf(mm, fmaxf(x0, x1));
          const float M1 = fmaxf(x0 + e0, x1 + e1);
          // ---- O's reference, moved seldom
          const bool move = M1 > MM + kSlack || (MM == -INFINITY && M1 != -INFINITY);
          if (__any_sync(kFull, move)) {
            const float al = move ? exp2_approx(MM - M1) : 1.0f;
            if (move) MM = M1;
            if (t > 0) {
              ok = __all_sync(kFull, wait_bar(bar(kODone + half), (t - 1) & 1, abort));
              if (!ok) break;
              fence_after();
              // a register's worth of columns at a time: s stays live
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= al;
                tmem_st32(to + c, reinterpret_cast<const uint32_t*>(o));
              }
              tmem_wait_st();
            }
          }
          const float mz = or_zero(m1), Mz = or_zero(MM);
          l *= exp2_approx(mm - mz);
          mm = m1;
          const auto weigh = [&](float c, float e, uint32_t col) {
            const float ref = Mz - e - kShift;
            const bool far = ref + kShift - mz > kFar;
            float a0 = 0.0f, a1 = 0.0f;
            if (__any_sync(kFull, far)) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                a0 += s[i] == -INFINITY ? 0.0f : exp2_approx(fmaf(s[i], c, -mz));
            }
            uint32_t p[32];
            float b0 = 0.0f, b1 = 0.0f;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              float y0, y1;
              fma2s(y0, y1, s[i], s[i + 1], c, -ref);
              if (!full) {  // -inf * 0
                y0 = s[i] == -INFINITY ? -INFINITY : y0;
                y1 = s[i + 1] == -INFINITY ? -INFINITY : y1;
              }
              y0 = exp2_approx(y0);
              y1 = exp2_approx(y1);
              b0 += y0;
              b1 += y1;
              p[i / 2] = pack16<true>(y0, y1);
            }
            tmem_st32(col, p);
            a1 = (b0 + b1) * exp2_approx(ref - mz);
            l += far ? a0 : a1;
          };
          weigh(c1, e1, tp + 32);
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          tmem_wait_ld();
          if (!full) mask(0, sc.z >= 0.0f);
          weigh(c0, e0, tp);
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + half));
      }
      // ---- the output row
      if (ok && nt > 0) ok = __all_sync(kFull, wait_bar(bar(kODone + half), (nt - 1) & 1, abort));
      if (ok && !idle) {
        fence_after();
        const bool some = mm != -INFINITY;
        const float inv = some ? __frcp_rn(l) : 0.0f;
        const float f = some ? exp2_approx(MM - mm - kShift) : 0.0f;
        const float lse2 = some ? mm + __log2f(l) : -INFINITY;
        const int64_t orow = (int64_t)tok * a.Hq + h;
        const int64_t prow = (int64_t)blockIdx.x * kItemRows + half * kHalfRows + rl;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          if (nt > 0) {
            tmem_ld32(to + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = some ? o[i] * inv * f : 0.0f;
          if (!live) {
          } else if (a.splits > 1) {
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
          if (a.splits > 1)
            a.part_lse[prow] = lse2;
          else if (a.lse)
            a.lse[orow] = lse2 * kLn2;
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------- converters
    const int cw = warp - kConvWarp;
    const int32_t* table = a.table + m.b * a.tstride;
    constexpr int kRowLanes = D / 16;              // 16-byte pieces of a row of codes
    constexpr int kKRows = 32 / kRowLanes;         // key rows of one warp load
    constexpr int kKLoads = kTile / (4 * kKRows);  // key loads of a lane and tile
    // values: a warp step covers 64 keys (16 lanes x 4 rows) x 32 d (2 lanes)
    constexpr int kVSteps = (kTile / 64) * (D / 32) / 4;
    uint4 kreg[kKLoads], vreg[kVSteps][4];
    int page0 = -1, page1 = -1;  // of the tile whose loads come next

    const auto pages = [&](int t) {
      page0 = page1 = -1;
      if (t >= nt) return;
      const int kb = key_of_tile(m, m.t0 + t);
      if (kb < m.hi) page0 = __ldg(table + kb / kPage);
      if (kb + kPage < m.hi) page1 = __ldg(table + kb / kPage + 1);
    };
    const auto page_ok = [&](int p) { return p >= 0 && p < a.num_blocks; };
    const auto load_k = [&](int t) {
      const int kb = key_of_tile(m, m.t0 + t);
#pragma unroll
      for (int i = 0; i < kKLoads; ++i) {
        const int key = (cw * kKLoads + i) * kKRows + lane / kRowLanes;
        const int p = key < kPage ? page0 : page1;
        kreg[i] = make_uint4(0, 0, 0, 0);
        if (page_ok(p) && kb + key < m.hi)
          kreg[i] = __ldg(reinterpret_cast<const uint4*>(
              a.kc + p * a.cstride + ((int64_t)m.head * kPage + key % kPage) * D +
              lane % kRowLanes * 16));
      }
    };
    const auto load_v = [&](int t, int p0, int p1) {
      const int kb = key_of_tile(m, m.t0 + t);
#pragma unroll
      for (int i = 0; i < kVSteps; ++i) {
        const int step = cw * kVSteps + i;
        const int kh = step / (D / 32), d = step % (D / 32) * 32 + lane / 16 * 16;
        const int p = kh == 0 ? p0 : p1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = lane % 16 * 4 + j;
          vreg[i][j] = make_uint4(0, 0, 0, 0);
          if (page_ok(p) && kb + kh * kPage + key < m.hi)
            vreg[i][j] = __ldg(reinterpret_cast<const uint4*>(
                a.vc + p * a.cstride + ((int64_t)m.head * kPage + key) * D + d));
        }
      }
    };
    pages(0);
    if (nt > 0) load_k(0);
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const int stage = t % kStages;
      const uint32_t parity = (uint32_t)(t / kStages + 1) & 1u;
      const int p0 = page0, p1 = page1;
      load_v(t, p0, p1);
      pages(t + 1);
      // ---- keys: [key][d]
      if (t >= kStages) ok = __all_sync(kFull, wait_bar(bar(kKEmpty + stage), parity, abort));
      if (!ok) break;
      if (cw == 0 && lane == 0) {
        const int kb = key_of_tile(m, m.t0 + t);
        float4 sc = make_float4(1.0f, 1.0f, -1.0f, -1.0f);
        if (page_ok(p0)) {
          sc.x = a.ks[p0 * a.sstride + m.head];
          sc.z = fabsf(a.vs[p0 * a.sstride + m.head]);
        } else if (kb < m.hi) {
          flag_error(a.err, FP4IDX_ERRFLAG_PAGE);
        }
        if (page_ok(p1)) {
          sc.y = a.ks[p1 * a.sstride + m.head];
          sc.w = fabsf(a.vs[p1 * a.sstride + m.head]);
        } else if (kb + kPage < m.hi) {
          flag_error(a.err, FP4IDX_ERRFLAG_PAGE);
        }
        ctl.scales[t % kScaleRing] = sc;
      }
      {
        const uint32_t dst = sk + stage * kv_bytes(D);
#pragma unroll
        for (int i = 0; i < kKLoads; ++i) {
          const int key = (cw * kKLoads + i) * kKRows + lane / kRowLanes;
          const int c = lane % kRowLanes;  // d 16c .. 16c + 15
          const uint32_t u[4] = {kreg[i].x, kreg[i].y, kreg[i].z, kreg[i].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) e4m3x4_to_f16x2(u[j], o[2 * j], o[2 * j + 1]);
          const uint32_t row = dst + c / 4 * (kTile * 128) + key * 128;
          // the lanes of the second column block store their upper half first:
          // the two blocks lie on the same banks
          const int flip = c / 4;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int w = e ^ flip;
            const uint32_t at = row + (((c % 4) * 2 + w) ^ (key & 7)) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at),
                         "r"(w ? o[4] : o[0]), "r"(w ? o[5] : o[1]), "r"(w ? o[6] : o[2]),
                         "r"(w ? o[7] : o[3])
                         : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKFull + stage));
      }
      if (t + 1 < nt) load_k(t + 1);
      // ---- values: [d][key]
      if (t >= kStages) ok = __all_sync(kFull, wait_bar(bar(kVEmpty + stage), parity, abort));
      if (!ok) break;
      {
        const uint32_t dst = sv + stage * kv_bytes(D);
#pragma unroll
        for (int i = 0; i < kVSteps; ++i) {
          const int step = cw * kVSteps + i;
          const int kh = step / (D / 32), d0 = step % (D / 32) * 32 + lane / 16 * 16;
          const uint32_t blk = dst + kh * (D * 128);
          const int q = lane % 16;  // keys 4q .. 4q + 3: 8 bytes of a row
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // d0 + 4c ..
            const uint32_t r0 = (&vreg[i][0].x)[c], r1 = (&vreg[i][1].x)[c];
            const uint32_t r2 = (&vreg[i][2].x)[c], r3 = (&vreg[i][3].x)[c];
            // byte pairs (key 0, key 1) and (2, 3) of four d
            const uint32_t a01 = prmt(r0, r1, 0x5140u), a23 = prmt(r0, r1, 0x7362u);
            const uint32_t b01 = prmt(r2, r3, 0x5140u), b23 = prmt(r2, r3, 0x7362u);
            uint32_t lo[4], hi[4];
            e4m3x4_to_f16x2(a01, lo[0], lo[1]);
            e4m3x4_to_f16x2(a23, lo[2], lo[3]);
            e4m3x4_to_f16x2(b01, hi[0], hi[1]);
            e4m3x4_to_f16x2(b23, hi[2], hi[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = d0 + 4 * c + j;
              const uint32_t at = blk + d * 128 + (((q / 2) ^ (d & 7)) * 16) + (q % 2) * 8;
              asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(lo[j]), "r"(hi[j])
                           : "memory");
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kVFull + stage));
      }
    }
  } else if (lane == 0 && nt > 0) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t kQkDesc = f16_idesc(kTile), kPvDesc = f16_idesc(D);
    const auto issue_s = [&](int half, int stage) {
      const uint32_t qa = sq + half * kHalves * kQHalf, kb = sk + stage * kv_bytes(D);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k % 4) * 32;
        mma_ss(tmem + half * 128, sw128_desc(qa + k / 4 * kQHalf + off),
               sw128_desc(kb + k / 4 * (kTile * 128) + off), kQkDesc, k > 0);
      }
      mma_commit(bar(kSFull + half));
    };
    const auto issue_o = [&](int half, int stage, bool first) {
      const uint32_t vb = sv + stage * kv_bytes(D);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(tmem + 256 + half * D, tmem + half * 128 + 64 + k * 8,
               sw128_desc(vb + k / 4 * (D * 128) + (k % 4) * 32), kPvDesc, !first || k > 0);
      mma_commit(bar(kODone + half));
    };
    bool ok = wait_bar(bar(kKFull), 0, abort);
    for (int h = 0; h < halves && ok; ++h) {
      ok = wait_bar(bar(kQFull + h), 0, abort);
      if (!ok) break;
      fence_after();
      issue_s(h, 0);
    }
    if (ok) mma_commit(bar(kKEmpty));
    for (int t = 0; t < nt && ok; ++t) {
      const int stage = t % kStages, next = (t + 1) % kStages;
      ok = wait_bar(bar(kVFull + stage), (uint32_t)(t / kStages) & 1u, abort);
      for (int h = 0; h < halves && ok; ++h) {
        ok = wait_bar(bar(kPFull + h), t & 1, abort);
        if (!ok) break;
        fence_after();
        issue_o(h, stage, t == 0);
        if (t + 1 < nt) {
          if (h == 0) ok = wait_bar(bar(kKFull + next), (uint32_t)((t + 1) / kStages) & 1u, abort);
          if (!ok) break;
          issue_s(h, next);
        }
      }
      if (!ok) break;
      mma_commit(bar(kVEmpty + stage));
      if (t + 1 < nt) mma_commit(bar(kKEmpty + next));
    }
  }

  __syncwarp();
  fence_before();
  __syncthreads();
  if (*abort) {
    // MMAs in flight land before TMEM and shared memory are released
    if (tid == kMmaWarp * 32) {
      flag_error(a.err, FP4IDX_ERRFLAG_TIMEOUT);
      const uint32_t b = bar(kQFull);  // re-used: one arrival by the commit
      asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(b) : "memory");
      mbar_init(b, 1);
      fence_mbar_init();
      mma_commit(b);
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

// Joins the partial outputs of an item's key ranges: weights 2^(lse - max),
// in order.  A warp per row; grid: items (without the ranges) x 8 rows.
template <int D>
__global__ __launch_bounds__(256) void join_tiles_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kBlocks = kItemRows / 8;
  const int i = blockIdx.x / kBlocks;
  const int rl = blockIdx.x % kBlocks * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int per = a.batch * a.Hkv;
  const int rc = a.rc_max - 1 - i / per, b = i % per / a.Hkv, head = i % per % a.Hkv;
  int q0 = b * a.max_q, n = a.max_q;
  if (a.starts) {
    q0 = __ldg(a.starts + b);
    n = min(max(__ldg(a.starts + b + 1) - q0, 0), a.max_q);
  }
  const int r = rc * kItemRows + rl;
  const int tok = q0 + r / a.G;
  if (r >= n * a.G || tok < 0 || tok >= a.T) return;
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s)
    top = fmaxf(top, a.part_lse[((int64_t)i * a.splits + s) * kItemRows + rl]);
  constexpr int kV = D / 32;
  float o[kV], den = 0.0f;
#pragma unroll
  for (int j = 0; j < kV; ++j) o[j] = 0.0f;
  if (top != -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const int64_t row = ((int64_t)i * a.splits + s) * kItemRows + rl;
      const float w = exp2_approx(a.part_lse[row] - top);
      den += w;
#pragma unroll
      for (int j = 0; j < kV; ++j) o[j] = fmaf(a.part_out[row * D + lane * kV + j], w, o[j]);
    }
    const float inv = __frcp_rn(den);
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j] *= inv;
  }
  const int64_t orow = (int64_t)tok * a.Hq + head * a.G + r % a.G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + lane * kV);
#pragma unroll
  for (int j = 0; j < kV; j += 2) dst[j / 2] = pack16(a.half, o[j], o[j + 1]);
  if (a.lse && lane == 0)
    a.lse[orow] = top == -INFINITY ? -INFINITY : (top + __log2f(den)) * kLn2;
}

template <int D>
fp4idx_status launch_d(const AttnArgs& a, cudaStream_t stream) {
  static SmemOnce once;
  if (!once.set(tiles_kernel<D>, smem_bytes(D))) return FP4IDX_ERR_CUDA;
  const int64_t items = (int64_t)a.batch * a.Hkv * a.rc_max;
  if (launch_kernel(tiles_kernel<D>, (unsigned)(items * a.splits), kThreads, smem_bytes(D), stream,
                    a) != cudaSuccess)
    return FP4IDX_ERR_CUDA;
  if (a.splits == 1) return FP4IDX_OK;
  return launch_after(join_tiles_kernel<D>, (unsigned)(items * (kItemRows / 8)), 256, stream, a) ==
                 cudaSuccess
             ? FP4IDX_OK
             : FP4IDX_ERR_CUDA;
}

}  // namespace

fp4idx_status launch_tiles(const AttnArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace fp4idx_impl
