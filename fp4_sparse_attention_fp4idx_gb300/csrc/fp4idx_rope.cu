// fp4idx_rope.cu -- rotary positions of the main queries and keys, with one to
// four position axes (fp4idx_rope_qk, defined in include/fp4idx_step.h).
//
// What bounds it.  Each element is read and written once, 4 bytes, against three
// operations: HBM.  The cosines and sines of a token are shared by its heads.
//
// Layout.  A unit is 8 pairs of a row, two 16-byte words.  A warp takes a token
// and a range of its heads, queries' before keys'; a lane keeps its 8 cosines
// and sines in registers over the heads where a row's units divide a warp (they
// are loaded again for each head, from L1, where not).  Which axis turns a pair
// is two bits of a table made on the host.

#include "fp4idx_attn.cuh"
#include "fp4idx_step.h"

namespace fp4idx_impl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 512;
constexpr int kUnroll = 4;  // units of a lane in flight

struct RopeSide {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_ts, in_hs, out_ts, out_hs;
};

struct RopeArgs {
  RopeSide q, k;
  int32_t q_heads, heads;  // of q; of both
  const int64_t* positions;
  int64_t axis_stride;
  int32_t axes;
  const float* cos;
  const float* sin;
  int64_t max_pos;
  int32_t half;      // pairs of a row
  int32_t units;     // half / 8
  int32_t tail;      // 16-byte words of a row that are copied
  int32_t per_warp;  // heads of a warp
  int32_t splits;    // warps of a token
  int64_t T;
  uint32_t* err;
  uint32_t axis_bits[kMaxPairs / 16];  // pair i: bits 2 (i % 16) of word i / 16
};

// (a cos - b sin, b cos + a sin), every step rounded.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

template <bool kHalf, bool kNeox, bool kFixed>
__global__ __launch_bounds__(kThreads) void rope_kernel(const __grid_constant__ RopeArgs a) {
  const int lane = threadIdx.x % 32;
  const int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int64_t t = w / a.splits;
  if (t >= a.T) return;
  const int h0 = (int)(w - t * a.splits) * a.per_warp;
  const int h1 = min(h0 + a.per_warp, a.heads);
  int64_t pos[4];
  bool ok = true;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    pos[x] = x < a.axes ? __ldg(a.positions + x * a.axis_stride + t) : 0;
    ok = ok && pos[x] >= 0 && pos[x] < a.max_pos;
  }
  if (!ok) {
    if (h0 == 0 && lane == 0) flag_error(a.err, FP4IDX_ERRFLAG_POSITION);
    return;
  }
  // the angles of unit u's pairs
  float c[8], s[8];
  const auto angles = [&](int u) {
    const uint32_t axis = a.axis_bits[u / 2] >> (u % 2 * 16) & 0xffffu;
    const auto row = [&](uint32_t x) {
      const int64_t p = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
      return p * a.half + u * 8;
    };
    if (axis == (axis & 3u) * 0x5555u) {  // one axis turns them all
      const int64_t at = row(axis & 3u);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 x = ld_f4(a.cos + at + i), y = ld_f4(a.sin + at + i);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = row(axis >> (2 * i) & 3u) + i;
        c[i] = __ldg(a.cos + at);
        s[i] = __ldg(a.sin + at);
      }
    }
  };
  const auto place = [&](int h, const uint16_t*& in, uint16_t*& out) {
    const bool key = h >= a.q_heads;
    const int hh = key ? h - a.q_heads : h;
    const RopeSide& side = key ? a.k : a.q;
    in = side.in + t * side.in_ts + hh * side.in_hs;
    out = side.out + t * side.out_ts + hh * side.out_hs;
  };
  // the two words of a unit
  const auto first = [&](int u) { return kNeox ? u * 8 : u * 16; };
  const int gap = kNeox ? a.half : 8;

  const int end = h1 * a.units;
  if (kFixed) angles(lane % a.units);
  for (int j = h0 * a.units + lane; j < end; j += 32 * kUnroll) {
    uint4 x[kUnroll], y[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      if (j + 32 * e >= end) continue;
      const int h = (j + 32 * e) / a.units, u = (j + 32 * e) - h * a.units;
      const uint16_t* in;
      uint16_t* out;
      place(h, in, out);
      x[e] = *reinterpret_cast<const uint4*>(in + first(u));
      y[e] = *reinterpret_cast<const uint4*>(in + first(u) + gap);
    }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      if (j + 32 * e >= end) continue;
      const int h = (j + 32 * e) / a.units, u = (j + 32 * e) - h * a.units;
      if (!kFixed) angles(u);
      const uint16_t* in;
      uint16_t* out;
      place(h, in, out);
      uint32_t v[8] = {x[e].x, x[e].y, x[e].z, x[e].w, y[e].x, y[e].y, y[e].z, y[e].w};
      if constexpr (kNeox) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 p = unpack16<kHalf>(v[i]), q = unpack16<kHalf>(v[i + 4]);
          turn(p.x, q.x, c[2 * i], s[2 * i]);
          turn(p.y, q.y, c[2 * i + 1], s[2 * i + 1]);
          v[i] = pack16<kHalf>(p.x, p.y);
          v[i + 4] = pack16<kHalf>(q.x, q.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 p = unpack16<kHalf>(v[i]);
          turn(p.x, p.y, c[i], s[i]);
          v[i] = pack16<kHalf>(p.x, p.y);
        }
      }
      *reinterpret_cast<uint4*>(out + first(u)) = make_uint4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<uint4*>(out + first(u) + gap) = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
  // ---- what is not turned
  for (int j = h0 * a.tail + lane; j < h1 * a.tail; j += 32) {
    const int h = j / a.tail, u = j - h * a.tail;
    const uint16_t* in;
    uint16_t* out;
    place(h, in, out);
    if (in == out) continue;
    const int at = 2 * a.half + u * 8;
    *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(in + at);
  }
}

template <bool kHalf, bool kNeox>
cudaError_t launch_rope(const RopeArgs& a, unsigned grid, cudaStream_t s) {
  return 32 % a.units == 0 ? launch_kernel(rope_kernel<kHalf, kNeox, true>, grid, kThreads, 0, s, a)
                           : launch_kernel(rope_kernel<kHalf, kNeox, false>, grid, kThreads, 0, s,
                                           a);
}

}  // namespace
}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" fp4idx_status fp4idx_rope_qk(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
    int64_t q_out_token_stride, int64_t q_out_head_stride, int64_t q_heads, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
    int64_t k_out_head_stride, int64_t k_heads, int dtype, int64_t head_dim,
    const int64_t* positions, int64_t axis_stride, const int32_t* sections, int num_axes,
    int axis_order, const float* cos, const float* sin, int64_t max_pos, int64_t rope_dim,
    int rope_style, int64_t num_tokens, uint32_t* err_flags, void* stream) {
  if (num_tokens < 0) return FP4IDX_ERR_SHAPE;
  if (num_tokens == 0) return FP4IDX_OK;
  if (!q || !q_out || (k_heads > 0 && (!k || !k_out)) || !positions || !sections || !cos || !sin)
    return FP4IDX_ERR_NULL;
  if (num_tokens >= (1ll << 31) || q_heads < 1 || q_heads >= (1 << 20) || k_heads < 0 ||
      k_heads >= (1 << 20) || head_dim < 16 || head_dim > 2 * kMaxPairs || head_dim % 8 ||
      rope_dim < 16 || rope_dim > head_dim || rope_dim % 16 || num_axes < 1 || num_axes > 4 ||
      max_pos < 1 || max_pos >= (1ll << 40))
    return FP4IDX_ERR_SHAPE;
  if (!dtype_ok(dtype) ||
      (rope_style != FP4IDX_ROPE_NEOX && rope_style != FP4IDX_ROPE_INTERLEAVED) ||
      (axis_order != FP4IDX_AXES_SECTIONS && axis_order != FP4IDX_AXES_INTERLEAVED))
    return FP4IDX_ERR_ARG;
  const int half = (int)(rope_dim / 2);
  int64_t sum = 0;
  for (int x = 0; x < num_axes; ++x) {
    if (sections[x] < 0) return FP4IDX_ERR_ARG;
    sum += sections[x];
  }
  if (sum != half) return FP4IDX_ERR_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) ||
      q_token_stride % 8 || q_head_stride % 8 || q_out_token_stride % 8 || q_out_head_stride % 8 ||
      (k_heads > 0 && (k_token_stride % 8 || k_head_stride % 8 || k_out_token_stride % 8 ||
                       k_out_head_stride % 8)) ||
      !aligned(positions, 8) || !aligned(cos, 16) || !aligned(sin, 16) || !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  RopeArgs a = {};
  a.q = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_token_stride,
         q_head_stride, q_out_token_stride, q_out_head_stride};
  a.k = {static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_token_stride,
         k_head_stride, k_out_token_stride, k_out_head_stride};
  a.q_heads = (int32_t)q_heads;
  a.heads = (int32_t)(q_heads + k_heads);
  a.positions = positions;
  a.axis_stride = axis_stride;
  a.axes = num_axes;
  a.cos = cos;
  a.sin = sin;
  a.max_pos = max_pos;
  a.half = half;
  a.units = half / 8;
  a.tail = (int32_t)(head_dim - rope_dim) / 8;
  a.T = num_tokens;
  a.err = err_flags;
  for (int i = 0, x = 0, left = sections[0]; i < half; ++i) {
    int axis;
    if (axis_order == FP4IDX_AXES_INTERLEAVED) {
      axis = i % num_axes;
      if (i / num_axes >= sections[axis]) axis = 0;
    } else {
      while (left == 0) left = sections[++x];
      --left;
      axis = x;
    }
    a.axis_bits[i / 16] |= (uint32_t)axis << (i % 16 * 2);
  }
  // A warp takes kUnroll units a lane; where the tokens are too few to fill the
  // GPU so, one unit.
  int64_t per = 32 * kUnroll / a.units;
  if (per < 1) per = 1;
  if (num_tokens * ((a.heads + per - 1) / per) < 4 * kMaxGrid * kWarps) per = 32 / a.units;
  if (per < 1) per = 1;
  a.per_warp = (int32_t)per;
  a.splits = (int32_t)((a.heads + per - 1) / per);
  const int64_t blocks = (num_tokens * a.splits + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return FP4IDX_ERR_SHAPE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool h = dtype == FP4IDX_FP16;
  const unsigned grid = (unsigned)blocks;
  const cudaError_t st = rope_style == FP4IDX_ROPE_NEOX
                             ? (h ? launch_rope<true, true>(a, grid, s)
                                  : launch_rope<false, true>(a, grid, s))
                             : (h ? launch_rope<true, false>(a, grid, s)
                                  : launch_rope<false, false>(a, grid, s));
  return st == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA;
}
