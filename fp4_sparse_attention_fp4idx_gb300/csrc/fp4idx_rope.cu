// fp4idx_rope.cu -- rotary positions of the main queries and keys, with one to
// four position axes (fp4idx_rope_qk, defined in include/fp4idx_step.h).
//
// What bounds it.  Each element is read and written once, 4 bytes, against three
// operations: HBM.  The cosines and sines of a token are shared by its heads.
// Measured: 16,384 tokens of 40 heads of 128 in 53 us, 6.3 TB/s, 93% of the copy rate;
// 30,011 tokens of 18 heads with three axes 48 us, 5.8 TB/s.
//
// Layout.  A unit is 8 pairs of a row, two 16-byte words; what is not turned is
// copied by units of two words more.  A thread keeps the cosines and sines of one
// unit of a token in registers and turns that unit in every `groups`-th head,
// queries' before keys', kUnroll of them in flight; its first rows are asked for
// before the angles, whose addresses wait for the positions.  Consecutive threads
// take a head's units, then the next head's, so that a warp reads a run of memory.
// Which axis turns a pair is two bits of a table made on the host.

#include <utility>

#include "fp4idx_attn.cuh"
#include "fp4idx_step.h"

namespace fp4idx_impl {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;
constexpr int kUnroll = 4;  // heads of a thread in flight

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
  int32_t units;     // of a row: half / 8 that are turned, the others copied
  int32_t groups;    // threads that share a token's unit
  FastDiv by_units, by_groups;
  int32_t tail;      // 16-byte words of a row that are copied
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

template <bool kHalf, bool kNeox>
__global__ __launch_bounds__(kThreads, 3) void rope_kernel(const __grid_constant__ RopeArgs a) {
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;  // unit u, group g, token t
  const uint32_t heads_id = a.by_units.div(id);
  const int u = (int)(id - heads_id * a.units);
  const uint32_t t = a.by_groups.div(heads_id);
  const int g = (int)(heads_id - t * a.groups);
  if (t >= a.T) return;
  int64_t pos[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    pos[x] = x < a.axes ? __ldg(a.positions + x * a.axis_stride + t) : 0;
  const auto in_at = [&](int h) {
    return h < a.q_heads ? a.q.in + t * a.q.in_ts + h * a.q.in_hs
                         : a.k.in + t * a.k.in_ts + (h - a.q_heads) * a.k.in_hs;
  };
  const auto out_at = [&](int h) {
    return h < a.q_heads ? a.q.out + t * a.q.out_ts + h * a.q.out_hs
                         : a.k.out + t * a.k.out_ts + (h - a.q_heads) * a.k.out_hs;
  };
  // the two words of the unit (a copied one may lack the second)
  const bool turned = u * 8 < a.half;
  const int copy = 2 * a.half + (u - a.half / 8) * 16;
  const int first = !turned ? copy : kNeox ? u * 8 : u * 16;
  const int second = turned && kNeox ? first + a.half : first + 8;
  const bool both = turned || second < 2 * a.half + a.tail * 8;
  uint4 x[kUnroll], y[kUnroll];
  const auto load = [&](int h) {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e)
      if (h + e * a.groups < a.heads) {
        const uint16_t* in = in_at(h + e * a.groups);
        x[e] = *reinterpret_cast<const uint4*>(in + first);
        if (both) y[e] = *reinterpret_cast<const uint4*>(in + second);
      }
  };
  load(g);
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) ok = ok && pos[i] >= 0 && pos[i] < a.max_pos;
  if (!ok) {
    if (u == 0 && g == 0) flag_error(a.err, FP4IDX_ERRFLAG_POSITION);
    return;
  }
  float c[8], s[8];
  const uint32_t axis = turned ? a.axis_bits[u / 2] >> (u % 2 * 16) & 0xffffu : 0u;
  const auto row = [&](uint32_t i) {
    const int64_t p = i == 0 ? pos[0] : i == 1 ? pos[1] : i == 2 ? pos[2] : pos[3];
    return p * a.half + u * 8;
  };
  if (!turned) {
  } else if (axis == (axis & 3u) * 0x5555u) {  // one axis turns them all
    const int64_t at = row(axis & 3u);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 v = ld_f4(a.cos + at + i), w = ld_f4(a.sin + at + i);
      c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
      s[i] = w.x, s[i + 1] = w.y, s[i + 2] = w.z, s[i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = row(axis >> (2 * i) & 3u) + i;
      c[i] = __ldg(a.cos + at);
      s[i] = __ldg(a.sin + at);
    }
  }
  for (int h = g;;) {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      if (h + e * a.groups >= a.heads) continue;
      if (turned) {
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
        x[e] = make_uint4(v[0], v[1], v[2], v[3]);
        y[e] = make_uint4(v[4], v[5], v[6], v[7]);
      }
      uint16_t* out = out_at(h + e * a.groups);
      *reinterpret_cast<uint4*>(out + first) = x[e];
      if (both) *reinterpret_cast<uint4*>(out + second) = y[e];
    }
    h += kUnroll * a.groups;
    if (h >= a.heads) break;
    load(h);
  }
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
  if (num_tokens >= (1ll << 31) || q_heads < 1 || q_heads > 65535 || k_heads < 0 ||
      q_heads + k_heads > 65535 || head_dim < 16 || head_dim > 2 * kMaxPairs || head_dim % 8 ||
      rope_dim < 16 || rope_dim > head_dim || rope_dim % 16 || num_axes < 1 || num_axes > 4 ||
      max_pos < 1 || max_pos >= (1ll << 40))
    return FP4IDX_ERR_SHAPE;
  if (!dtype_ok(dtype) ||
      (rope_style != FP4IDX_ROPE_NEOX && rope_style != FP4IDX_ROPE_INTERLEAVED) ||
      (axis_order != FP4IDX_AXES_SECTIONS && axis_order != FP4IDX_AXES_INTERLEAVED))
    return FP4IDX_ERR_ARG;
  // in place is row by row
  const auto moves = [&](const void* in, const void* out, int64_t heads, int64_t ts, int64_t hs,
                         int64_t ots, int64_t ohs) {
    return in == out && ((num_tokens > 1 && ts != ots) || (heads > 1 && hs != ohs));
  };
  if (moves(q, q_out, q_heads, q_token_stride, q_head_stride, q_out_token_stride,
            q_out_head_stride) ||
      (k_heads > 0 && moves(k, k_out, k_heads, k_token_stride, k_head_stride, k_out_token_stride,
                            k_out_head_stride)))
    return FP4IDX_ERR_ARG;
  const int half = (int)(rope_dim / 2);
  int64_t sum = 0;
  for (int x = 0; x < num_axes; ++x) {
    if (sections[x] < 0) return FP4IDX_ERR_ARG;
    sum += sections[x];
  }
  if (sum != half) return FP4IDX_ERR_ARG;
  if (q_token_stride % 8 || q_head_stride % 8 || q_out_token_stride % 8 || q_out_head_stride % 8 ||
      (k_heads > 0 && (k_token_stride % 8 || k_head_stride % 8 || k_out_token_stride % 8 ||
                       k_out_head_stride % 8)))
    return FP4IDX_ERR_ALIGN;
  // two threads would write one row of an output
  const auto overlap = [&](int64_t heads, int64_t ts, int64_t hs) {
    int64_t near = ts < 0 ? -ts : ts, far = hs < 0 ? -hs : hs, n = num_tokens;
    if (heads == 1) return num_tokens > 1 && near < head_dim;
    if (num_tokens == 1) return far < head_dim;
    if (near > far) {
      std::swap(near, far);
      n = heads;
    }
    return near < head_dim || far < head_dim || (n - 1) > (far - head_dim) / near;
  };
  if (overlap(q_heads, q_out_token_stride, q_out_head_stride) ||
      (k_heads > 0 && overlap(k_heads, k_out_token_stride, k_out_head_stride)))
    return FP4IDX_ERR_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) ||
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
  // In place nothing needs to be copied.
  const bool in_place = q == q_out && (k_heads == 0 || k == k_out);
  if (in_place) a.tail = 0;
  a.units = half / 8 + (a.tail + 1) / 2;
  // A thread takes 8 heads (angles read once for 512 bytes of rows); where the
  // tokens are too few to fill the GPU so, fewer.
  const int64_t ids = num_tokens * a.units;
  int64_t per = 2 * kUnroll;
  while (per > 1 && ids * ((a.heads + per - 1) / per) < (int64_t)kMaxGrid * 1024) per /= 2;
  a.groups = (int32_t)((a.heads + per - 1) / per);
  a.by_units = make_fastdiv((uint32_t)a.units);
  a.by_groups = make_fastdiv((uint32_t)a.groups);
  const int64_t blocks = (ids * a.groups + kThreads - 1) / kThreads;
  if (ids * a.groups >= (1ll << 32) - kThreads) return FP4IDX_ERR_SHAPE;
  const bool h = dtype == FP4IDX_FP16;
  auto* kern = rope_style == FP4IDX_ROPE_NEOX
                   ? (h ? rope_kernel<true, true> : rope_kernel<false, true>)
                   : (h ? rope_kernel<true, false> : rope_kernel<false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t st = cudaLaunchKernelEx(&cfg, kern, a);
  return st == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA;
}
