// Appending new tokens to the 4-bit cache, and reading tokens back.
//
// K is rotated as in fox_append.cu, but to the nearest bf16 of the exact a cos - b sin: the 4-bit form has borders everywhere, and a
// value on the other side of one is a whole step away. Kahan's difference of products (one product's rounding error by a fused
// multiply-add, taken off the fused difference) is within 1.5 units of the last place of fp32; where that leaves open on which side of
// a border of bf16 the value lies (1 of 10000), 64 bits decide, in which the products are exact.
//
// A thread holds 8 channels, four neighbours a block: its largest magnitude by two shuffles, one scale byte by the first of them, a
// word of codes by each (fox_four.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_append.cuh"
#include "fox_four.h"

namespace fox {
namespace {

struct Append4Params : AppendParams {
  uint8_t* ks;
  uint8_t* vs;
};

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
}

// a c - b s in 64 bits, rounded to odd in fp32: what then rounds to bf16 is rounded once.
__device__ __noinline__ float turned_exactly(float a, float c, float b, float s) {
  const double x = static_cast<double>(a) * c - static_cast<double>(b) * s;
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}
// a c - b s, to be rounded to bf16.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  const float p = __fmul_rn(b, s), e = __fmaf_rn(b, s, -p);
  const float r = __fsub_rn(__fmaf_rn(a, c, -p), e);
  const uint32_t near = (__float_as_uint(r) & 0xFFFFu) - 0x7FFCu;
  return near <= 8u ? turned_exactly(a, c, b, s) : r;
}

// Eight channels from c0 on of a head whose first `rot` are rotated; `mine` and `other` hold them and their partners'
// (of `pairs` they are their own).
__device__ __forceinline__ void turn8(float* x, const float* other, int c0, const float* cs, const float* sn, int rot,
                                      int pairs) {
  if (pairs) {
    const float4 c = *reinterpret_cast<const float4*>(cs + c0 / 2), s = *reinterpret_cast<const float4*>(sn + c0 / 2);
    const float co[4] = {c.x, c.y, c.z, c.w}, si[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = turned(a, co[i], b, si[i]);
      x[2 * i + 1] = turned(b, co[i], -a, si[i]);
    }
    return;
  }
  const bool first = c0 < rot / 2;
  const int at = first ? c0 : c0 - rot / 2;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(cs + at + i), s = *reinterpret_cast<const float4*>(sn + at + i);
    const float co[4] = {c.x, c.y, c.z, c.w}, si[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i + j] = turned(x[i + j], co[j], first ? other[i + j] : -other[i + j], si[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void copy_rows4(const Append4Params& p, RowPlace* places) {
  const PagedArgs& a = p.a;
  const int hs = a.d == 128 ? 4 : 3, hp = 1 << hs, blocks = a.d / kFourBlock;  // units of a head
  const int nk = a.Hkv << hs;
  const CopyShape x = copy_shape(2 * nk + (p.qn ? a.H << hs : 0));
  const int tid = threadIdx.x, lane = tid & 31, block = blockIdx.x - p.gate_blocks;
  const int chunk = block % x.chunks, row0 = block / x.chunks * (kRows * x.side);
  const int sub = x.side > 1 ? tid / x.per_row : 0, at = x.side > 1 ? tid - sub * x.per_row : chunk * kThreads + tid;
  // Units of a row are a multiple of 8 (16 with 128 channels) and so are a block's: a head's lie in neighbouring lanes.
  const bool live = at < x.per_row && sub < x.side, is_v = at >= nk && at < 2 * nk, is_q = at >= 2 * nk;
  const int w = is_q ? at - 2 * nk : is_v ? at - nk : at, h = w >> hs, j = w & (hp - 1), c0 = j * 8;
  const long long stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_q ? p.qn : is_v ? p.vn : p.kn) +
                             (size_t)(row0 + sub) * stride + h * a.d + c0;
  uint4 u[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    u[i] = make_uint4(0, 0, 0, 0);
    if (live && row0 + sub + i * x.side < a.rows) u[i] = __ldcs(reinterpret_cast<const uint4*>(src));
    src += x.side * stride;
  }
  const int rows = min(kRows * x.side, a.rows - row0);
  for (int r = tid; r < rows; r += kThreads) places[r] = row_place(p, row0 + r);
  __syncthreads();
  const int half = p.rot / 16;  // units of half the rotated channels
  const int partner = (lane & ~(hp - 1)) | (j < half ? j + half : j - half);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = i * x.side + sub;
    float f[8], o[8];
    unpack8(u[i], f);
    if (p.rot > 0 && !p.pairs) {
      uint4 y;
      y.x = __shfl_sync(0xffffffffu, u[i].x, partner);
      y.y = __shfl_sync(0xffffffffu, u[i].y, partner);
      y.z = __shfl_sync(0xffffffffu, u[i].z, partner);
      y.w = __shfl_sync(0xffffffffu, u[i].w, partner);
      unpack8(y, o);
    }
    const RowPlace g = live && r < rows ? places[r] : RowPlace{-1, 0, 0};
    if (g.page >= 0 && !is_v && c0 < p.rot) {
      turn8(f, o, c0, p.cos + (size_t)g.pos * (p.rot / 2), p.sin + (size_t)g.pos * (p.rot / 2), p.rot, p.pairs);
      u[i] = pack8(f);
      unpack8(u[i], f);
    }
    float most = 0.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      most = fmaxf(most, fabsf(f[e]));
      nan |= f[e] != f[e];
    }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    if (g.page < 0) continue;
    if (is_q) {
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.qo) + ((size_t)(row0 + r) * a.H + h) * a.d + c0), u[i]);
      continue;
    }
    odd |= nan || most > 430080.f;
    const uint32_t byte = four_scale_byte(most);
    const float inv = byte ? 1.f / four_scale(byte) : 0.f;
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) code |= four_code(f[e], inv) << (4 * e);
    const int b = j >> 2, t = j & 3;
    uint8_t* row = static_cast<uint8_t*>(is_v ? a.v : a.k) + four_row(a, g.page, h, g.slot);
    *reinterpret_cast<uint32_t*>(row + (is_v ? four_v_word(b, t, g.slot, blocks) : four_k_word(b, t, blocks))) =
        is_v ? code : four_k_order(code);
    if (t == 0) {
      if (is_v)
        p.vs[four_scale_row(a, g.page, h, g.slot & ~15) + four_v_scale(b, g.slot, blocks)] = static_cast<uint8_t>(byte);
      else
        p.ks[four_scale_row(a, g.page, h, g.slot) + b] = static_cast<uint8_t>(byte);
    }
  }
  if (odd && a.err) atomicOr(a.err, DEV_ERR_RANGE);
}

__global__ void __launch_bounds__(kThreads, 8) cache_append4_kernel(const Append4Params p) {
  __shared__ union {
    float zs[128][kGateHeads + 1];
    RowPlace places[kBlockRows];
  } sh;
  grid_dep_wait();
  grid_dep_trigger();
  if (static_cast<int>(blockIdx.x) < p.gate_blocks)
    gate_block(p, sh.zs);
  else
    copy_rows4(p, sh.places);
}

// The values of rows, 8 channels a thread: s u has 7 significant bits, so bf16 has it exactly.
struct Read4Params : AppendParams {
  const uint8_t* ks;
  const uint8_t* vs;
  __nv_bfloat16* ko;
  __nv_bfloat16* vo;
};
__global__ void __launch_bounds__(kThreads, 8) cache_read4_kernel(const Read4Params p) {
  __shared__ RowPlace places[kBlockRows];
  grid_dep_wait();
  grid_dep_trigger();
  const PagedArgs& a = p.a;
  const int hs = a.d == 128 ? 4 : 3, blocks = a.d / kFourBlock, nk = a.Hkv << hs;
  const CopyShape x = copy_shape(2 * nk);
  const int tid = threadIdx.x, chunk = blockIdx.x % x.chunks, row0 = blockIdx.x / x.chunks * (kRows * x.side);
  const int sub = x.side > 1 ? tid / x.per_row : 0, at = x.side > 1 ? tid - sub * x.per_row : chunk * kThreads + tid;
  const bool live = at < x.per_row && sub < x.side, is_v = at >= nk;
  const int w = is_v ? at - nk : at, h = w >> hs, j = w & ((1 << hs) - 1), b = j >> 2, t = j & 3;
  const int rows = min(kRows * x.side, a.rows - row0);
  for (int r = tid; r < rows; r += kThreads) places[r] = row_place(p, row0 + r);
  __syncthreads();
  if (!live) return;
  __nv_bfloat16* out = is_v ? p.vo : p.ko;
  const long long stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = i * x.side + sub;
    if (r >= rows) break;
    const RowPlace g = places[r];
    if (g.page < 0) continue;
    const uint8_t* row = static_cast<const uint8_t*>(is_v ? a.v : a.k) + four_row(a, g.page, h, g.slot);
    uint32_t code =
        *reinterpret_cast<const uint32_t*>(row + (is_v ? four_v_word(b, t, g.slot, blocks) : four_k_word(b, t, blocks)));
    if (!is_v) code = four_k_code(code);
    const float s = four_scale(is_v ? p.vs[four_scale_row(a, g.page, h, g.slot & ~15) + four_v_scale(b, g.slot, blocks)]
                                    : p.ks[four_scale_row(a, g.page, h, g.slot) + b]);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = s * static_cast<float>(static_cast<int>(code >> (4 * e) & 15u) - 8);
    __stcs(reinterpret_cast<uint4*>(out + (size_t)(row0 + r) * stride + h * a.d + j * 8), pack8(f));
  }
}

int row_units4(const PagedArgs& a, bool with_q) { return (2 * a.Hkv + (with_q ? a.H : 0)) * (a.d / 8); }

}  // namespace

bool append4_fits(const PagedArgs& a, bool with_q) { return append_blocks(a, row_units4(a, with_q)).fit(); }

cudaError_t launch_cache_append4(const CacheAppendArgs& x, void* ks, void* vs, cudaStream_t s) {
  Append4Params p = {};
  static_cast<AppendParams&>(p) = append_params(x);
  p.ks = static_cast<uint8_t*>(ks);
  p.vs = static_cast<uint8_t*>(vs);
  return launch_append(cache_append4_kernel, p, row_units4(p.a, p.qn != nullptr), s);
}

cudaError_t launch_cache_read4(const CacheAppendArgs& x, void* ks, void* vs, cudaStream_t s) {
  Read4Params p = {};
  static_cast<AppendParams&>(p) = append_params(x);
  p.ks = static_cast<const uint8_t*>(ks);
  p.vs = static_cast<const uint8_t*>(vs);
  p.ko = static_cast<__nv_bfloat16*>(const_cast<void*>(x.k));
  p.vo = static_cast<__nv_bfloat16*>(const_cast<void*>(x.v));
  TraceScope trace("cache_read", s);
  const cudaError_t e = launch_dependent(cache_read4_kernel, dim3(static_cast<unsigned>(append_blocks(p.a, row_units4(p.a, false)).copies)),
                                         dim3(kThreads), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fox
