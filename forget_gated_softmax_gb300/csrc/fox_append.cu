// Appending new tokens to the paged cache: K (rotated by its position where asked), V and the gates.
//
// Rotation of the first `dim` channels of a head by the angles of the token's position, given as
// tables cos, sin [max_pos, dim / 2]:  (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin) with
// (a, b) = (i, i + dim / 2), or (2i, 2i + 1) with `pairs`. The products and the sum are fp32 and
// round once, to the cache's type.
//
// One launch does copies and gates, in different blocks (the gates' first: they are few and slow). Where a
// sequence may bring more than one page, the scan of the pages' bases follows (gates, scan and copies in three
// launches: 6 prompts of up to 16384 tokens 268 against 262 us, 4 of up to 2000 36.6 against 31, 2 of 257 17 against
// 15.4).
//
// Bound by memory: each of k, v (q) read once and written once. 6 prompts of up to 16384 tokens (1.44 GB) take
// 258 us, 5.6 TB/s (262 with g_low); one token of 128 sequences 4.0 us of GPU time among others in a graph, the launch and a
// few dependent trips to memory (with and without g_low).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_append.cuh"

namespace fox {
namespace {

// Work of the copy: units of two 16-byte chunks of one head of a row, in the order k, v, q heads.
// Rotates two chunks: wx at channel c0 of the head, wy its partner's, or its neighbour with `pairs`.
template <typename T>
__device__ __forceinline__ void turn(uint4& wx, uint4& wy, int c0, const float* cs, const float* sn, int pairs) {
  constexpr int kN = Vec<T>::kN;
  float x[kN], y[kN], u[kN], v[kN];
  Vec<T>::unpack(wx, x);
  Vec<T>::unpack(wy, y);
  if (pairs) {
    // neighbouring chunks: kN angles side by side
    float co[kN], si[kN];
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      *reinterpret_cast<float4*>(co + i) = *reinterpret_cast<const float4*>(cs + c0 / 2 + i);
      *reinterpret_cast<float4*>(si + i) = *reinterpret_cast<const float4*>(sn + c0 / 2 + i);
    }
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const int j = i / 2, k = (kN + i) / 2;
      u[i] = x[i] * co[j] - x[i + 1] * si[j];
      u[i + 1] = x[i + 1] * co[j] + x[i] * si[j];
      v[i] = y[i] * co[k] - y[i + 1] * si[k];
      v[i + 1] = y[i + 1] * co[k] + y[i] * si[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 co = *reinterpret_cast<const float4*>(cs + c0 + i);
      const float4 si = *reinterpret_cast<const float4*>(sn + c0 + i);
      const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[i + j] = x[i + j] * cc[j] - y[i + j] * ss[j];
        v[i + j] = y[i + j] * cc[j] + x[i + j] * ss[j];
      }
    }
  }
  wx = Vec<T>::pack(u);
  wy = Vec<T>::pack(v);
}

// A thread has one unit of kRows rows: what it copies is worked out once, since instructions are what bounds
// this copy besides memory. The loads of k, v, q come first; the look-ups of the rows' pages and positions
// run meanwhile.
template <typename T>
__device__ __forceinline__ void copy_rows(const AppendParams& p, RowPlace* places) {
  constexpr int kN = Vec<T>::kN;
  const PagedArgs& a = p.a;
  const int hs = (kN == 8 ? 2 : 3) + (a.d == 128), hp = 1 << hs;  // units of a head
  const int nk = a.Hkv << hs;
  const CopyShape x = copy_shape(2 * nk + (p.qn ? a.H << hs : 0));
  const int tid = threadIdx.x, block = blockIdx.x - p.gate_blocks;
  const int chunk = block % x.chunks, row0 = block / x.chunks * (kRows * x.side);
  const int sub = x.side > 1 ? tid / x.per_row : 0, at = x.side > 1 ? tid - sub * x.per_row : chunk * kThreads + tid;
  const bool live = at < x.per_row && sub < x.side, is_v = at >= nk && at < 2 * nk, is_q = at >= 2 * nk;
  const int w = is_q ? at - 2 * nk : is_v ? at - nk : at, h = w >> hs, j = w & (hp - 1);
  // The unit's chunks: a channel range and its partner in the rotation, or two neighbours.
  const int half_chunks = p.rot / kN / 2;
  const bool apart = !is_v && !p.pairs && j < half_chunks;
  const int c0 = (apart ? j : 2 * j) * kN, c1 = apart ? c0 + half_chunks * kN : c0 + kN;
  const long long stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const T* src = static_cast<const T*>(is_q ? p.qn : is_v ? p.vn : p.kn) + (size_t)(row0 + sub) * stride + h * a.d;
  uint4 u[kRows], v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (live && row0 + sub + i * x.side < a.rows) {
      u[i] = __ldcs(reinterpret_cast<const uint4*>(src + c0));
      v[i] = __ldcs(reinterpret_cast<const uint4*>(src + c1));
    }
    src += x.side * stride;
  }
  const int rows = min(kRows * x.side, a.rows - row0);
  for (int r = tid; r < rows; r += kThreads) places[r] = row_place(p, row0 + r);
  __syncthreads();
  if (!live) return;
  const bool turned = !is_v && c0 < p.rot;
  T* base = is_q ? static_cast<T*>(p.qo) + ((size_t)(row0 + sub) * a.H + h) * a.d
                 : static_cast<T*>(is_v ? a.v : a.k) + (size_t)h * a.page_size * a.d;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = i * x.side + sub;
    if (r >= rows) break;
    const RowPlace g = places[r];
    if (g.page < 0) continue;
    if (turned)
      turn<T>(u[i], v[i], c0, p.cos + (size_t)g.pos * (p.rot / 2), p.sin + (size_t)g.pos * (p.rot / 2), p.pairs);
    T* dst = base + (is_q ? (size_t)i * x.side * a.H * a.d : kv_offset(a, g.page, 0, g.slot));
    // stored as data that is not needed next: the other way measured 9 % slower on long prompts
    __stcs(reinterpret_cast<uint4*>(dst + c0), u[i]);
    __stcs(reinterpret_cast<uint4*>(dst + c1), v[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 8) cache_append_kernel(const AppendParams p) {
  __shared__ union {
    float zs[128][kGateHeads + 1];
    RowPlace places[kBlockRows];
  } sh;
  grid_dep_wait();
  grid_dep_trigger();
  if (static_cast<int>(blockIdx.x) < p.gate_blocks)
    gate_block(p, sh.zs);
  else
    copy_rows<T>(p, sh.places);
}

}  // namespace

static int row_units(const PagedArgs& a, bool with_q, bool f32) {
  return (2 * a.Hkv + (with_q ? a.H : 0)) * (a.d / (f32 ? Vec<float>::kN : Vec<__nv_bfloat16>::kN) / 2);
}

bool append_fits(const PagedArgs& a, bool with_q, bool f32) {
  return append_blocks(a, row_units(a, with_q, f32)).fit();
}

cudaError_t launch_cache_append(const CacheAppendArgs& x, bool f32, cudaStream_t s) {
  const AppendParams p = append_params(x);
  const int units = row_units(p.a, p.qn != nullptr, f32);
  return f32 ? launch_append(cache_append_kernel<float>, p, units, s)
             : launch_append(cache_append_kernel<__nv_bfloat16>, p, units, s);
}

}  // namespace fox
