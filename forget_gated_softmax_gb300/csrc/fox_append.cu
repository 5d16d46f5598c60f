// Appending new tokens to the paged cache: K (rotated by its position where asked), V and the
// gates, in one launch, or two where a sequence can bring more tokens than a page holds.
//
// Rotation of the first `dim` channels of a head by the angles of the token's position, given as
// tables cos, sin [max_pos, dim / 2]:  (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin) with
// (a, b) = (i, i + dim / 2), or (2i, 2i + 1) with `pairs`. The products and the sum are fp32 and
// round once, to the cache's type.
//
// Gates: with a_t = log sigmoid(z_t), g of a token is the sum of a from its page's first token on
// (fp32) and gbase of a page the sum before it (fp64 arithmetic, kept as two fp32). A page's sums
// are a warp scan that goes on from the page's last held value; a page that opens in this call
// takes its base from the page before.
//
// Bound by memory: each of k, v (q) read once and written once. One thread makes one 16-byte chunk
// of the output; a rotated chunk reads its partner chunk as well, which another thread of the warp
// has in L1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_internal.h"
#include "fox_paged.h"
#include "fox_ptx.cuh"

namespace fox {
namespace {

constexpr int kThreads = 256;
constexpr int kGateHeads = 32;  // heads of one gate block

struct AppendParams {
  PagedArgs a;
  const void* kn;
  const void* vn;
  const float* z;
  const void* qn;
  void* qo;
  long long k_stride, v_stride, z_stride, q_stride;  // elements from one token to the next
  const float* cos;
  const float* sin;
  int max_pos, rot, pairs;
  int copy_blocks, blocks_per_row;  // blocks [0, copy_blocks) copy, the others scan gates
  int page_chunks, head_groups;     // gate block: (sequence, page chunk, head group)
  int scan_bases;                   // bases of pages after a sequence's first are left to base_scan_kernel
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// The chunk of channels [c, c + kN) of one head, rotated. `src` points at the head's channel 0.
template <typename T>
__device__ __forceinline__ uint4 turned_chunk(const T* src, int c, const float* cs, const float* sn, int rot,
                                              int pairs) {
  constexpr int kN = Vec<T>::kN;
  const uint4 w = *reinterpret_cast<const uint4*>(src + c);
  if (c >= rot) return w;
  float x[kN], y[kN];
  Vec<T>::unpack(w, x);
  if (pairs) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float co = cs[(c + i) / 2], si = sn[(c + i) / 2];
      y[i] = x[i] * co - x[i + 1] * si;
      y[i + 1] = x[i + 1] * co + x[i] * si;
    }
  } else {
    const int half = rot / 2;
    const bool low = c < half;
    float p[kN];
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + (low ? c + half : c - half)), p);
    const int a0 = low ? c : c - half;
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 co = *reinterpret_cast<const float4*>(cs + a0 + i);
      const float4 si = *reinterpret_cast<const float4*>(sn + a0 + i);
      const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i + j] = x[i + j] * cc[j] + (low ? -p[i + j] : p[i + j]) * ss[j];
    }
  }
  return Vec<T>::pack(y);
}

template <typename T>
__device__ __forceinline__ void copy_row(const AppendParams& p) {
  constexpr int kN = Vec<T>::kN;
  const PagedArgs& a = p.a;
  const int row = blockIdx.x / p.blocks_per_row, part = blockIdx.x % p.blocks_per_row;
  const int b = seq_of_row(a, row);
  if (b < 0) return;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (bad || row < s.row0 || row >= s.row0 + s.n) {
    if (bad && threadIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return;
  }
  if (s.own < 0) return;  // idle
  const int own = s.own - s.n + (row - s.row0);
  const int page = own_page(a, b, own), slot = own % a.page_size;
  const int pos = a.prefix_len + own;
  const bool no_page = page < 0, no_pos = p.rot > 0 && pos >= p.max_pos;
  if (no_page || no_pos) {
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return;
  }
  const int ch = a.d / kN;  // chunks of a head
  const int nk = a.Hkv * ch, nq = p.qn ? a.H * ch : 0;
  const float* cs = p.rot ? p.cos + (size_t)pos * (p.rot / 2) : nullptr;
  const float* sn = p.rot ? p.sin + (size_t)pos * (p.rot / 2) : nullptr;
  const T* kn = static_cast<const T*>(p.kn) + (size_t)row * p.k_stride;
  const T* vn = static_cast<const T*>(p.vn) + (size_t)row * p.v_stride;
  for (int u = part * kThreads + threadIdx.x; u < 2 * nk + nq; u += p.blocks_per_row * kThreads) {
    if (u < 2 * nk) {
      const int w = u < nk ? u : u - nk, h = w / ch, c = (w % ch) * kN;
      T* dst = static_cast<T*>(u < nk ? a.k : a.v) + kv_offset(a, page, h, slot) + c;
      const T* src = (u < nk ? kn : vn) + (size_t)h * a.d;
      const uint4 val = u < nk ? turned_chunk<T>(src, c, cs, sn, p.rot, p.pairs)
                               : *reinterpret_cast<const uint4*>(src + c);
      *reinterpret_cast<uint4*>(dst) = val;
    } else {
      const int w = u - 2 * nk, h = w / ch, c = (w % ch) * kN;
      const T* src = static_cast<const T*>(p.qn) + (size_t)row * p.q_stride + (size_t)h * a.d;
      *reinterpret_cast<uint4*>(static_cast<T*>(p.qo) + ((size_t)row * a.H + h) * a.d + c) =
          turned_chunk<T>(src, c, cs, sn, p.rot, p.pairs);
    }
  }
}

__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

// Log gates of tokens [t0, t0 + m) (rows row0 + t) and heads [h0, h0 + nh) into zs[token][head]; 0 past m.
__device__ __forceinline__ void stage_gates(const AppendParams& p, int row0, int m, int h0, int nh,
                                            float (*zs)[kGateHeads + 1]) {
  for (int e = threadIdx.x; e < m * kGateHeads; e += kThreads) {
    const int t = e / kGateHeads, h = e % kGateHeads;
    zs[t][h] = h < nh ? log_sigmoid(p.z[(size_t)(row0 + t) * p.z_stride + h0 + h]) : 0.f;
  }
}

// Inclusive sums of zs[0 .. m)[h] on top of `before`, four tokens a lane. The same sums, in the
// same order, whoever forms them.
__device__ __forceinline__ void scan_column(const float (*zs)[kGateHeads + 1], int m, int h, int lane, float before,
                                            float* incl) {
  float run = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = lane * 4 + e;
    run += t < m ? zs[t][h] : 0.f;
    incl[e] = run;
  }
  float x = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const float shift = before + (x - run);
#pragma unroll
  for (int e = 0; e < 4; ++e) incl[e] += shift;
}

__device__ __forceinline__ void put_base(float* gbase, size_t at, double c) {
  const float hi = static_cast<float>(c);
  *reinterpret_cast<float2*>(gbase + at) = make_float2(hi, static_cast<float>(c - static_cast<double>(hi)));
}

// c of the last token before own token `own`, head h: 0 where there is none.
__device__ __forceinline__ double gate_before(const PagedArgs& a, int b, int own, int h, bool* bad) {
  const int before = a.prefix_len + own - 1;
  if (before < 0) return 0.0;
  const int page = own > 0 ? own_page(a, b, own - 1) : prefix_page(a, before);
  if (page < 0) {
    *bad = true;
    return 0.0;
  }
  const int slot = (own > 0 ? own - 1 : before) % a.page_size;
  const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
  return static_cast<double>(base.x) + base.y + a.g[g_offset(a, page, h, slot)];
}

// Gates of the new tokens of one sequence that fall into one page.
__device__ __forceinline__ void gate_block(const AppendParams& p, float (*zs)[kGateHeads + 1]) {
  const PagedArgs& a = p.a;
  const int S = a.page_size;
  int idx = blockIdx.x - p.copy_blocks;
  const int hg = idx % p.head_groups;
  idx /= p.head_groups;
  const int chunk = idx % p.page_chunks, b = idx / p.page_chunks;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (bad) {
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return;
  }
  if (s.own < 0 || s.n == 0) return;
  const int first = s.own - s.n;                // own index of the first new token
  const int p0 = first / S * S;                 // first page's first token
  const int lo = max(first, p0 + chunk * S), hi = min(s.own, p0 + (chunk + 1) * S);
  if (lo >= hi) return;
  const int m = hi - lo, slot0 = lo % S;
  const int page = own_page(a, b, lo);
  const int page_before = chunk > 0 ? own_page(a, b, lo - 1) : 0;
  if (page < 0 || page_before < 0) {
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = hg * kGateHeads, nh = min(kGateHeads, a.H - h0);
  // With one page before this one in the call (no base scan follows), its new tokens are summed
  // here once more: their block may not have written yet. Its base and the value it goes on from
  // were there before the call, as it would otherwise hold a whole page of new tokens.
  const bool redo = chunk > 0 && !p.scan_bases;
  const int m1 = lo - first, slot1 = first % S;
  double open[kGateHeads / (kThreads / 32)];
  bool no_page = false;
  if (redo) {
    stage_gates(p, s.row0, m1, h0, nh, zs);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kGateHeads / (kThreads / 32); ++i) {
    const int hl = warp + i * (kThreads / 32), h = h0 + hl;
    open[i] = 0.0;
    if (hl >= nh) continue;
    if (redo) {
      float incl[4];
      const float was = slot1 > 0 ? a.g[g_offset(a, page_before, h, slot1 - 1)] : 0.f;
      scan_column(zs, m1, hl, lane, was, incl);
      // the sum over the whole page stands in lane 31, whatever m1 is
      const float last = __shfl_sync(0xffffffffu, incl[3], 31);
      if (slot1 > 0) {
        const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page_before, h));
        open[i] = static_cast<double>(base.x) + base.y + last;
      } else {
        open[i] = gate_before(a, b, first, h, &no_page) + last;
      }
    } else if (chunk == 0 && slot0 == 0) {
      open[i] = gate_before(a, b, first, h, &no_page);
    }
  }
  if (redo) __syncthreads();
  stage_gates(p, s.row0 + (lo - first), m, h0, nh, zs);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGateHeads / (kThreads / 32); ++i) {
    const int hl = warp + i * (kThreads / 32), h = h0 + hl;
    if (hl >= nh) continue;
    float incl[4];
    const float was = slot0 > 0 ? a.g[g_offset(a, page, h, slot0 - 1)] : 0.f;
    scan_column(zs, m, hl, lane, was, incl);
    float* dst = a.g + g_offset(a, page, h, slot0);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane * 4 + e < m) dst[lane * 4 + e] = incl[e];
    if (slot0 == 0 && (chunk == 0 || redo) && lane == 0) put_base(a.gbase, gbase_offset(a, page, h), open[i]);
  }
  if (no_page && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams p) {
  __shared__ float zs[128][kGateHeads + 1];
  grid_dep_trigger();
  if (static_cast<int>(blockIdx.x) < p.copy_blocks)
    copy_row<T>(p);
  else
    gate_block(p, zs);
}

// Bases of the pages after a sequence's first one: base_k = base_0 + sum of the full pages' sums.
// One warp a (sequence, head), 32 pages a step, fp64.
__global__ void __launch_bounds__(kThreads) base_scan_kernel(const AppendParams p) {
  grid_dep_wait();
  const PagedArgs& a = p.a;
  const int S = a.page_size;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)a.B * a.H) return;
  const int b = static_cast<int>(w / a.H), h = static_cast<int>(w % a.H);
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (s.own < 0 || s.n == 0) return;
  const int p0 = (s.own - s.n) / S, pl = (s.own - 1) / S;  // first and last page index of the new tokens
  if (pl == p0) return;
  const int id0 = own_page(a, b, p0 * S);
  if (id0 < 0) return;  // reported by its gate block
  const float2 base0 = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, id0, h));
  double carry = static_cast<double>(base0.x) + base0.y;
  for (int k = p0 + 1; k <= pl; k += 32) {
    const int kk = k + lane;
    const bool in = kk <= pl;
    const int prev = in ? own_page(a, b, (kk - 1) * S) : -1, id = in ? own_page(a, b, kk * S) : -1;
    double x = prev >= 0 ? static_cast<double>(a.g[g_offset(a, prev, h, S - 1)]) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (id >= 0) put_base(a.gbase, gbase_offset(a, id, h), carry + x);
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
}

template <typename T>
cudaError_t launch(AppendParams p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  const int units = (2 * a.Hkv + (p.qn ? a.H : 0)) * (a.d / Vec<T>::kN);
  // Up to four chunks a thread: fewer leave the row's index look-up standing out.
  p.blocks_per_row = ceil_div(units, 4 * kThreads);
  const long long copy = (long long)a.rows * p.blocks_per_row;
  p.page_chunks = ceil_div(a.max_new, a.page_size) + 1;
  p.head_groups = ceil_div(a.H, kGateHeads);
  p.scan_bases = a.max_new > a.page_size;
  const long long gates = (long long)a.B * p.page_chunks * p.head_groups;
  if (copy + gates > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.copy_blocks = static_cast<int>(copy);
  {
    TraceScope trace("cache_append", s);
    cache_append_kernel<T><<<static_cast<unsigned>(copy + gates), kThreads, 0, s>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.scan_bases) return e;
  const long long warps = (long long)a.B * a.H;
  {
    TraceScope trace("cache_base_scan", s);
    e = launch_dependent(base_scan_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(kThreads), 0, s, p);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& x, bool f32, cudaStream_t s) {
  AppendParams p = {};
  p.a = x.a;
  p.kn = x.k;
  p.vn = x.v;
  p.z = x.z;
  p.qn = x.q;
  p.qo = x.q_out;
  p.k_stride = x.k_stride;
  p.v_stride = x.v_stride;
  p.z_stride = x.z_stride;
  p.q_stride = x.q_stride;
  p.cos = x.cos;
  p.sin = x.sin;
  p.max_pos = x.max_pos;
  p.rot = x.rot;
  p.pairs = x.pairs;
  return f32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // namespace fox
