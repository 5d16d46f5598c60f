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
// Bound by memory: each of k, v (q) read once and written once.
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
  int copy_blocks;                  // blocks [0, copy_blocks) copy, the others scan gates
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

// Work of the copy: units of two 16-byte chunks of one head of a row, (k, v, q heads) x (chunk pairs). A
// pair is a channel range and its partner in the rotation, so that each chunk is read once; channels that
// are not rotated, or whose partners are in the same chunk, go in neighbouring pairs.
__device__ __forceinline__ void pair_of(int j, int rot_chunks, bool apart, int* c0, int* c1) {
  const bool turned = apart && 2 * j < rot_chunks;
  *c0 = turned ? j : 2 * j;
  *c1 = turned ? j + rot_chunks / 2 : 2 * j + 1;
}

// Rotates two chunks (x at channel c0, y at c1 of the head).
template <typename T>
__device__ __forceinline__ void turn(uint4& wx, uint4& wy, int c0, int c1, const float* cs, const float* sn, int rot,
                                     int pairs) {
  constexpr int kN = Vec<T>::kN;
  if (c0 >= rot) return;
  float x[kN], y[kN], u[kN], v[kN];
  Vec<T>::unpack(wx, x);
  Vec<T>::unpack(wy, y);
  if (pairs) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float ca = cs[(c0 + i) / 2], sa = sn[(c0 + i) / 2], cb = cs[(c1 + i) / 2], sb = sn[(c1 + i) / 2];
      u[i] = x[i] * ca - x[i + 1] * sa;
      u[i + 1] = x[i + 1] * ca + x[i] * sa;
      v[i] = y[i] * cb - y[i + 1] * sb;
      v[i + 1] = y[i + 1] * cb + y[i] * sb;
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

// Where a row's copies go.
struct RowPlace {
  int page, slot, pos;  // page -1: the row is not appended
};

__device__ __forceinline__ RowPlace row_place(const AppendParams& p, int row) {
  const PagedArgs& a = p.a;
  RowPlace x = {-1, 0, 0};
  const int b = seq_of_row(a, row);
  if (b < 0) return x;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (!bad && row >= s.row0 && row < s.row0 + s.n && s.own >= 0) {
    const int own = s.own - s.n + (row - s.row0);
    x.page = own_page(a, b, own);
    x.slot = own & (a.page_size - 1);
    x.pos = a.prefix_len + own;
    bad = x.page < 0 || (p.rot > 0 && x.pos >= p.max_pos);
    if (bad) x.page = -1;
  }
  if (bad && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  return x;
}

constexpr int kUnits = 4;                  // units of a thread, their loads in flight together
constexpr int kBlockRows = kThreads * kUnits / 8 + 2;  // most rows that a block's units touch (8 a row at least)

// A block's units lie side by side on the line of all rows' units. The loads of k, v, q need only that; they
// are asked for first, and the look-ups of the rows' pages and positions run meanwhile.
template <typename T>
__device__ __forceinline__ void copy_units(const AppendParams& p, RowPlace* places) {
  constexpr int kN = Vec<T>::kN;
  const PagedArgs& a = p.a;
  const int hs = (kN == 8 ? 2 : 3) + (a.d == 128), hp = 1 << hs;  // units of a head
  const int nk = a.Hkv * hp, per_row = 2 * nk + (p.qn ? a.H * hp : 0);
  const long long first = (long long)blockIdx.x * (kThreads * kUnits);
  const int row0 = first < 0x7fffffffLL ? static_cast<int>(first) / per_row : static_cast<int>(first / per_row);
  const int off = static_cast<int>(first - (long long)row0 * per_row);
  const int rot_chunks = p.rot / kN;
  uint4 x[kUnits], y[kUnits];
  int row[kUnits], at[kUnits];  // at: the unit in its row
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = off + i * kThreads + threadIdx.x;
    row[i] = u / per_row;
    at[i] = u - row[i] * per_row;
    const int w = at[i] < nk ? at[i] : at[i] < 2 * nk ? at[i] - nk : at[i] - 2 * nk;
    int c0, c1;
    pair_of(w & (hp - 1), at[i] >= nk && at[i] < 2 * nk ? 0 : rot_chunks, !p.pairs, &c0, &c1);
    const bool is_v = at[i] >= nk && at[i] < 2 * nk, is_q = at[i] >= 2 * nk;
    const T* src = static_cast<const T*>(is_q ? p.qn : is_v ? p.vn : p.kn) +
                   (size_t)(row0 + row[i]) * (is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride) + (size_t)(w >> hs) * a.d;
    if (row0 + row[i] < a.rows) {
      x[i] = __ldcs(reinterpret_cast<const uint4*>(src + c0 * kN));
      y[i] = __ldcs(reinterpret_cast<const uint4*>(src + c1 * kN));
    }
  }
  const int rows = min((off + kThreads * kUnits - 1) / per_row + 1, a.rows - row0);
  for (int r = threadIdx.x; r < rows; r += kThreads) places[r] = row_place(p, row0 + r);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (row0 + row[i] >= a.rows) continue;
    const RowPlace g = places[row[i]];
    if (g.page < 0) continue;
    const bool is_v = at[i] >= nk && at[i] < 2 * nk, is_q = at[i] >= 2 * nk;
    const int w = is_q ? at[i] - 2 * nk : is_v ? at[i] - nk : at[i], h = w >> hs;
    int c0, c1;
    pair_of(w & (hp - 1), is_v ? 0 : rot_chunks, !p.pairs, &c0, &c1);
    if (!is_v && p.rot)
      turn<T>(x[i], y[i], c0 * kN, c1 * kN, p.cos + (size_t)g.pos * (p.rot / 2), p.sin + (size_t)g.pos * (p.rot / 2), p.rot,
              p.pairs);
    T* dst = is_q ? static_cast<T*>(p.qo) + ((size_t)(row0 + row[i]) * a.H + h) * a.d
                  : static_cast<T*>(is_v ? a.v : a.k) + kv_offset(a, g.page, h, g.slot);
    *reinterpret_cast<uint4*>(dst + c0 * kN) = x[i];
    *reinterpret_cast<uint4*>(dst + c1 * kN) = y[i];
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
  __shared__ union {
    float zs[128][kGateHeads + 1];
    RowPlace places[kBlockRows];
  } sh;
  grid_dep_trigger();
  if (static_cast<int>(blockIdx.x) < p.copy_blocks)
    copy_units<T>(p, sh.places);
  else
    gate_block(p, sh.zs);
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
  constexpr int kSteps = 4;  // of 32 pages, their loads in flight together
  for (int k = p0 + 1; k <= pl; k += 32 * kSteps) {
    float full[kSteps];
    int id[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int kk = k + 32 * i + lane;
      const int prev = kk <= pl ? own_page(a, b, (kk - 1) * S) : -1;
      id[i] = kk <= pl ? own_page(a, b, kk * S) : -1;
      full[i] = prev >= 0 ? a.g[g_offset(a, prev, h, S - 1)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      double x = full[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (id[i] >= 0) put_base(a.gbase, gbase_offset(a, id[i], h), carry + x);
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
}

template <typename T>
cudaError_t launch(AppendParams p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  const long long units = (long long)a.rows * ((2 * a.Hkv + (p.qn ? a.H : 0)) * (a.d / Vec<T>::kN / 2));
  const long long copy = (units + kThreads * kUnits - 1) / (kThreads * kUnits);
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
