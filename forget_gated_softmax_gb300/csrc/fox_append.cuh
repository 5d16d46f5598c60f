// What the appends to the paged cache share, whatever K and V are held in: the parameter block, where a row goes, and the
// gates' running sums.
//
// Gates: with a_t = log sigmoid(z_t), g of a token is the sum of a from its page's first token on
// (fp32) and gbase of a page the sum before it (fp64 arithmetic, kept as two fp32). A page's sums
// go on from the page's last held value, token after token in two fp32 or, of many tokens, by a warp scan in
// fp32 on top of it; a page that opens in this call takes its base from the page before. A sum that
// goes on from g alone goes on from a rounded value: token by token, a_t below half a step of g are then
// lost one after the other. g_low holds what g leaves of the sum, so that every g is rounded once.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_cache.h"
#include "fox_ptx.cuh"

namespace fox {
namespace {

constexpr int kThreads = 128;
constexpr int kGateHeads = 32;  // heads of one gate block
constexpr int kFewTokens = 8;   // up to so many of a sequence are summed token after token, not by scans (one token of
                                // 128 sequences: 8.9 us, by scans 13.3; 8 of 32: 9.3 and 10.5; 16 of 32: 11.5 and 10.9)

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
  float* g_low;
  int gate_blocks;                  // blocks [0, gate_blocks) sum gates, the others copy
  int page_chunks, head_groups;     // gate block: (sequence, page chunk, head group)
  int scan_bases;                   // bases of pages after a sequence's first are left to base_scan_kernel
};

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
    if (bad) x = {-1, 0, 0};
  }
  if (bad && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  return x;
}

__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

// Log gates of tokens [t0, t0 + m) (rows row0 + t) and heads [h0, h0 + nh) into zs[token][head]; 0 past m.
__device__ __forceinline__ void stage_gates(const AppendParams& p, int row0, int m, int h0, int nh,
                                            float (*zs)[kGateHeads + 1]) {
#pragma unroll 4
  for (int e = threadIdx.x; e < m * kGateHeads; e += kThreads) {
    const int t = e / kGateHeads, h = e % kGateHeads;
    zs[t][h] = h < nh ? log_sigmoid(p.z[(size_t)(row0 + t) * p.z_stride + h0 + h]) : 0.f;
  }
}

// Inclusive sums of zs[0 .. m)[h], four tokens a lane: token t's in lane t / 4, incl[t % 4]. The same sums, in the
// same order, whoever forms them (further lanes' are of another order, also where they add zeros).
__device__ __forceinline__ void scan_column(const float (*zs)[kGateHeads + 1], int m, int h, int lane, float* incl) {
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
  const float shift = x - run;
#pragma unroll
  for (int e = 0; e < 4; ++e) incl[e] += shift;
}

// A page's running sum in two fp32, |lo| at most half a step of hi.
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 add(Sum2 x, float a) {
  const float s = __fadd_rn(x.hi, a), t = __fsub_rn(s, x.hi);
  const float e = __fadd_rn(__fsub_rn(x.hi, __fsub_rn(s, t)), __fsub_rn(a, t)) + x.lo;  // x.hi + a = s + rounding error
  const float hi = __fadd_rn(s, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s))};
}
// What a page's slot holds: g and, where it is kept, what g leaves of the sum. That is at most half a step of g;
// anything else there (of a page's earlier use, or never written) is no such thing and counts as 0.
__device__ __forceinline__ Sum2 held_sum(const AppendParams& p, size_t at) {
  const float g = p.a.g[at], low = p.g_low ? p.g_low[at] : 0.f;
  return {g, fabsf(low) <= fabsf(g) * 0x1p-24f ? low : 0.f};
}
// The value of a sum that goes to a slot, as the slot will hold it.
__device__ __forceinline__ double as_held(const AppendParams& p, Sum2 x) {
  return p.g_low ? static_cast<double>(x.hi) + x.lo : static_cast<double>(x.hi);
}
__device__ __forceinline__ void put_sum(const AppendParams& p, size_t at, Sum2 x) {
  p.a.g[at] = x.hi;
  if (p.g_low) p.g_low[at] = x.lo;
}

__device__ __forceinline__ void put_base(float* gbase, size_t at, double c) {
  const float hi = static_cast<float>(c);
  *reinterpret_cast<float2*>(gbase + at) = make_float2(hi, static_cast<float>(c - static_cast<double>(hi)));
}

__device__ __forceinline__ double base_of(const PagedArgs& a, int page, int h) {
  const float2 x = __ldcg(reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h)));
  return static_cast<double>(x.x) + x.y;
}

// c of the last token before own token `own`, head h: 0 where there is none.
__device__ __forceinline__ double gate_before(const AppendParams& p, int b, int own, int h, bool* bad) {
  const PagedArgs& a = p.a;
  const int before = a.prefix_len + own - 1;
  if (before < 0) return 0.0;
  const int page = own > 0 ? own_page(a, b, own - 1) : prefix_page(a, before);
  if (page < 0) {
    *bad = true;
    return 0.0;
  }
  const int slot = (own > 0 ? own - 1 : before) & (a.page_size - 1);
  return base_of(a, page, h) + as_held(p, held_sum(p, g_offset(a, page, h, slot)));
}

// Gates of the new tokens of one sequence that fall into one page.
__device__ __forceinline__ void gate_block(const AppendParams& p, float (*zs)[kGateHeads + 1]) {
  const PagedArgs& a = p.a;
  const int S = a.page_size;
  int idx = blockIdx.x;
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
  const int p0 = first & ~(S - 1);              // first page's first token
  const int lo = max(first, p0 + chunk * S), hi = min(s.own, p0 + (chunk + 1) * S);
  if (lo >= hi) return;
  const int m = hi - lo, slot0 = lo & (S - 1);
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
  const bool redo = chunk > 0 && !p.scan_bases, opens = slot0 == 0 && (chunk == 0 || redo);
  const int m1 = redo ? lo - first : 0, slot1 = first & (S - 1);
  bool no_page = false;
  if (s.n <= kFewTokens) {
    // Steps of generation: a lane a head, token after token. By the sequence's count, not the block's, so that a page's
    // sum is the same where the next page's block forms it once more.
    if (warp > 0 || lane >= nh) return;
    const int h = h0 + lane;
    const float* z = p.z + (size_t)s.row0 * p.z_stride + h;
    Sum2 run = {0.f, 0.f};
    if (slot0 > 0) run = held_sum(p, g_offset(a, page, h, slot0 - 1));
    if (opens) {
      double c = redo && slot1 > 0 ? base_of(a, page_before, h) : gate_before(p, b, first, h, &no_page);
      Sum2 before = {0.f, 0.f};
      if (redo && slot1 > 0) before = held_sum(p, g_offset(a, page_before, h, slot1 - 1));
#pragma unroll 1
      for (int t = 0; t < m1; ++t) before = add(before, log_sigmoid(z[(size_t)t * p.z_stride]));
      put_base(a.gbase, gbase_offset(a, page, h), c + as_held(p, before));
    }
    const size_t dst = g_offset(a, page, h, slot0);
    z += (size_t)(lo - first) * p.z_stride;
#pragma unroll 1
    for (int t = 0; t < m; ++t) {
      run = add(run, log_sigmoid(z[(size_t)t * p.z_stride]));
      put_sum(p, dst + t, run);
    }
    if (no_page && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return;
  }
  if (opens) {
    if (redo) {
      stage_gates(p, s.row0, m1, h0, nh, zs);
      __syncthreads();
    }
#pragma unroll 2
    for (int hl = warp; hl < nh; hl += kThreads / 32) {
      const int h = h0 + hl;
      double c = redo && slot1 > 0 ? base_of(a, page_before, h) : gate_before(p, b, first, h, &no_page);
      if (redo) {
        float incl[4];
        scan_column(zs, m1, hl, lane, incl);
        const int t = (m1 - 1) & 3;  // of the page's last token, as its block writes it
        const float sum = __shfl_sync(0xffffffffu, t < 2 ? (t ? incl[1] : incl[0]) : t < 3 ? incl[2] : incl[3], (m1 - 1) >> 2);
        c += slot1 > 0 ? as_held(p, add(held_sum(p, g_offset(a, page_before, h, slot1 - 1)), sum)) : sum;
      }
      if (lane == 0) put_base(a.gbase, gbase_offset(a, page, h), c);
    }
    if (redo) __syncthreads();
  }
  stage_gates(p, s.row0 + (lo - first), m, h0, nh, zs);
  __syncthreads();
#pragma unroll 2
  for (int hl = warp; hl < nh; hl += kThreads / 32) {
    const int h = h0 + hl;
    float incl[4];
    scan_column(zs, m, hl, lane, incl);
    const size_t dst = g_offset(a, page, h, slot0);
    if (slot0 == 0) {  // all but a sequence's first page: the scan's sums as they are
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane * 4 + e < m) a.g[dst + lane * 4 + e] = incl[e];
      if (p.g_low) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (lane * 4 + e < m) p.g_low[dst + lane * 4 + e] = 0.f;
      }
      continue;
    }
    const Sum2 before = held_sum(p, dst - 1);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane * 4 + e < m) put_sum(p, dst + lane * 4 + e, add(before, incl[e]));
  }
  if (no_page && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
}

// Bases of the pages after a sequence's first one: base_k = base_0 + sum of the full pages' sums.
// One warp a (sequence, head), 32 pages a step, fp64.
__global__ void __launch_bounds__(kThreads) base_scan_kernel(const AppendParams p) {
  grid_dep_trigger();
  // Lengths and tables are the caller's: only what the gates' blocks write has to be waited for.
  const PagedArgs& a = p.a;
  const int S = a.page_size;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const bool live = w < (long long)a.B * a.H;
  const int b = live ? static_cast<int>(w / a.H) : 0, h = live ? static_cast<int>(w % a.H) : 0;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  const int p0 = (s.own - s.n) / S, pl = (s.own - 1) / S;  // first and last page index of the new tokens
  const int id0 = live && s.own >= 0 && s.n > 0 && pl > p0 ? own_page(a, b, p0 * S) : -1;
  if (id0 < 0) {  // nothing to do, or reported by its gate block
    grid_dep_wait();
    return;
  }
  double carry = 0.0;
  constexpr int kSteps = 4;  // of 32 pages, their loads in flight together
  for (int k = p0 + 1; k <= pl; k += 32 * kSteps) {
    float full[kSteps], low[kSteps];
    int id[kSteps], before[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int kk = k + 32 * i + lane;
      const int prev = kk <= pl ? own_page(a, b, (kk - 1) * S) : -1;
      id[i] = kk <= pl ? own_page(a, b, kk * S) : -1;
      before[i] = prev;
    }
    if (k == p0 + 1) {
      grid_dep_wait();
      carry = base_of(a, id0, h);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const size_t at = before[i] >= 0 ? g_offset(a, before[i], h, S - 1) : 0;
      full[i] = before[i] >= 0 ? __ldcg(a.g + at) : 0.f;
      low[i] = before[i] >= 0 && p.g_low ? __ldcg(p.g_low + at) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      double x = static_cast<double>(full[i]) + low[i];
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

// Sixteen bytes of a row as fp32 values.
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

constexpr int kRows = 4;                        // rows of a thread, their loads in flight together
constexpr int kBlockRows = kRows * kThreads / 8;  // most rows of a block (8 units a row at least)

// How a block's threads go over a row's units: a chunk of them, or, with fewer units than threads, several
// rows side by side.
struct CopyShape {
  int per_row, chunks, side;  // units of a row; chunks of a row; rows side by side
};
__host__ __device__ __forceinline__ CopyShape copy_shape(int per_row) {
  return {per_row, ceil_div(per_row, kThreads), per_row < kThreads ? kThreads / per_row : 1};
}

struct AppendBlocks {
  int page_chunks, head_groups;
  long long gates, copies;
  bool fit() const { return gates + copies <= 0x7fffffffLL; }  // a grid
};
inline AppendBlocks append_blocks(const PagedArgs& a, int row_units, int thread_rows = kRows) {
  const CopyShape x = copy_shape(row_units);
  AppendBlocks n;
  n.page_chunks = ceil_div(a.max_new, a.page_size) + 1;
  n.head_groups = ceil_div(a.H, kGateHeads);
  n.gates = (long long)a.B * n.page_chunks * n.head_groups;
  n.copies = (long long)ceil_div(a.rows, thread_rows * x.side) * x.chunks;
  return n;
}

inline AppendParams append_params(const CacheAppendArgs& x) {
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
  p.g_low = x.g_low;
  return p;
}

// The launches of one append by `kernel`, whose blocks behind the gates' copy rows of `row_units` units each, `thread_rows` a
// thread; Params is AppendParams or has it as its base.
template <typename Params>
cudaError_t launch_append(void (*kernel)(const Params), Params p, int row_units, cudaStream_t s, int thread_rows = kRows) {
  const PagedArgs& a = p.a;
  const AppendBlocks n = append_blocks(a, row_units, thread_rows);
  p.page_chunks = n.page_chunks;
  p.head_groups = n.head_groups;
  p.scan_bases = a.max_new > a.page_size;
  p.gate_blocks = static_cast<int>(n.gates);
  cudaError_t e;
  {
    TraceScope trace("cache_append", s);
    e = launch_dependent(kernel, dim3(static_cast<unsigned>(n.gates + n.copies)), dim3(kThreads), 0, s, p);
  }
  if (e == cudaSuccess && p.scan_bases) {
    TraceScope trace("cache_base_scan", s);
    const long long warps = (long long)a.B * a.H;
    e = launch_dependent(base_scan_kernel, dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32))),
                         dim3(kThreads), 0, s, static_cast<const AppendParams&>(p));
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace fox
