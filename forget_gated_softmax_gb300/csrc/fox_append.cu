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
// Gates: with a_t = log sigmoid(z_t), g of a token is the sum of a from its page's first token on
// (fp32) and gbase of a page the sum before it (fp64 arithmetic, kept as two fp32). A page's sums
// go on from the page's last held value, token after token in two fp32 or, of many tokens, by a warp scan in
// fp32 on top of it; a page that opens in this call takes its base from the page before. A sum that
// goes on from g alone goes on from a rounded value: token by token, a_t below half a step of g are then
// lost one after the other. g_low holds what g leaves of the sum, so that every g is rounded once.
//
// Bound by memory: each of k, v (q) read once and written once. 6 prompts of up to 16384 tokens (1.44 GB) take
// 258 us, 5.6 TB/s (262 with g_low); one token of 128 sequences 4.0 us of GPU time among others in a graph, the launch and a
// few dependent trips to memory (with and without g_low).
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

struct AppendBlocks {
  int page_chunks, head_groups;
  long long gates, copies;
};
AppendBlocks append_blocks(const PagedArgs& a, bool with_q, int vec) {
  const CopyShape x = copy_shape((2 * a.Hkv + (with_q ? a.H : 0)) * (a.d / vec / 2));
  AppendBlocks n;
  n.page_chunks = ceil_div(a.max_new, a.page_size) + 1;
  n.head_groups = ceil_div(a.H, kGateHeads);
  n.gates = (long long)a.B * n.page_chunks * n.head_groups;
  n.copies = (long long)ceil_div(a.rows, kRows * x.side) * x.chunks;
  return n;
}

template <typename T>
cudaError_t launch(AppendParams p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  const AppendBlocks n = append_blocks(a, p.qn != nullptr, Vec<T>::kN);
  const long long gates = n.gates, copy = n.copies;
  p.page_chunks = n.page_chunks;
  p.head_groups = n.head_groups;
  p.scan_bases = a.max_new > a.page_size;
  p.gate_blocks = static_cast<int>(gates);
  cudaError_t e;
  {
    TraceScope trace("cache_append", s);
    e = launch_dependent(cache_append_kernel<T>, dim3(static_cast<unsigned>(gates + copy)), dim3(kThreads), 0, s, p);
  }
  if (e == cudaSuccess && p.scan_bases) {
    TraceScope trace("cache_base_scan", s);
    const long long warps = (long long)a.B * a.H;
    e = launch_dependent(base_scan_kernel, dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32))),
                         dim3(kThreads), 0, s, p);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool append_fits(const PagedArgs& a, bool with_q, bool f32) {
  const AppendBlocks n = append_blocks(a, with_q, f32 ? Vec<float>::kN : Vec<__nv_bfloat16>::kN);
  return n.gates + n.copies <= 0x7fffffffLL;
}

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
  p.g_low = x.g_low;
  return f32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // namespace fox
