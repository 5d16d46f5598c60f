// What the decode kernels and their merge share: the parameter block, the work line and the layout
// of the partial results.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_internal.h"
#include "fox_paged.h"
#include "fox_ptx.cuh"

namespace fox {

// Work on the shared prefix (fox_prefix.cu).
struct PrefixPlan {
  int hp, head_chunks;  // query heads of a row tile; such chunks of a key head's group
  int tpt;              // tokens of a row tile: its row r is token r / hp, head r % hp
  int row_tiles;        // of one key head: token blocks x head chunks, the chunks of a block side by side
  int items;            // of one key head: pairs of row tiles, or the only row tile
  int kap_tiles;        // gate terms of a stage: one set, or one a row tile
  int key_tiles;        // 0: no shared prefix
  int workers;
  float2* ml;           // [(worker + item) * 2 + stream][128] maximum (against c_last) and sum
  float* po;            // [(worker + item) * 2 + stream][128][d]
};

struct DecodeParams {
  PagedArgs a;
  const void* q;
  long long q_stride;  // elements from one row to the next
  float scale2;        // scale * log2 e
  int bias_from_j;
  int walk_prefix;     // the items walk the prefix's keys themselves (nothing shares it out)
  void* o;
  float* lse;
  // Own items
  int Rt, Rs, RTmax;   // rows of a row tile; rows kept of a slot; most row tiles of a sequence
  int Gp;              // rows of a token (padded_group)
  int workers, warps;  // workers, and of one CTA
  int* cum;            // [B + 1] units of one key head before each sequence, for the merge of a shared prefix
  uint32_t* count;     // [CTAs] arrivals at the item that reaches past this CTA's end; 0 between calls
  float2* ml;          // [slots][Rs] row maximum (log2 units) and sum of a partial result
  float* po;           // [slots][Rs][d] its weighted sum of V
  PrefixPlan pre;
};

// Unit offsets of the sequences into cum[0 .. B] (shared memory), by the whole block.
// `scratch` holds one value a warp. Ends with a block barrier.
__device__ __forceinline__ void scan_units(const DecodeParams& p, int* cum, int* scratch) {
  const PagedArgs& a = p.a;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = ceil_div(a.B, nt), b0 = tid * each, b1 = min(a.B, b0 + each);
  int mine = 0;
  bool any_bad = false;
  for (int b = b0; b < b1; ++b) {
    bool bad;
    const SeqInfo s = seq_info(a, b, &bad);
    any_bad |= bad;
    const int u = seq_units(a, s, p.Rt, p.Gp, p.walk_prefix);
    cum[b] = u;
    mine += u;
  }
  if (any_bad && blockIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int before = x - mine;
  for (int w = 0; w < warp; ++w) before += scratch[w];
  for (int b = b0; b < b1; ++b) {
    const int u = cum[b];
    cum[b] = before;
    before += u;
  }
  if (b0 < a.B && b1 == a.B) cum[a.B] = before;
  __syncthreads();
}

// The sequence whose units hold unit u of a key head (cum[b] <= u < cum[b + 1]).
__device__ __forceinline__ int find_seq(const int* cum, int B, int u) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A place on the work line: unit `tile` (of `tiles`) of item (hkv, b, rt).
struct Place {
  int hkv, b, rt, tile;
  int tiles, rts;  // key tiles and row tiles of the sequence
  SeqInfo s;
};

__device__ __forceinline__ void load_seq(const DecodeParams& p, Place& c) {
  bool bad;
  c.s = seq_info(p.a, c.b, &bad);
  c.tiles = ceil_div(walk_keys(p.a, c.s, p.walk_prefix), kKeyTile);
  c.rts = ceil_div(c.s.n * p.Gp, p.Rt);
}

// Unit u of the line (0 <= u < cum[B] * Hkv).
__device__ __forceinline__ Place place_of(const DecodeParams& p, const int* cum, int u) {
  Place c;
  const int per_head = cum[p.a.B];
  c.hkv = u / per_head;
  u -= c.hkv * per_head;
  c.b = find_seq(cum, p.a.B, u);
  load_seq(p, c);
  u -= cum[c.b];
  c.rt = u / c.tiles;
  c.tile = u - c.rt * c.tiles;
  return c;
}

// `by` units on, which the item has; then the next item's first unit, where that was its last and more
// units follow on the line.
__device__ __forceinline__ void advance(const DecodeParams& p, Place& c, int by, bool more) {
  c.tile += by;
  if (c.tile < c.tiles || !more) return;
  c.tile = 0;
  if (++c.rt < c.rts) return;
  c.rt = 0;
  do {
    if (++c.b == p.a.B) {
      c.b = 0;
      ++c.hkv;
    }
    load_seq(p, c);
  } while (c.tiles == 0 || c.rts == 0);
}

// A cumulative log gate (natural log) as an unevaluated sum of two fp32.
struct Gate2 {
  float hi, lo;
};
__device__ __forceinline__ Gate2 gate_sum(const PagedArgs& a, int page, int slot, int h) {
  const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
  const float g = a.g[g_offset(a, page, h, slot)];
  // base.x + g = s + e exactly (the rounding error of an fp32 sum is an fp32 value)
  const float s = __fadd_rn(base.x, g), t = __fsub_rn(s, base.x);
  const float e = __fadd_rn(__fsub_rn(base.x, __fsub_rn(s, t)), __fsub_rn(g, t));
  return {s, e + base.y};
}

// The page of own token p, page 0 with a report where the table has none.
__device__ __forceinline__ int own_page_or_0(const PagedArgs& a, int b, int p) {
  const int page = own_page(a, b, p);
  if (page < 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  return max(page, 0);
}

template <typename T>
__device__ __forceinline__ void put_out(T* dst, const float* f, int n);
template <>
__device__ __forceinline__ void put_out<float>(float* dst, const float* f, int n) {
  for (int i = 0; i < n; i += 2) *reinterpret_cast<float2*>(dst + i) = make_float2(f[i], f[i + 1]);
}
template <>
__device__ __forceinline__ void put_out<__nv_bfloat16>(__nv_bfloat16* dst, const float* f, int n) {
  for (int i = 0; i < n; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(f[i], f[i + 1]);
}

// Slot of a worker's partial result of an item, in rows of ml and po.
__device__ __forceinline__ size_t slot_of(const DecodeParams& p, int worker, int hkv, int b, int rt) {
  return (size_t)(worker + ((long long)hkv * p.a.B + b) * p.RTmax + rt) * p.Rs;
}

// ---- items that reach past one worker's range ----
// A worker's last segment of such an item stays in shared memory (`Kept`); a first segment whose item
// ends inside the worker's range goes to the worker's slot. At the end the block joins the kept segments
// of each item: to the output where the item lies in the block, else to the slot of the item's first
// worker in the block. An item then has one partial result a block, and one more where its last worker
// left a first segment and is not the first of its block. The block that brings the last of them joins
// them all, so that no second kernel is needed. The order of the sums is fixed, whoever joins.
template <int kRows, int kWarps>
struct Kept {
  int i0[kWarps];  // the kept segment's item, by its first unit; -1: none
  Place at[kWarps];
  float m[kWarps][kRows], l[kWarps][kRows];
};

constexpr int kJoinMost = 32;  // partial results whose weights stand in shared memory at a time

// One float4 column of one row of an item to O; with c4 == 0 the row's LSE as well.
template <typename T, int D>
__device__ __forceinline__ void put_column(const DecodeParams& p, const Place& at, int r, int c4, float4 v, float m, float l) {
  const int G = p.a.H / p.a.Hkv, rr = at.rt * p.Rt + r, t = rr / p.Gp, g = rr - t * p.Gp;
  if (g >= G) return;
  const size_t row = (size_t)(at.s.row0 + t) * p.a.H + at.hkv * G + g;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  put_out<T>(static_cast<T*>(p.o) + row * D + c4 * 4, o, 4);
  if (c4 == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Adds a partial result's column to (v, m, l), whose maximum follows.
__device__ __forceinline__ void add_column(float4& v, float& m, float& l, float4 x, float xm, float xl) {
  const float top = fmaxf(m, xm), safe = top == -INFINITY ? 0.f : top;
  const float a = ex2_approx(m - safe), b = ex2_approx(xm - safe);
  v.x = v.x * a + x.x * b;
  v.y = v.y * a + x.y * b;
  v.z = v.z * a + x.z * b;
  v.w = v.w * a + x.w * b;
  l = l * a + xl * b;
  m = top;
}

// By the whole block, at its end. Row r of warp w's kept segment lies at rows + w * warp_pitch + r * row_pitch
// (floats). `wgt`: [kJoinMost][kRows], `part`: [threads] of shared memory, clear of the kept rows.
// With a shared prefix every item is left to the merge that follows, its partial results as above.
template <typename T, int D, int kRows, int kWarps>
__device__ __forceinline__ void join_items(const DecodeParams& p, const int* cum, int total, int each,
                                           const Kept<kRows, kWarps>& kept, const float* rows, int warp_pitch,
                                           int row_pitch, float* wgt, float4* part) {
  constexpr int kThreads = 32 * kWarps, C4 = D / 4;
  __shared__ Place ends[2];
  __shared__ int first_block[2], blocks[2], last[2];
  __shared__ float row_m[kRows], row_l[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const bool shared = p.pre.key_tiles > 0;  // the merge with the prefix's results follows: nothing is final here
  __syncthreads();
  // 1. The kept segments of each item.
  for (int i = 0; i < kWarps; ++i) {
    const int i0 = kept.i0[i];
    if (i0 < 0 || (i > 0 && kept.i0[i - 1] == i0)) continue;
    int k1 = i + 1;
    while (k1 < kWarps && kept.i0[k1] == i0) ++k1;
    const Place& at = kept.at[i];
    const int i1 = i0 + at.tiles - 1, w1 = i1 / each;
    // the item's last worker left a first segment in its slot
    const bool more = min(total, (w1 + 1) * each) > i1 + 1;
    const bool here = !shared && i0 / each / kWarps == cta && w1 / kWarps == cta;
    const size_t slot = slot_of(p, cta * kWarps + i, at.hkv, at.b, at.rt);
    const size_t slot1 = slot_of(p, w1, at.hkv, at.b, at.rt);
    const int R = min(p.Rt, at.s.n * p.Gp - at.rt * p.Rt);
    for (int f = tid; f < R * C4; f += kThreads) {
      const int r = f / C4, c4 = f - r * C4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float m = -INFINITY, l = 0.f;
      for (int k = i; k < k1; ++k)
        add_column(v, m, l, *reinterpret_cast<const float4*>(rows + k * warp_pitch + r * row_pitch + c4 * 4), kept.m[k][r],
                   kept.l[k][r]);
      if (here) {
        if (more) {
          const float2 y = __ldcg(p.ml + slot1 + r);
          add_column(v, m, l, __ldcg(reinterpret_cast<const float4*>(p.po + (slot1 + r) * D) + c4), y.x, y.y);
        }
        put_column<T, D>(p, at, r, c4, v, m, l);
      } else {
        *reinterpret_cast<float4*>(p.po + (slot + r) * D + c4 * 4) = v;
        if (c4 == 0) p.ml[slot + r] = make_float2(m, l);
      }
    }
  }
  if (shared) return;
  // 2. The items that the block's range begins and ends inside of: at most one each, perhaps the same.
  const int U0 = min(total, cta * kWarps * each), U1 = min(total, U0 + kWarps * each);
  __syncthreads();
  if (tid < 2) {
    int f = -1, n = 0;
    if (U0 < U1) {
      const Place at = place_of(p, cum, tid ? U1 - 1 : U0);
      const int i0 = at.hkv * cum[p.a.B] + cum[at.b] + at.rt * at.tiles, i1 = i0 + at.tiles - 1;
      f = i0 / each / kWarps;
      n = i1 / each / kWarps - f + 1;
      if (tid == 0 ? i0 >= U0 : (i1 < U1 || i0 < U0)) n = 0;  // not cut at this end, or the other end's too
      ends[tid] = at;
    }
    int is_last = 0;
    if (n > 1) {
      __threadfence();
      if (static_cast<int>(atomicAdd(p.count + f, 1u)) + 1 == n) {
        p.count[f] = 0u;
        is_last = 1;
        __threadfence();
      }
    }
    first_block[tid] = f;
    blocks[tid] = n;
    last[tid] = is_last;
  }
  __syncthreads();
  for (int e = 0; e < 2; ++e) {
    if (!last[e]) continue;
    const Place& at = ends[e];
    const int i0 = at.hkv * cum[p.a.B] + cum[at.b] + at.rt * at.tiles, i1 = i0 + at.tiles - 1;
    const int w0 = i0 / each, w1 = i1 / each, c0 = first_block[e], nb = blocks[e], c1 = c0 + nb - 1;
    const int n = nb + (min(total, (w1 + 1) * each) > i1 + 1 && w1 > c1 * kWarps);
    const size_t slot = slot_of(p, 0, at.hkv, at.b, at.rt);
    // rows of ml and po where partial result k begins
    auto row_of = [&](int k) {
      const int w = k == 0 ? w0 : k < nb ? (c0 + k) * kWarps : w1;
      return slot + (size_t)w * p.Rs;
    };
    const int R = min(p.Rt, at.s.n * p.Gp - at.rt * p.Rt), F = R * C4;
    const int deal = F <= kThreads / 2 ? kThreads / F : 1, mine = deal > 1 ? tid / F : 0;
    for (int r = warp; r < R; r += kWarps) {
      float m = -INFINITY, l = 0.f;
      for (int k = lane; k < n; k += 32) {
        const float2 y = __ldcg(p.ml + row_of(k) + r);
        const float top = fmaxf(m, y.x), safe = top == -INFINITY ? 0.f : top;
        l = l * ex2_approx(m - safe) + y.y * ex2_approx(y.x - safe);
        m = top;
      }
      float top = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float safe = top == -INFINITY ? 0.f : top;
      l *= ex2_approx(m - safe);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) {
        row_m[r] = safe;
        row_l[r] = l;
      }
      // the first ones' weights
      if (lane < n) wgt[lane * kRows + r] = ex2_approx(__ldcg(p.ml + row_of(lane) + r).x - safe);
    }
    __syncthreads();
    // Columns of four channels; with few of them the partial results are dealt out to the threads too.
    for (int f = deal > 1 ? tid - mine * F : tid; f < F; f += kThreads) {
      if (mine >= deal) break;
      const int r = f / C4, c4 = f - r * C4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kBatch = 12;  // loads in flight
      for (int k = mine; k < n; k += kBatch * deal) {
        float4 y[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          y[j] = __ldcg(reinterpret_cast<const float4*>(p.po + (row_of(min(k + j * deal, n - 1)) + r) * D) + c4);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int kk = k + j * deal;
          float w = 0.f;
          if (kk < n)
            w = kk < kJoinMost ? wgt[kk * kRows + r] : ex2_approx(__ldcg(p.ml + row_of(kk) + r).x - row_m[r]);
          v.x = fmaf(w, y[j].x, v.x);
          v.y = fmaf(w, y[j].y, v.y);
          v.z = fmaf(w, y[j].z, v.z);
          v.w = fmaf(w, y[j].w, v.w);
        }
      }
      if (deal == 1)
        put_column<T, D>(p, at, r, c4, v, row_m[r], row_l[r]);
      else
        part[tid] = v;
    }
    __syncthreads();
    if (deal > 1 && tid < F) {
      float4 v = part[tid];
      for (int k = 1; k < deal; ++k) {
        const float4 y = part[k * F + tid];
        v.x += y.x;
        v.y += y.y;
        v.z += y.z;
        v.w += y.w;
      }
      const int r = tid / C4;
      put_column<T, D>(p, at, r, tid - r * C4, v, row_m[r], row_l[r]);
    }
    __syncthreads();
  }
}

// Rows of idle sequences: O = 0, LSE = -inf. The blocks share the sequences out.
template <typename T, int D>
__device__ __forceinline__ void clear_idle_rows(const DecodeParams& p) {
  for (int b = blockIdx.x; b < p.a.B; b += gridDim.x) {
    bool bad;
    const SeqInfo s = seq_info(p.a, b, &bad);
    if (s.own >= 0) continue;
    const size_t at = (size_t)s.row0 * p.a.H, n = (size_t)s.n * p.a.H;
    const float zero[2] = {0.f, 0.f};
    for (size_t e = threadIdx.x; e < n * (D / 2); e += blockDim.x) put_out<T>(static_cast<T*>(p.o) + at * D + 2 * e, zero, 2);
    for (size_t e = threadIdx.x; e < n; e += blockDim.x) p.lse[at + e] = -INFINITY;
  }
}

// The bf16 kernel on the tensor cores (fox_decode_mma.cu): its row tile for `rows` rows a sequence
// and key head, the workers of a CTA, its launch.
int decode_mma_rows(int rows);
int decode_mma_warps(int d);
cudaError_t launch_decode_mma(const DecodeParams& p, cudaStream_t s);
PrefixPlan prefix_plan(const PagedArgs& a);
cudaError_t launch_prefix(const DecodeParams& p, cudaStream_t s);

}  // namespace fox
