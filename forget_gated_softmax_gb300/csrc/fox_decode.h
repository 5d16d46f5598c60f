// What the decode kernels and their merge share: the parameter block, the work line and the layout
// of the partial results.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_cache.h"
#include "fox_ptx.cuh"

namespace fox {

// Work on the shared prefix (fox_prefix.cu).
struct PrefixPlan {
  int hp, head_chunks;  // query heads of a row tile; such chunks of a key head's group
  int tpt;              // tokens of a row tile: its row r is head r / tpt, token r % tpt
  int row_tiles;        // of one key head: token blocks x head chunks, the chunks of a block side by side
  int items;            // of one key head: pairs of row tiles, or the only row tile
  int kap_tiles;        // gate terms of a stage: one set, or one a row tile
  int key_tiles;        // 0: no shared prefix
  int line, each;       // units of an item on the work line (its key tiles, then perhaps empty ones); of a CTA
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
  const uint8_t* ks;   // scales of a 4-bit cache
  const uint8_t* vs;
  // Own items
  int Rt, Rs;          // rows of a row tile; rows kept of a slot
  Numbering num;       // of the items
  int Gp;              // rows of a token (padded_group)
  uint32_t gp_inv;     // ceil(2^32 / Gp), for token_of; 0: Gp is 1
  int workers, warps;  // workers, and of one CTA
  int* cum;            // [B + 1] units of one key head before each sequence, for the merge of a shared prefix
  uint32_t* count;     // [CTAs] arrivals at the item that reaches past this CTA's end; 0 between calls
  float2* ml;          // [slots][Rs] row maximum (log2 units) and sum of a partial result
  float* po;           // [slots][Rs][d] its weighted sum of V
  PrefixPlan pre;
};

// Row r's token: r / Gp by a multiplication (exact while max_new * Gp^2 < 2^32, which decode_fits checks).
__device__ __forceinline__ int token_of(const DecodeParams& p, int r) {
  return p.gp_inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.gp_inv)) : r;
}

// The sequences as every CTA holds them in shared memory, [B + 1]: units of one key head before the
// sequence, its first row (its rows end where the next one's begin), its tokens after the prefix (SeqInfo;
// kBadSeq: left out). The kernels run most of their code once a launch, and then wait for instructions as
// much as for data: what they look up is made compact here once.
struct SeqEntry {
  int u0, row0, own;
};
constexpr int kBadSeq = -2;
struct Seq {
  int u0, row0, n, own;
};

// The end of the rows of all sequences before b0, which are those that the threads before this one have. Apart from the
// code that most calls run.
static __device__ __noinline__ int rows_before(const DecodeParams& p, int b0, int b1, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int end = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    bool bad;
    const SeqInfo s = seq_info(p.a, b, &bad);  // without rows where bad
    end = max(end, s.row0 + s.n);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end = max(end, y);
  }
  if (lane == 31) scratch[warp] = end;
  end = __shfl_up_sync(0xffffffffu, end, 1);
  if (lane == 0) end = 0;
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < warp; ++w) end = max(end, scratch[w]);
  __syncthreads();
  return end;
}

// Fills seqs[0 .. B] by the whole block; `scratch` holds one value a warp. Ends with a block barrier. Where items are
// numbered by rows, a sequence whose rows begin before the end of an earlier one's is left out.
__device__ __forceinline__ void scan_sequences(const DecodeParams& p, SeqEntry* seqs, int* scratch) {
  const PagedArgs& a = p.a;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = ceil_div(a.B, nt), b0 = tid * each, b1 = min(a.B, b0 + each);
  int mine = 0, rows_end = 0;
  bool any_bad = false;
  if (p.num.by_rows()) rows_end = rows_before(p, b0, b1, scratch);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    bool bad;
    SeqInfo s = seq_info(a, b, &bad);
    if (p.num.by_rows() && !bad) {
      if (s.row0 < rows_end) {
        bad = true;
        s = {0, 0, -1};
      }
      rows_end = max(rows_end, s.row0 + s.n);
    }
    any_bad |= bad;
    seqs[b] = {mine, first_row(a, b), bad ? kBadSeq : s.own};
    mine += seq_units(a, s, p.Rt, p.Gp, p.walk_prefix);
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
#pragma unroll 1
  for (int w = 0; w < warp; ++w) before += scratch[w];
#pragma unroll 1
  for (int b = b0; b < b1; ++b) seqs[b].u0 += before;
  if (b0 < a.B && b1 == a.B) seqs[a.B] = {before + mine, first_row(a, a.B), kBadSeq};
  __syncthreads();
}

// A place on the work line: unit `tile` (of `tiles`) of item (hkv, b, rt).
struct Place {
  int hkv, b, rt, tile;
  int tiles, rts;  // key tiles and row tiles of the sequence
  int i0;          // the item's first unit
  Seq s;
};

__device__ __forceinline__ void load_seq(const DecodeParams& p, const SeqEntry* seqs, Place& c) {
  const SeqEntry e = seqs[c.b];
  c.s = {e.u0, e.row0, seqs[c.b + 1].row0 - e.row0, e.own};
  c.tiles = walk_tiles(p.a, c.s.own, p.walk_prefix);
  c.rts = (c.s.n * p.Gp + p.Rt - 1) / p.Rt;
}

// Unit u of the line (0 <= u < total).
static __device__ __noinline__ Place place_of(const DecodeParams& p, const SeqEntry* seqs, int u) {
  Place c;
  const int per_head = seqs[p.a.B].u0;
  c.hkv = u / per_head;
  const int in_head = u - c.hkv * per_head;
  int lo = 0, hi = p.a.B;  // seqs[lo].u0 <= in_head < seqs[hi].u0
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seqs[mid].u0 <= in_head)
      lo = mid;
    else
      hi = mid;
  }
  c.b = lo;
  load_seq(p, seqs, c);
  const int in_seq = in_head - c.s.u0;
  c.rt = in_seq / c.tiles;
  c.tile = in_seq - c.rt * c.tiles;
  c.i0 = u - c.tile;
  return c;
}

// The first unit of the next item; there is one.
static __device__ __noinline__ void next_item(const DecodeParams& p, const SeqEntry* seqs, Place& c) {
  c.i0 += c.tiles;
  c.tile = 0;
  if (++c.rt < c.rts) return;
  c.rt = 0;
#pragma unroll 1
  do {
    if (++c.b == p.a.B) {
      c.b = 0;
      ++c.hkv;
    }
    load_seq(p, seqs, c);
  } while (c.tiles == 0 || c.rts == 0);
}

// A cumulative log gate (natural log) as an unevaluated sum of two fp32.
struct Gate2 {
  float hi, lo;
};
__device__ __forceinline__ Gate2 gate_sum(float2 base, float g) {
  // base.x + g = s + e exactly (the rounding error of an fp32 sum is an fp32 value)
  const float s = __fadd_rn(base.x, g), t = __fsub_rn(s, base.x);
  const float e = __fadd_rn(__fsub_rn(base.x, __fsub_rn(s, t)), __fsub_rn(g, t));
  return {s, e + base.y};
}
__device__ __forceinline__ Gate2 gate_sum(const PagedArgs& a, int page, int slot, int h) {
  return gate_sum(*reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h)), a.g[g_offset(a, page, h, slot)]);
}

// A table entry as a page; page 0 with a report where it is none.
__device__ __forceinline__ int checked_page(const PagedArgs& a, int id) {
  const bool ok = id >= 0 && id < a.num_pages;
  if (!ok && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  return ok ? id : 0;
}
// The page of own token p, page 0 with a report where the table has none.
__device__ __forceinline__ int own_page_or_0(const PagedArgs& a, int b, int p) {
  const int page = own_page(a, b, p);
  if (page < 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  return max(page, 0);
}

// ---- asynchronous copies to shared memory, in groups of the thread ----
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where there are none to copy (src is then not read).
__device__ __forceinline__ void cp_async16_or_0(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// K and V pass through the L2 cache as what may go first, also where other row tiles, or other sequences behind the
// same prefix, read them again: what every call needs again (its code, the tables, partial results) then stays. One
// sequence of 65536 tokens: 56.1 -> 52.9 us; 32 behind 16384 shared ones, by the prefix kernel: 53.2 -> 52.3. Read again,
// without the hint and with it: 16 sequences of 4096 with 28 rows a key head (two row tiles) 117.2 and 114.0, with 64 (four)
// 215 and 208; one of 2048 with 2048 new tokens 776 and 777; 8 behind 2000 walked shared tokens 24.5 and 24.3; 256 behind 32768
// (four items a key head) 183 and 184.
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t x;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(x));
  return x;
}
__device__ __forceinline__ void tma_load_4d_by(uint64_t policy, void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                               int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

template <int D, int NT>
struct MmaLayout {
  static constexpr int kWarps = D == 128 ? 4 : 8;
  // 128 KB on the way to an SM. A third stage measured no faster where bandwidth decides, and the SMs'
  // shares of it less equal, so that the last finished later (one sequence of 65536: 52 against 49 us).
  static constexpr int kStages = 2;
  static constexpr int kRows = 8 * NT;
  static constexpr int kTileBytes = kKeyTile * D * 2;  // K or V of a stage
  static constexpr int kQBytes = kRows * D * 2;        // an item's Q: chunk c (16 bytes) of row r at c ^ (r & 7)
  static constexpr int kOutStride = D + 4;             // a result row in shared memory, in floats
  static_assert(kRows * kOutStride * 4 <= 2 * kTileBytes, "results pass through a stage that was read");
};

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Four channels to O.
template <typename T>
__device__ __forceinline__ void put4(T* dst, float4 v);
template <>
__device__ __forceinline__ void put4<float>(float* dst, float4 v) {
  *reinterpret_cast<float4*>(dst) = v;
}
template <>
__device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16* dst, float4 v) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Slot of a worker's partial result of an item, in rows of ml and po.
__device__ __forceinline__ int slot_of(const DecodeParams& p, int worker, const Place& at) {
  return (worker + at.hkv * p.num.items + first_item(p.num, at.b, at.s.row0) + at.rt) * p.Rs;
}
// Rows that a row tile has.
__device__ __forceinline__ int rows_of(const DecodeParams& p, const Place& at) {
  return min(p.Rt, at.s.n * p.Gp - at.rt * p.Rt);
}

// One float4 column of a row of an item to O, and with c4 == 0 the row's LSE.
template <typename T, int D>
__device__ __noinline__ void put_column(const DecodeParams& p, const Place& at, int r, int c4, float4 v, float m, float l) {
  const int G = p.a.H / p.a.Hkv, rr = at.rt * p.Rt + r, t = token_of(p, rr), g = rr - t * p.Gp;
  if (g >= G) return;  // an empty row
  const size_t row = (size_t)(at.s.row0 + t) * p.a.H + at.hkv * G + g;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  put4<T>(static_cast<T*>(p.o) + row * D + c4 * 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
  if (c4 == 0) p.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
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
  float m[kWarps][kRows], l[kWarps][kRows];  // of the warp's latest segment
};

// A finished segment's rows (rows + r * pitch, floats of shared memory), of these r0 to r1 - 1, by one warp: to O where the worker
// had the whole item, else to its slot.
template <typename T, int D>
__device__ __forceinline__ void leave_rows(const DecodeParams& p, const Place& at, int worker, bool whole, const float* rows,
                                           int pitch, const float* m, const float* l, int r0 = 0, int r1 = 1 << 16) {
  constexpr int C4 = D / 4;
  const int lane = threadIdx.x & 31, slot = slot_of(p, worker, at), F = min(rows_of(p, at), r1) * C4;
#pragma unroll 1
  for (int f = r0 * C4 + lane; f < F; f += 32) {
    const int r = f / C4, c4 = f % C4;
    const float4 v = *reinterpret_cast<const float4*>(rows + r * pitch + c4 * 4);
    if (whole) {
      put_column<T, D>(p, at, r, c4, v, m[r], l[r]);
    } else {
      *reinterpret_cast<float4*>(p.po + (size_t)(slot + r) * D + c4 * 4) = v;
      if (c4 == 0) p.ml[slot + r] = make_float2(m[r], l[r]);
    }
  }
}

// Columns with their row's maximum and sum, joined to one.
struct Column {
  float4 v;
  float m, l;
};
__device__ __forceinline__ void add_column(Column& a, float4 x, float xm, float xl) {
  const float top = fmaxf(a.m, xm), safe = top == -INFINITY ? 0.f : top;
  const float s = ex2_approx(a.m - safe), t = ex2_approx(xm - safe);
  a.v.x = a.v.x * s + x.x * t;
  a.v.y = a.v.y * s + x.y * t;
  a.v.z = a.v.z * s + x.z * t;
  a.v.w = a.v.w * s + x.w * t;
  a.l = a.l * s + xl * t;
  a.m = top;
}

// The items that a block's range of the line begins and ends inside of: at most one each, perhaps the same.
struct BlockEnds {
  Place at[2];
  int first[2], blocks[2];  // first CTA of the item; its CTAs, 0 where none is cut there (or it is the other end's)
};
template <int kWarps>
__device__ __forceinline__ void find_ends(const DecodeParams& p, const SeqEntry* seqs, int total, int each, BlockEnds& x) {
  const int tid = threadIdx.x, U0 = min(total, static_cast<int>(blockIdx.x) * kWarps * each);
  const int U1 = min(total, U0 + kWarps * each);
  if (tid >= 2) return;
  int first = 0, blocks = 0;
  if (U0 < U1) {
    const Place at = place_of(p, seqs, tid ? U1 - 1 : U0);
    const int i1 = at.i0 + at.tiles - 1;
    if (tid ? i1 >= U1 && at.i0 >= U0 : at.i0 < U0) {
      first = at.i0 / (each * kWarps);
      blocks = i1 / (each * kWarps) - first + 1;
    }
    x.at[tid] = at;
  }
  x.first[tid] = first;
  x.blocks[tid] = blocks;
}

// By the whole block, at its end. Row r of warp w's kept segment lies at rows + w * warp_pitch + r * row_pitch
// (floats). `offs`: [CTAs + 1] and `part`: [threads] of shared memory, clear of the kept rows.
// With a shared prefix every item is left to the merge that follows, its partial results as above.
template <typename T, int D, int kRows, int kWarps>
__device__ __forceinline__ void join_items(const DecodeParams& p, const SeqEntry* seqs, int total, int each,
                                           const Kept<kRows, kWarps>& kept, const BlockEnds& ends, const float* rows, int warp_pitch,
                                           int row_pitch, int* offs, Column* part) {
  constexpr int kThreads = 32 * kWarps, C4 = D / 4;
  __shared__ int results[2];
  const int tid = threadIdx.x, cta = blockIdx.x, w_cta = cta * kWarps;
  const bool shared = p.pre.key_tiles > 0;
  const int U0 = min(total, w_cta * each), U1 = min(total, U0 + kWarps * each);
  __syncthreads();
  // 1. The kept segments of each item.
#pragma unroll 1
  for (int i = 0, k1; i < kWarps; i = k1) {
    k1 = i + 1;
    const int i0 = kept.i0[i];
    if (i0 < 0) continue;
    while (k1 < kWarps && kept.i0[k1] == i0) ++k1;
    const Place& at = kept.at[i];
    const int slot = slot_of(p, w_cta + i, at), i_end = i0 + at.tiles;
    const bool here = !shared && i0 >= U0 && i_end <= U1;
    // the item ends inside the next worker's range, which left that part in its slot
    const int more = here && i_end > (w_cta + k1) * each ? slot_of(p, w_cta + k1, at) : -1;
    const int F = rows_of(p, at) * C4;
#pragma unroll 1
    for (int f = tid; f < F; f += kThreads) {
      const int r = f / C4, c4 = f % C4;
      Column c = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
#pragma unroll 1
      for (int k = i; k < k1; ++k)
        add_column(c, *reinterpret_cast<const float4*>(rows + k * warp_pitch + r * row_pitch + c4 * 4), kept.m[k][r],
                   kept.l[k][r]);
      if (more >= 0) {
        const float2 y = __ldcg(p.ml + more + r);
        add_column(c, __ldcg(reinterpret_cast<const float4*>(p.po + (size_t)(more + r) * D) + c4), y.x, y.y);
      }
      if (here) {
        put_column<T, D>(p, at, r, c4, c.v, c.m, c.l);
      } else {
        *reinterpret_cast<float4*>(p.po + (size_t)(slot + r) * D + c4 * 4) = c.v;
        if (c4 == 0) p.ml[slot + r] = make_float2(c.m, c.l);
      }
    }
  }
  if (shared) return;
  __syncthreads();
  // 2. Which of the block's cut items it brings the last part of, and where that item's parts lie.
  if (tid < 2) {
    int n = 0;
    const int blocks = U0 < U1 ? ends.blocks[tid] : 0, first = ends.first[tid];
    if (blocks > 1) {
      __threadfence();
      if (static_cast<int>(atomicAdd(p.count + first, 1u)) + 1 == blocks) {
        p.count[first] = 0u;
        __threadfence();
        n = blocks;
      }
    }
    results[tid] = n;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int nb = results[e];
    if (nb == 0) continue;
    const Place& at = ends.at[e];
    const int i_end = at.i0 + at.tiles, w0 = at.i0 / each, w1 = (i_end - 1) / each, c0 = w0 / kWarps;
    const int n = nb + (w1 > (c0 + nb - 1) * kWarps && i_end < min(total, (w1 + 1) * each));
    for (int k = tid; k < n; k += kThreads)
      offs[k] = slot_of(p, k == 0 ? w0 : k < nb ? (c0 + k) * kWarps : w1, at);
    __syncthreads();
    // Columns of four channels; with few of them the partial results are dealt out to the threads too.
    const int F = rows_of(p, at) * C4, deal = F <= kThreads / 2 ? kThreads / F : 1;
    const int mine = deal > 1 ? tid / F : 0;
#pragma unroll 1
    for (int f = tid - mine * F; f < F && mine < deal; f += kThreads) {
      const int r = f / C4, c4 = f % C4;
      Column c = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
      constexpr int kBatch = 8;  // partial results whose loads are in flight together
#pragma unroll 1
      for (int k = mine; k < n; k += kBatch * deal) {
        float4 y[kBatch];
        float2 z[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int row = offs[min(k + j * deal, n - 1)] + r;
          y[j] = __ldcg(reinterpret_cast<const float4*>(p.po + (size_t)row * D) + c4);
          z[j] = __ldcg(p.ml + row);
        }
        float top = c.m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) top = fmaxf(top, z[j].x);  // one counted twice changes no maximum
        const float safe = top == -INFINITY ? 0.f : top, s = ex2_approx(c.m - safe);
        c.v = make_float4(c.v.x * s, c.v.y * s, c.v.z * s, c.v.w * s);
        c.l *= s;
        c.m = top;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const float t = k + j * deal < n ? ex2_approx(z[j].x - safe) : 0.f;
          c.v.x = fmaf(t, y[j].x, c.v.x);
          c.v.y = fmaf(t, y[j].y, c.v.y);
          c.v.z = fmaf(t, y[j].z, c.v.z);
          c.v.w = fmaf(t, y[j].w, c.v.w);
          c.l = fmaf(t, z[j].y, c.l);
        }
      }
      if (deal > 1)
        part[tid] = c;
      else
        put_column<T, D>(p, at, r, c4, c.v, c.m, c.l);
    }
    __syncthreads();
    if (deal > 1 && tid < F) {
      Column c = part[tid];
#pragma unroll 1
      for (int k = 1; k < min(deal, n); ++k) {  // the others had none
        const Column& o = part[k * F + tid];
        add_column(c, o.v, o.m, o.l);
      }
      put_column<T, D>(p, at, tid / C4, tid % C4, c.v, c.m, c.l);
    }
    __syncthreads();
  }
}

// Rows of idle sequences: O = 0, LSE = -inf. The blocks share the sequences out.
template <typename T, int D>
__device__ __forceinline__ void clear_idle_rows(const DecodeParams& p, const SeqEntry* seqs) {
#pragma unroll 1
  for (int b = blockIdx.x; b < p.a.B; b += gridDim.x) {
    const SeqEntry s = seqs[b];
    if (s.own >= 0 || s.own == kBadSeq) continue;
    const size_t at = (size_t)s.row0 * p.a.H, n = (size_t)(seqs[b + 1].row0 - s.row0) * p.a.H;
#pragma unroll 1
    for (size_t e = threadIdx.x; e < n * (D / 4); e += blockDim.x)
      put4<T>(static_cast<T*>(p.o) + (at * D + 4 * e), make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll 1
    for (size_t e = threadIdx.x; e < n; e += blockDim.x) p.lse[at + e] = -INFINITY;
  }
}

// The bf16 kernel on the tensor cores (fox_decode_mma.cu): its row tile for `rows` rows a sequence
// and key head, the workers of a CTA, its launch.
int decode_mma_rows(int rows);
int decode_mma_warps(int d);
cudaError_t launch_decode_mma(const DecodeParams& p, cudaStream_t s);
// The fp32 kernel (fox_decode_f32.cu): row tile, workers of a CTA, CTAs of an SM, launch.
int decode_f32_rows(int rows);
constexpr int kF32Warps = 4;
// CTAs: of 64 channels two fit an SM's shared memory (16 heads, 16 sequences of up to 1000: 49 -> 37.6 us against one, 4 of up
// to 2000: 33 -> 27.5, with the tables' entries asked for ahead; eight warps in one CTA were as fast there, but crowd short
// calls on few SMs).
constexpr int f32_ctas(int d) { return d == 128 ? kSMs : 2 * kSMs; }
cudaError_t launch_decode_f32(const DecodeParams& p, cudaStream_t s);
// The kernel of the 4-bit cache (fox_decode4.cu), as the bf16 one's.
int decode4_rows(int rows);
int decode4_warps(const PagedArgs& a, int Rt);
cudaError_t launch_decode4(const DecodeParams& p, cudaStream_t s);
// A 4-bit cache's shared prefix, K spread out to bf16 and V to fp16 (exactly) in the pool `to` of its pages in their order, with their gates and
// their table, for the prefix kernel.
cudaError_t launch_spread4(const DecodeParams& p, const PagedArgs& to, cudaStream_t s);
PrefixPlan prefix_plan(const PagedArgs& a);
cudaError_t launch_prefix(const DecodeParams& p, bool v16, cudaStream_t s);  // v16: V in fp16

}  // namespace fox
