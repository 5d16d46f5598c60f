// Attention of the newest tokens of every sequence over the paged cache in fp32, on CUDA cores, and
// the launches of fox_decode.
//
// Math ("Forgetting Transformer (FoX) Attention" module source, ForgettingAttention.forward, for
// the rows of the newest tokens): x_ij = scale q_i . k_j + c_i - c_j over the keys j <= pos_i of
// the row's sequence, O_i = softmax_j(x_ij) V, LSE_i = ln sum_j exp(x_ij). One pass over the keys
// with the running maximum and sum, in log2 units; c_i - c_j is formed as
// (c_i - base of key j's page, in fp64) - (the key's sum within the page), so that it keeps fp32
// accuracy at any length.
//
// One warp is one worker of the work line (fox_paged.h). Scores: a lane owns a key, the rows'
// dot products run over its row of K. Values: a lane owns d / 32 channels.
#include "fox_decode.h"

namespace fox {
namespace {

constexpr int kSimtWarps = 4;
constexpr int kSimtRows = 8;
constexpr int kSimtCtas = 4;  // CTAs of an SM

__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  f[0] = w.x;
  f[1] = w.y;
  f[2] = w.z;
  f[3] = w.w;
}

template <int D>
__global__ void __launch_bounds__(32 * kSimtWarps, kSimtCtas) decode_simt_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int E = D / 32;
  extern __shared__ Seq seqs[];  // [B + 1]
  __shared__ int scratch[kSimtWarps];
  __shared__ __align__(16) float qs[kSimtWarps][kSimtRows][D];  // scaled queries; at the end the kept rows
  __shared__ Gate2 ci[kSimtWarps][kSimtRows];
  __shared__ int offs[kSMs * kSimtCtas + 1];
  __shared__ Column part[32 * kSimtWarps];
  __shared__ BlockEnds ends;
  __shared__ Kept<kSimtRows, kSimtWarps> kept;
  const PagedArgs& a = p.a;
  scan_sequences(p, seqs, scratch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv, Gp = p.Gp, S = a.page_size, P = a.prefix_len;
  const int total = seqs[a.B].u0 * a.Hkv, each = units_per_worker(total, p.workers);
  const int w = blockIdx.x * kSimtWarps + warp;
  const int u0 = min(total, w * each);
  const int u1 = min(total, u0 + each);
  int left = u1 - u0;
  Place at;
  if (left > 0) at = place_of(p, seqs, u0);
  if (lane == 0) kept.i0[warp] = -1;
  find_ends<kSimtWarps>(p, seqs, total, each, ends);
  while (left > 0) {
    // A segment: key tiles tile0 .. tile1 - 1 of one item.
    const Seq s = at.s;
    const int b = at.b, hkv = at.hkv, rt = at.rt;
    const int keys = s.own + P, tile0 = at.tile, tile1 = min(at.tiles, tile0 + left);
    const int R = rows_of(p, at);

    __syncwarp();
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      const int rr = rt * p.Rt + r, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1);
      const float* src = static_cast<const float*>(p.q) + (size_t)(s.row0 + t) * p.q_stride + (size_t)h * D;
      for (int c = lane * 4; c < D; c += 128) {
        float f[4];
        load4(src + c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) qs[warp][r][c + e] = f[e] * p.scale2;
      }
      if (lane == 0) {
        const int i = s.own - s.n + t;
        ci[warp][r] = gate_sum(a, own_page_or_0(a, b, i), i & (S - 1), h);
      }
    }
    __syncwarp();

    float m[kSimtRows], l[kSimtRows], acc[kSimtRows][E];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    }
    for (int tile = tile0; tile < tile1; ++tile) {
      const int j = tile * kKeyTile + lane;
      const bool in = j < keys;
      int page = -1, slot = 0;
      if (in) {
        const int own = j - P;
        page = j < P ? prefix_page(a, j) : own_page(a, b, own);
        slot = (j < P ? j : own) & (S - 1);
        if (page < 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
      }
      const size_t kv = page >= 0 ? kv_offset(a, page, hkv, slot) : 0;
      float sc[kSimtRows];
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) sc[r] = 0.f;
      if (page >= 0) {
        const float* kp = static_cast<const float*>(a.k) + kv;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
          float f[4];
          load4(kp + c, f);
#pragma unroll
          for (int r = 0; r < kSimtRows; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(&qs[warp][r][c]);
            sc[r] = fmaf(qv.x, f[0], fmaf(qv.y, f[1], fmaf(qv.z, f[2], fmaf(qv.w, f[3], sc[r]))));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) {
        float x = -INFINITY;
        if (r < R && page >= 0) {
          const int rr = rt * p.Rt + r, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1);
          if (j <= P + s.own - s.n + t) {
            const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
            const float beta = (ci[warp][r].hi - base.x) + (ci[warp][r].lo - base.y);
            const int gs = p.bias_from_j ? slot - 1 : slot;
            const float gj = gs >= 0 ? a.g[g_offset(a, page, h, gs)] : 0.f;
            x = fmaf(beta - gj, kLog2e, sc[r]);
          }
        }
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m[r], top);
        const float safe = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2_approx(m[r] - safe);
        const float w_ = ex2_approx(x - safe);
        m[r] = mn;
        l[r] = l[r] * alpha + w_;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= alpha;
        sc[r] = w_;
      }
      const int nk = min(kKeyTile, keys - tile * kKeyTile);
#pragma unroll 4
      for (int jj = 0; jj < nk; ++jj) {
        const size_t at = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(kv), jj);
        const int pg = __shfl_sync(0xffffffffu, page, jj);
        if (pg < 0) continue;
        const float* vp = static_cast<const float*>(a.v) + at + lane * E;
        float f[E];
        if (E == 4) {
          load4(vp, f);
        } else {
          const float2 wv = *reinterpret_cast<const float2*>(vp);
          f[0] = wv.x;
          f[1] = wv.y;
        }
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          const float pr = __shfl_sync(0xffffffffu, sc[r], jj);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[r][e] = fmaf(pr, f[e], acc[r][e]);
        }
      }
    }
    // Results: rows in shared memory, where the queries were, for the block to join with its neighbours', or
    // finished, or to the worker's slot.
    const bool alone = at.i0 >= u0 && at.i0 + at.tiles <= u1, keep = !alone && tile1 - tile0 == left;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        kept.m[warp][r] = m[r];
        kept.l[warp][r] = sum;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) qs[warp][r][lane * E + e] = acc[r][e];
    }
    if (keep && lane == 0) {
      kept.i0[warp] = at.i0;
      kept.at[warp] = at;
    }
    __syncwarp();
    if (!keep) leave_rows<float, D>(p, at, w, alone, &qs[warp][0][0], D, kept.m[warp], kept.l[warp]);
    left -= tile1 - tile0;
    at.tile = tile1;
    if (tile1 == at.tiles && left > 0) next_item(p, seqs, at);
  }
  clear_idle_rows<float, D>(p, seqs);
  join_items<float, D, kSimtRows, kSimtWarps>(p, seqs, total, each, kept, ends, &qs[0][0][0], kSimtRows * D, D, offs, part);
}

// One output row (query row, query head): the partial results of its own item and of the shared prefix
// joined, in a fixed order, by one warp, or with few rows (deal = kMergeWarps) by a block's warps, which
// deal them out. What bounds it is latency: a row has up to some dozens of results of 4 d bytes.
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const __grid_constant__ DecodeParams p,
                                                                       const int deal) {
  constexpr int E = D / 32;
  const PagedArgs& a = p.a;
  __shared__ float sums[kMergeWarps][D];
  __shared__ float2 mls[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int id = deal > 1 ? blockIdx.x : blockIdx.x * kMergeWarps + warp, part = deal > 1 ? warp : 0;
  const int row = id / a.H, h = id - row * a.H;
  if (row >= a.rows) return;  // whole blocks where the warps deal
  // What the call was given may be read before the kernels ahead are through.
  const int b = seq_of_row(a, row);
  if (b < 0) return;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (bad || row < s.row0 || row >= s.row0 + s.n || s.own < 0) return;  // idle rows are written already
  const int G = a.H / a.Hkv, hkv = h / G, hl = h - hkv * G;
  const int pos = s.own - s.n + (row - s.row0), last = a.prefix_len - 1, mask = a.page_size - 1;
  const Gate2 ci = gate_sum(a, own_page_or_0(a, b, pos), pos & mask, h);
  const Gate2 cl = gate_sum(a, max(prefix_page(a, last), 0), last & mask, h);
  const float shift = ((ci.hi - cl.hi) + (ci.lo - cl.lo)) * kLog2e;  // what the row's prefix scores lack
  // The prefix's partial results: of result i, ml and po lie `step` rows further on.
  const PrefixPlan& x = p.pre;
  const int tile = row / x.tpt * x.head_chunks + hl / x.hp;
  const bool both = x.row_tiles == 1;  // the streams are two results, else this row is one stream's
  const int item = hkv * x.items + (both ? 0 : tile / 2);
  const int v0 = item * x.line / x.each, v1 = (item * x.line + x.key_tiles - 1) / x.each;
  const int n_pre = (v1 - v0 + 1) * (both ? 2 : 1), step = both ? kTile : 2 * kTile;
  const size_t pre0 = ((size_t)(v0 + item) * 2 + (both ? 0 : tile & 1)) * kTile + hl % x.hp * x.tpt + row % x.tpt;
  grid_dep_wait();
  const int tiles = ceil_div(s.own, kKeyTile), r = (row - s.row0) * p.Gp + hl, rt = r / p.Rt;
  const int per_head = __ldcg(p.cum + a.B), each = units_per_worker(per_head * a.Hkv, p.workers);
  const int i0 = hkv * per_head + __ldcg(p.cum + b) + rt * tiles;
  // The own item's: one a block of workers, and its last worker's own where that is another (join_items).
  const int i1 = i0 + tiles - 1, w0 = i0 / each, w1 = i1 / each, c0 = w0 / p.warps, c1 = w1 / p.warps, nb = c1 - c0 + 1;
  const int n_own = nb + (w1 > w0 && w1 > c1 * p.warps && min(per_head * a.Hkv, (w1 + 1) * each) > i1 + 1);
  const int n = n_own + n_pre, own0 = ((hkv * a.B + b) * p.RTmax + rt) * p.Rs + r - rt * p.Rt;
  float m = -INFINITY, l = 0.f, acc[E] = {};
#pragma unroll 1
  for (int first = 0; first < n; first += 32 * deal) {
    // lane i: where this warp's i-th result lies, its maximum and sum
    const int i = first + lane * deal + part;
    const float* src = nullptr;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (i < n_own) {
      const int at = own0 + (i == 0 ? w0 : i < nb ? (c0 + i) * p.warps : w1) * p.Rs;
      ml = __ldcg(p.ml + at);
      src = p.po + (size_t)at * D;
    } else if (i < n) {
      const size_t at = pre0 + (size_t)(i - n_own) * step;
      ml = __ldcg(x.ml + at);
      ml.x += shift;
      src = x.po + at * D;
    }
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const float safe = top == -INFINITY ? 0.f : top;
    const float alpha = ex2_approx(m - safe), wgt = ex2_approx(ml.x - safe);
    m = top;
    l = l * alpha + ml.y * wgt;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= alpha;
    // A result without weight is not read: a stream without keys wrote no sums of V.
    unsigned has = __ballot_sync(0xffffffffu, wgt != 0.f);
#pragma unroll 1
    while (has) {
      constexpr int kBatch = 8;  // results whose loads are in flight together
      float2 z[kBatch][E / 2];
      float f[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = has ? __ffs(has) - 1 : 0;
        f[j] = has ? __shfl_sync(0xffffffffu, wgt, k) : 0.f;
        const float* at = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k));
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
          z[j][e] = has ? __ldcg(reinterpret_cast<const float2*>(at + lane * E) + e) : make_float2(0.f, 0.f);
        has &= has - 1;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          acc[2 * e] = fmaf(f[j], z[j][e].x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(f[j], z[j][e].y, acc[2 * e + 1]);
        }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
  for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
  if (lane == 0) mls[warp] = make_float2(m, l);
  if (deal > 1)
    __syncthreads();
  else
    __syncwarp();
  // Two channels a thread; with one warp a row, its lanes take them in turn.
#pragma unroll 1
  for (int ch = (deal > 1 ? threadIdx.x : lane) * 2; ch < D; ch += 64 * deal) {
  const int w0_ = deal > 1 ? 0 : warp, w1_ = deal > 1 ? kMergeWarps : warp + 1;
  float top = -INFINITY;
#pragma unroll 1
  for (int w = w0_; w < w1_; ++w) top = fmaxf(top, mls[w].x);
  const float safe = top == -INFINITY ? 0.f : top;
  float o0 = 0.f, o1 = 0.f, sum = 0.f;
#pragma unroll 1
  for (int w = w0_; w < w1_; ++w) {
    const float t = ex2_approx(mls[w].x - safe);
    o0 = fmaf(t, sums[w][ch], o0);
    o1 = fmaf(t, sums[w][ch + 1], o1);
    sum = fmaf(t, mls[w].y, sum);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t at = (size_t)row * a.H + h;
  *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + at * D + ch) = pack_bf16x2(o0 * inv, o1 * inv);
  if (ch == 0) p.lse[at] = sum > 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
  }
}

template <int D>
cudaError_t launch_merge(const DecodeParams& p, cudaStream_t s) {
  TraceScope trace("decode_merge", s);
  // Dealing pays while its blocks are on the SMs at once (32 x 32 rows: 17 -> 12 us; 256 x 32: 21 -> 37 us).
  const int rows = p.a.rows * p.a.H, deal = rows <= kSMs * 12 ? kMergeWarps : 1;
  const cudaError_t e =
      launch_dependent(prefix_merge_kernel<D>, dim3(deal > 1 ? rows : ceil_div(rows, kMergeWarps)),
                       dim3(32 * kMergeWarps), 0, s, p, deal);
  return e != cudaSuccess ? e : cudaGetLastError();
}

struct DecodeLayout {
  int Rt, Gp, Rs, RTmax, workers;
  size_t cum, ml, po, pml, ppo, end;
  PrefixPlan pre;
  long long po_rows;
};

DecodeLayout decode_layout(const PagedArgs& a, bool f32) {
  DecodeLayout L;
  const int G = a.H / a.Hkv;
  L.Rt = f32 ? kSimtRows : decode_mma_rows(a.max_new * G);
  L.Gp = padded_group(G, L.Rt);
  const int most = a.max_new * L.Gp;
  L.Rs = most < L.Rt ? most : L.Rt;
  L.RTmax = ceil_div(most, L.Rt);
  L.workers = f32 ? kSMs * kSimtCtas * kSimtWarps : kSMs * decode_mma_warps(a.d);
  const size_t slots = (size_t)L.workers + (size_t)a.B * a.Hkv * L.RTmax;
  L.cum = kCacheHeaderBytes;
  L.po_rows = (long long)slots * L.Rs;
  L.ml = align_up(L.cum + sizeof(int) * ((size_t)a.B + 1), 256);
  L.po = align_up(L.ml + sizeof(float2) * slots * L.Rs, 256);
  L.pml = align_up(L.po + sizeof(float) * slots * L.Rs * a.d, 256);
  L.ppo = L.end = L.pml;
  L.pre = PrefixPlan{};
  if (!f32 && a.prefix_len > 0) {
    L.pre = prefix_plan(a);
    const size_t rows = ((size_t)L.pre.workers + (size_t)a.Hkv * L.pre.items) * 2 * kTile;
    L.ppo = align_up(L.pml + sizeof(float2) * rows, 256);
    L.end = align_up(L.ppo + sizeof(float) * rows * a.d, 256);
  }
  return L;
}

template <int D>
cudaError_t launch_simt(const DecodeParams& p, cudaStream_t s) {
  const size_t smem = sizeof(Seq) * ((size_t)p.a.B + 1);
  const cudaError_t e =
      cudaFuncSetAttribute(decode_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode", s);
  decode_simt_kernel<D><<<kSMs * kSimtCtas, 32 * kSimtWarps, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool decode_fits(const PagedArgs& a, bool f32) {
  const DecodeLayout L = decode_layout(a, f32);
  return most_units(a, L.Rt, L.Gp) < 0x7fffffffLL - L.workers &&
         (unsigned long long)a.max_new * L.Gp * L.Gp < (1ull << 32) && L.po_rows < 0x7fffffffLL &&
         (L.pre.key_tiles == 0 || (long long)a.Hkv * L.pre.items * L.pre.line < 0x7fffffffLL - L.pre.each);
}

size_t decode_workspace_bytes(const PagedArgs& a, bool f32) { return decode_layout(a, f32).end; }

cudaError_t launch_decode(const DecodeArgs& x, bool f32, char* ws, cudaStream_t s) {
  const DecodeLayout L = decode_layout(x.a, f32);
  DecodeParams p = {};
  p.a = x.a;
  p.q = x.q;
  p.q_stride = x.q_stride;
  p.scale2 = x.scale * kLog2e;
  p.bias_from_j = x.bias_from_j;
  p.walk_prefix = f32;
  p.o = x.o;
  p.lse = x.lse;
  p.Rt = L.Rt;
  p.Rs = L.Rs;
  p.RTmax = L.RTmax;
  p.Gp = L.Gp;
  p.gp_inv = L.Gp > 1 ? static_cast<uint32_t>(((1ull << 32) + L.Gp - 1) / L.Gp) : 0u;
  p.workers = L.workers;
  p.warps = f32 ? kSimtWarps : decode_mma_warps(x.a.d);
  p.cum = reinterpret_cast<int*>(ws + L.cum);
  p.count = reinterpret_cast<uint32_t*>(ws + kErrWordBytes);
  p.ml = reinterpret_cast<float2*>(ws + L.ml);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pre = L.pre;
  p.pre.ml = reinterpret_cast<float2*>(ws + L.pml);
  p.pre.po = reinterpret_cast<float*>(ws + L.ppo);
  static_assert(kErrWordBytes + 4 * kSMs * kSimtCtas * kSimtWarps <= kCacheHeaderBytes, "counters of all workers");
  const cudaError_t e = p.pre.key_tiles > 0 ? launch_prefix(p, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if (f32) return x.a.d == 64 ? launch_simt<64>(p, s) : launch_simt<128>(p, s);
  const cudaError_t f = launch_decode_mma(p, s);
  if (f != cudaSuccess || p.pre.key_tiles == 0) return f;
  return x.a.d == 64 ? launch_merge<64>(p, s) : launch_merge<128>(p, s);
}

}  // namespace fox
