// fox_decode: workspace layout, launches, and the merge of a shared prefix's partial results.
#include "fox_decode.h"

namespace fox {
namespace {

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
  grid_dep_trigger();
  const int id = deal > 1 ? blockIdx.x : blockIdx.x * kMergeWarps + warp, part = deal > 1 ? warp : 0;
  const int row = id / a.H, h = id - row * a.H;
  // What the call was given may be read before the kernels ahead are through.
  const int b = row < a.rows ? seq_of_row(a, row) : -1;
  SeqInfo s;
  bool bad = b < 0;
  if (!bad) s = seq_info(a, b, &bad);
  if (bad || row < s.row0 || row >= s.row0 + s.n || s.own < 0) {  // whole blocks where the warps deal
    grid_dep_wait();  // idle rows are written already; but what follows this grid follows the others too
    return;
  }
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
  const int item0 = first_item(p.num, b, s.row0);
  grid_dep_wait();
  const int tiles = ceil_div(s.own, kKeyTile), r = (row - s.row0) * p.Gp + hl, rt = r / p.Rt;
  const int per_head = __ldcg(p.cum + a.B), each = units_per_worker(per_head * a.Hkv, p.workers);
  const int u0 = __ldcg(p.cum + b);
  if (p.num.by_rows() && u0 == __ldcg(p.cum + b + 1)) return;  // left out there (scan_sequences): nothing was written for it
  const int i0 = hkv * per_head + u0 + rt * tiles;
  // The own item's: one a block of workers, and its last worker's own where that is another (join_items).
  const int i1 = i0 + tiles - 1, w0 = i0 / each, w1 = i1 / each, c0 = w0 / p.warps, c1 = w1 / p.warps, nb = c1 - c0 + 1;
  const int n_own = nb + (w1 > w0 && w1 > c1 * p.warps && min(per_head * a.Hkv, (w1 + 1) * each) > i1 + 1);
  const int n = n_own + n_pre, own0 = (hkv * p.num.items + item0 + rt) * p.Rs + r - rt * p.Rt;
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
  int Rt, Gp, Rs, workers, warps;  // warps: workers of a CTA
  Numbering num;
  long long items;  // of a key head
  size_t cum, ml, po, pml, ppo, end;
  PrefixPlan pre;
  long long po_rows;
};

// Whether a prefix is worth sharing out: one kernel that walks it for every sequence takes as long as its
// K and V take to come (mostly from the L2 cache) so many times; sharing takes two more kernels, some
// microseconds here and there. At 47 MB walking took 19 to 23 us against 24 to 25, at 69 MB 24.7 and 28.3 against
// 24.8 and 28.7, at 78 MB 27.7 against 26.5, at 106 MB 31 against 25.5, at 150 MB 39 against 29.
bool share_prefix(const PagedArgs& a, int row_tiles) {
  return (long long)a.B * row_tiles * a.prefix_len * a.Hkv * a.d * 4 > (72ll << 20);
}

DecodeLayout decode_layout(const PagedArgs& a, bool f32) {
  DecodeLayout L;
  const int G = a.H / a.Hkv;
  L.Rt = f32 ? decode_f32_rows(a.max_new * G) : decode_mma_rows(a.max_new * G);
  L.Gp = padded_group(G, L.Rt);
  const int most = a.max_new * L.Gp;
  L.Rs = most < L.Rt ? most : L.Rt;
  const int row_tiles = ceil_div(most, L.Rt);  // of a sequence
  L.num = numbering(a, L.Gp, L.Rt == 1 ? 0 : L.Rt == 4 ? 2 : L.Rt == 8 ? 3 : 4, row_tiles, &L.items);
  L.warps = f32 ? kF32Warps : decode_mma_warps(a.d);
  L.workers = (f32 ? f32_ctas(a.d) : kSMs) * L.warps;
  const size_t slots = (size_t)L.workers + (size_t)a.Hkv * L.items;
  L.cum = kCacheHeaderBytes;
  L.po_rows = (long long)slots * L.Rs;
  L.ml = align_up(L.cum + sizeof(int) * ((size_t)a.B + 1), 256);
  L.po = align_up(L.ml + sizeof(float2) * slots * L.Rs, 256);
  L.pml = align_up(L.po + sizeof(float) * slots * L.Rs * a.d, 256);
  L.ppo = L.end = L.pml;
  L.pre = PrefixPlan{};
  if (!f32 && a.prefix_len > 0 && share_prefix(a, row_tiles)) {
    L.pre = prefix_plan(a);
    const size_t rows = ((size_t)L.pre.workers + (size_t)a.Hkv * L.pre.items) * 2 * kTile;
    L.ppo = align_up(L.pml + sizeof(float2) * rows, 256);
    L.end = align_up(L.ppo + sizeof(float) * rows * a.d, 256);
  }
  return L;
}

}  // namespace

bool decode_fits(const PagedArgs& a, bool f32) {
  const DecodeLayout L = decode_layout(a, f32);
  return line_fits(most_units(a, L.items), L.workers, L.warps) &&
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
  p.walk_prefix = x.a.prefix_len > 0 && L.pre.key_tiles == 0;
  p.o = x.o;
  p.lse = x.lse;
  p.Rt = L.Rt;
  p.Rs = L.Rs;
  p.num = L.num;
  p.Gp = L.Gp;
  p.gp_inv = L.Gp > 1 ? static_cast<uint32_t>(((1ull << 32) + L.Gp - 1) / L.Gp) : 0u;
  p.workers = L.workers;
  p.warps = L.warps;
  p.cum = reinterpret_cast<int*>(ws + L.cum);
  p.count = reinterpret_cast<uint32_t*>(ws + kErrWordBytes);
  p.ml = reinterpret_cast<float2*>(ws + L.ml);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pre = L.pre;
  p.pre.ml = reinterpret_cast<float2*>(ws + L.pml);
  p.pre.po = reinterpret_cast<float*>(ws + L.ppo);
  static_assert(kErrWordBytes + 4 * 2 * kSMs <= kCacheHeaderBytes, "a counter a CTA");
  const cudaError_t e = p.pre.key_tiles > 0 ? launch_prefix(p, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if (f32) return launch_decode_f32(p, s);
  const cudaError_t f = launch_decode_mma(p, s);
  if (f != cudaSuccess || p.pre.key_tiles == 0) return f;
  return x.a.d == 64 ? launch_merge<64>(p, s) : launch_merge<128>(p, s);
}

}  // namespace fox
