// Attention of the newest tokens over the 4-bit paged cache, on CUDA cores.
//
// The math is fox_decode_f32.cu's, with K and V as s u (fox_four.h). One warp is one worker of the work line (fox_paged.h); it
// turns a key tile into fp32 in shared memory, a lane a key, and goes over it row by row.
#include "fox_decode.h"
#include "fox_four.h"

namespace fox {
namespace {

constexpr int kWarps4 = 4, kRows4 = 8;

template <int D>
struct Layout4 {
  static constexpr int kKPitch = D + 1, kVPitch = D + 1;
  static constexpr int kWarpFloats = ((kKeyTile * (kKPitch + kVPitch) + 3) & ~3) + kRows4 * D;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps4) decode4_kernel(const __grid_constant__ DecodeParams p) {
  using L = Layout4<D>;
  constexpr int E = D / 32, W = kWarps4, NR = kRows4, NB = D / kFourBlock;
  extern __shared__ float4 smem4[];
  __shared__ int scratch[W];
  __shared__ int offs[kSMs + 1];
  __shared__ Column part[32 * W];
  __shared__ Kept<NR, W> kept;
  __shared__ BlockEnds ends;
  float* smem = reinterpret_cast<float*>(smem4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* ks = smem + warp * L::kWarpFloats;
  float* vs = ks + kKeyTile * L::kKPitch;
  float* qs = smem + (warp + 1) * L::kWarpFloats - NR * D;
  SeqEntry* seqs = reinterpret_cast<SeqEntry*>(smem + W * L::kWarpFloats);
  const PagedArgs& a = p.a;
  grid_dep_wait();
  grid_dep_trigger();
  scan_sequences(p, seqs, scratch);
  const int G = a.H / a.Hkv, Gp = p.Gp, S = a.page_size, P = a.prefix_len, tp = ceil_div(P, kKeyTile);
  const int total = seqs[a.B].u0 * a.Hkv, each = units_per_worker(total, p.workers);
  const int w = blockIdx.x * W + warp;
  const int u0 = min(total, w * each), u1 = min(total, u0 + each);
  int left = u1 - u0;
  if (lane == 0) kept.i0[warp] = -1;
  Place at;
  if (left > 0) at = place_of(p, seqs, u0);
  if (warp == 0) find_ends<W>(p, seqs, total, each, ends);
#pragma unroll 1
  while (left > 0) {
    const Seq s = at.s;
    const int hkv = at.hkv, rt = at.rt, tile0 = at.tile, tile1 = min(at.tiles, tile0 + left), R = rows_of(p, at);
    Gate2 ci = {0.f, 0.f};
#pragma unroll 1
    for (int r = 0; r < NR; ++r) {
      const int rr = rt * p.Rt + r, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1);
      for (int c = lane; c < D; c += 32)
        qs[r * D + c] = r < R ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[(size_t)(s.row0 + t) * p.q_stride +
                                                                                      (size_t)h * D + c]) : 0.f;
    }
    if (lane < R) {
      const int rr = rt * p.Rt + lane, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1), i = s.own - s.n + t;
      ci = gate_sum(a, own_page_or_0(a, at.b, i), i & (S - 1), h);
    }
    float m[NR], l[NR], acc[NR][E];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    }
#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      const bool pre = tile < tp;
      const int j = (pre ? tile : tile - tp) * kKeyTile + lane;
      const bool key = j < (pre ? P : s.own);
      const int page = !key ? 0 : pre ? checked_page(a, a.prefix[j >> a.page_shift]) : own_page_or_0(a, at.b, j);
      const int slot = j & (S - 1);
      const uint8_t* kr = static_cast<const uint8_t*>(a.k) + four_row(a, page, hkv, slot);
      const uint8_t* vr = static_cast<const uint8_t*>(a.v) + four_row(a, page, hkv, slot);
      const uint8_t* sk = p.ks + four_scale_row(a, page, hkv, slot);
      const uint8_t* sv = p.vs + four_scale_row(a, page, hkv, slot & ~15);
#pragma unroll 1
      for (int i = 0; i < NB * 4; ++i) {
        const int b = i >> 2, t = i & 3;
        const float fk = four_scale(sk[b]), fv = four_scale(sv[four_v_scale(b, slot, NB)]);
        const uint32_t wk = four_k_code(*reinterpret_cast<const uint32_t*>(kr + four_k_word(b, t, NB)));
        const uint32_t wv = *reinterpret_cast<const uint32_t*>(vr + four_v_word(b, t, slot, NB));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ks[lane * L::kKPitch + i * 8 + e] = key ? fk * (static_cast<int>(wk >> 4 * e & 15u) - 8) : 0.f;
          vs[lane * L::kVPitch + i * 8 + e] = key ? fv * (static_cast<int>(wv >> 4 * e & 15u) - 8) : 0.f;
        }
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int rr = rt * p.Rt + r, t = token_of(p, rr), g = rr - t * Gp, h = hkv * G + min(g, G - 1);
        float dot = 0.f;
#pragma unroll 8
        for (int c = 0; c < D; ++c) dot = fmaf(qs[r * D + c], ks[lane * L::kKPitch + c], dot);
        const float hi = __shfl_sync(0xffffffffu, ci.hi, r), lo = __shfl_sync(0xffffffffu, ci.lo, r);
        float x = -INFINITY;
        if (r < R && key && (pre || j <= s.own - s.n + t)) {
          const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
          const int gs = slot - p.bias_from_j;
          const float gj = gs >= 0 ? a.g[g_offset(a, page, h, gs)] : 0.f;
          x = fmaf((hi - base.x) + (lo - base.y) - gj, kLog2e, dot * p.scale2);
        }
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m[r], top), safe = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2_approx(m[r] - safe), wt = ex2_approx(x - safe);
        m[r] = mn;
        l[r] = l[r] * alpha + wt;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= alpha;
#pragma unroll 4
        for (int jj = 0; jj < kKeyTile; ++jj) {
          const float y = __shfl_sync(0xffffffffu, wt, jj);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[r][e] = fmaf(y, vs[jj * L::kVPitch + e * 32 + lane], acc[r][e]);
        }
      }
      __syncwarp();
    }
    const bool alone = at.i0 >= u0 && at.i0 + at.tiles <= u1, keep = !alone && tile1 - tile0 == left;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        kept.m[warp][r] = m[r];
        kept.l[warp][r] = sum;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) qs[r * D + e * 32 + lane] = acc[r][e];
    }
    if (keep && lane == 0) {
      kept.i0[warp] = at.i0;
      kept.at[warp] = at;
    }
    __syncwarp();
    if (!keep) leave_rows<__nv_bfloat16, D>(p, at, w, alone, qs, D, kept.m[warp], kept.l[warp]);
    __syncwarp();
    left -= tile1 - tile0;
    at.tile = tile1;
    if (tile1 == at.tiles && left > 0) next_item(p, seqs, at);
  }
  clear_idle_rows<__nv_bfloat16, D>(p, seqs);
  join_items<__nv_bfloat16, D, NR, W>(p, seqs, total, each, kept, ends, smem + L::kWarpFloats - NR * D, L::kWarpFloats, D, offs,
                                      part);
}

template <int D>
cudaError_t launch(const DecodeParams& p, cudaStream_t s) {
  using L = Layout4<D>;
  const size_t smem = sizeof(float) * kWarps4 * L::kWarpFloats + sizeof(SeqEntry) * ((size_t)p.a.B + 1);
  // One limit for every call (launch in fox_decode_mma.cu has the reason).
  constexpr size_t kLimit = sizeof(float) * kWarps4 * L::kWarpFloats + sizeof(SeqEntry) * (kMaxSeqs + 1);
  static_assert(kLimit <= 232448 - 16384, "shared memory, less the static part");
  const cudaError_t e =
      cudaFuncSetAttribute(decode4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLimit));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode4", s);
  const cudaError_t f = launch_dependent(decode4_kernel<D>, dim3(kSMs), dim3(32 * kWarps4), smem, s, p);
  return f != cudaSuccess ? f : cudaGetLastError();
}

}  // namespace

int decode4_rows(int) { return kRows4; }
int decode4_warps(int, int) { return kWarps4; }

cudaError_t launch_decode4(const DecodeParams& p, cudaStream_t s) {
  return p.a.d == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace fox
