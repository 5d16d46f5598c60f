// Attention of the newest tokens over the paged cache in fp32, on CUDA cores.
//
// Math ("Forgetting Transformer (FoX) Attention" module source, ForgettingAttention.forward, for
// the rows of the newest tokens): x_ij = scale q_i . k_j + c_i - c_j over the keys j <= pos_i of
// the row's sequence, O_i = softmax_j(x_ij) V, LSE_i = ln sum_j exp(x_ij). One pass over the keys
// with the running maximum and sum, in log2 units; c_i - c_j is (c_i - base of key j's page), in
// two fp32 each, less the key's sum within the page, so that it keeps fp32 accuracy at any length.
//
// One warp is one worker of the work line (fox_paged.h). A key tile's K and V come to shared memory
// whole, by asynchronous copies (a row of 512 bytes an instruction): K of the next tile while this one's
// V is used, V of the next while its K is. Scores: a lane owns a key, whose row it reads with the rows
// padded to different banks. Values: a lane owns d / 32 channels. The prefix's keys, where one is
// shared, are walked like the sequence's own. Bound by latency where they are short (2 sequences of 257: 13 us), by
// the few warps that shared memory leaves an SM where they are long, each with one K and one V tile at most on its way (16 of up
// to 1000 with 16 heads of 64 channels, 75 MB: 34.5 us, 39 % of it what memory takes).
#include "fox_decode.h"

namespace fox {
namespace {

template <int D, int NR>
struct F32Layout {
  static constexpr int kKPitch = D + 4;  // floats of a K row in shared memory
  static constexpr int kWarpFloats = kKeyTile * kKPitch + kKeyTile * D + NR * D;  // K, V, queries or kept rows
};

// NR: rows of a row tile. Loops over rows have no other bound: with one known only at run time every row was a
// branch (8 sequences of up to 3000 on 32 / 8 heads, 16 rows a key head: 347 -> 170 us; 4 of 2000 with 4 rows: 49.6 -> 33.5;
// 16 of 1000 with one, 64 channels: 37.6 -> 34.2).
template <int D, int NR>
__global__ void __launch_bounds__(32 * kF32Warps) decode_f32_kernel(const __grid_constant__ DecodeParams p) {
  using L = F32Layout<D, NR>;
  constexpr int E = D / 32, W = kF32Warps;
  extern __shared__ float4 smem4[];
  __shared__ int scratch[W];
  __shared__ Gate2 ci[W][NR];
  __shared__ int offs[2 * kSMs + 1];
  __shared__ Column part[32 * W];
  __shared__ Kept<NR, W> kept;
  __shared__ BlockEnds ends;
  float* smem = reinterpret_cast<float*>(smem4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* ks = smem + warp * L::kWarpFloats;
  float* vs = ks + kKeyTile * L::kKPitch;
  float* qs = vs + kKeyTile * D;  // [NR][D] scaled queries; at a segment's end its rows of O
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
  bool first = true;

  // This lane's key of a tile: its place in the pools, as elements and gate slot; page -1: no key.
  int page = -1, slot = 0;
  size_t kv = 0;
  // The table's entry comes a tile ahead of its use: its key's page; -1: none of the pool, reported and read as page 0;
  // -2: no key.
  auto look_up = [&](int tile) {
    const bool pre = tile < tp;
    const int j = (pre ? tile : tile - tp) * kKeyTile + lane;
    return j >= (pre ? P : at.s.own) ? -2 : pre ? prefix_page(a, j) : own_page(a, at.b, j);
  };
  auto find_key = [&](int tile, int id) {
    page = id == -1 ? 0 : max(id, -1);
    if (id == -1 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    slot = ((tile < tp ? tile : tile - tp) * kKeyTile + lane) & (S - 1);
    kv = page < 0 ? 0 : kv_offset(a, page, at.hkv, slot);
  };
  // Rows of K or V of the tile whose keys the lanes hold; zeros for no key.
  auto ask = [&](float* dst, int pitch, const void* pool) {
    constexpr int kPer = 128 / D;  // rows an instruction
    const int sub = lane / (D / 4), c = lane % (D / 4) * 4;
#pragma unroll 4
    for (int r = 0; r < kKeyTile; r += kPer) {
      const size_t off = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(kv), r + sub);
      const int pg = __shfl_sync(0xffffffffu, page, r + sub);
      cp_async16_or_0(smem_u32(dst + (r + sub) * pitch + c), static_cast<const float*>(pool) + off + c, pg >= 0);
    }
    cp_async_commit();
  };

#pragma unroll 1
  while (left > 0) {
    // A segment: key tiles tile0 .. tile1 - 1 of one item.
    const Seq s = at.s;
    const int hkv = at.hkv, rt = at.rt, tile0 = at.tile, tile1 = min(at.tiles, tile0 + left), R = rows_of(p, at);
    find_key(tile0, look_up(tile0));
    ask(ks, L::kKPitch, a.k);
    ask(vs, D, a.v);
#pragma unroll 1
    for (int r = 0; r < NR; ++r) {
      const int rr = rt * p.Rt + r, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1);
      const float* src = static_cast<const float*>(p.q) + (size_t)(s.row0 + t) * p.q_stride + (size_t)h * D;
      if (lane < D / 4) {
        const float4 f = r < R ? *reinterpret_cast<const float4*>(src + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(qs + r * D + lane * 4) =
            make_float4(f.x * p.scale2, f.y * p.scale2, f.z * p.scale2, f.w * p.scale2);
      }
    }
    if (lane < R) {
      const int rr = rt * p.Rt + lane, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1), i = s.own - s.n + t;
      ci[warp][lane] = gate_sum(a, own_page_or_0(a, at.b, i), i & (S - 1), h);
    }
    // the first own key that not all of the item's rows see (the slots behind the last one hold zeros)
    const int partly = s.n > 1 ? s.own - s.n + token_of(p, rt * p.Rt) + 1 : s.own + kKeyTile;
    if (first) find_ends<W>(p, seqs, total, each, ends);  // by the first warp's lanes, once
    first = false;
    __syncwarp();

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
      // own place of this lane's key: before every row's for the prefix
      const int j = tile < tp ? -1 : (tile - tp) * kKeyTile + lane;
      const int next = tile + 1 < tile1 ? look_up(tile + 1) : -2;
      // c_i - c_j of the rows, -inf where the key is none of a row's; on their way while K is waited for.
      float bias[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        bias[r] = -INFINITY;
        if (r >= R) continue;
        const int rr = rt * p.Rt + r, t = token_of(p, rr), h = hkv * G + min(rr - t * Gp, G - 1);
        if (page >= 0 && j <= s.own - s.n + t) {
          const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
          const int gs = slot - p.bias_from_j;
          const float gj = gs >= 0 ? a.g[g_offset(a, page, h, gs)] : 0.f;
          bias[r] = (ci[warp][r].hi - base.x) + (ci[warp][r].lo - base.y) - gj;
        }
      }
      cp_async_wait<1>();  // K
      __syncwarp();
      float sc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) sc[r] = 0.f;
#pragma unroll 2
      for (int c = 0; c < D; c += 4) {
        const float4 f = *reinterpret_cast<const float4*>(ks + lane * L::kKPitch + c);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(qs + r * D + c);
          sc[r] = fmaf(q.x, f.x, fmaf(q.y, f.y, fmaf(q.z, f.z, fmaf(q.w, f.w, sc[r]))));
        }
      }
      __syncwarp();
      if (tile + 1 < tile1) {
        find_key(tile + 1, next);
        ask(ks, L::kKPitch, a.k);
      } else {
        cp_async_commit();  // nothing: the groups stay in step
      }
      // Scores to weights.
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float x = bias[r] == -INFINITY ? -INFINITY : fmaf(bias[r], kLog2e, sc[r]);
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m[r], top), safe = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2_approx(m[r] - safe), wt = ex2_approx(x - safe);
        m[r] = mn;
        l[r] = l[r] * alpha + wt;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= alpha;
        sc[r] = wt;
      }
      cp_async_wait<1>();  // V
      __syncwarp();
      if (NR == 1 || tile < tp || (tile - tp) * kKeyTile + kKeyTile <= partly) {
#pragma unroll 4
        for (int jj = 0; jj < kKeyTile; ++jj) {
          float f[E];
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = vs[jj * D + lane * E + e];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float wt = __shfl_sync(0xffffffffu, sc[r], jj);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[r][e] = fmaf(wt, f[e], acc[r][e]);
          }
        }
      } else {
        // Keys that some of the rows do not see: a weight of 0 times an infinity or a NaN would be a NaN.
#pragma unroll 1
        for (int jj = 0; jj < kKeyTile; ++jj)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float wt = __shfl_sync(0xffffffffu, sc[r], jj);
            if (wt == 0.f) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[r][e] = fmaf(wt, vs[jj * D + lane * E + e], acc[r][e]);
          }
      }
      __syncwarp();
      if (tile + 1 < tile1)
        ask(vs, D, a.v);
      else
        cp_async_commit();
    }
    // Results: rows in shared memory, where the queries were, for the block to join with its neighbours', or
    // finished, or to the worker's slot.
    const bool alone = at.i0 >= u0 && at.i0 + at.tiles <= u1, keep = !alone && tile1 - tile0 == left;
    __syncwarp();
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
      for (int e = 0; e < E; ++e) qs[r * D + lane * E + e] = acc[r][e];
    }
    if (keep && lane == 0) {
      kept.i0[warp] = at.i0;
      kept.at[warp] = at;
    }
    __syncwarp();
    if (!keep) leave_rows<float, D>(p, at, w, alone, qs, D, kept.m[warp], kept.l[warp]);
    __syncwarp();
    left -= tile1 - tile0;
    at.tile = tile1;
    if (tile1 == at.tiles && left > 0) next_item(p, seqs, at);
  }
  clear_idle_rows<float, D>(p, seqs);
  join_items<float, D, NR, W>(p, seqs, total, each, kept, ends, smem + kKeyTile * (L::kKPitch + D), L::kWarpFloats, D,
                                    offs, part);
}

template <int D, int NR>
cudaError_t launch(const DecodeParams& p, cudaStream_t s) {
  using L = F32Layout<D, NR>;
  const size_t smem = sizeof(float) * kF32Warps * L::kWarpFloats + sizeof(SeqEntry) * ((size_t)p.a.B + 1);
  // One limit for every call (launch in fox_decode_mma.cu has the reason).
  constexpr size_t kLimit = sizeof(float) * kF32Warps * L::kWarpFloats + sizeof(SeqEntry) * (kMaxSeqs + 1);
  static_assert(kLimit <= 232448 - 16384, "shared memory, less the static part");
  const cudaError_t e = cudaFuncSetAttribute(decode_f32_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kLimit));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode", s);
  const cudaError_t f = launch_dependent(decode_f32_kernel<D, NR>, dim3(f32_ctas(D)), dim3(32 * kF32Warps), smem, s, p);
  return f != cudaSuccess ? f : cudaGetLastError();
}

}  // namespace

// The least that takes the most rows a sequence may bring a key head; more are tiles of 8.
int decode_f32_rows(int rows) { return rows <= 1 ? 1 : rows <= 4 ? 4 : 8; }

cudaError_t launch_decode_f32(const DecodeParams& p, cudaStream_t s) {
  if (p.a.d == 64) return p.Rt == 1 ? launch<64, 1>(p, s) : p.Rt == 4 ? launch<64, 4>(p, s) : launch<64, 8>(p, s);
  return p.Rt == 1 ? launch<128, 1>(p, s) : p.Rt == 4 ? launch<128, 4>(p, s) : launch<128, 8>(p, s);
}

}  // namespace fox
