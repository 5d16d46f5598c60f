// Attention of a batch to the prefix that its sequences share, computed once for all of them, bf16.
//
// c_i is constant along row i and cancels in the softmax, so against the prefix every query row of
// every sequence sees the same matrix of keys and the same bias c_last - c_j (c_last: the cumulative
// log gate of the prefix's last token). All rows of a key head therefore form one tall matrix: 128-row
// tiles against 128-key tiles on the tensor cores, K and V read from memory once for all sequences
// instead of once a sequence. The rows leave unnormalised partial results, which the merge joins with
// those of the sequences' own keys; the row's c_i - c_last enters there.
//
// A row tile is `tpt` tokens x `hp` query heads of the key head's group: rows are (token, head), one
// TMA box. Key tiles of an item (key head, row tiles) run from the last to the first: the bias falls
// with distance, so the first tile nearly always holds the row maximum. Work is split like the own
// keys' (fox_paged.h): the items' key tiles on one line, equal ranges of it to the CTAs, one CTA an SM.
//
// Two streams of softmax warps share the tensor core, each with its S and O in tensor memory:
//   more than one row tile a key head: an item is two row tiles, one a stream, on the same key tiles;
//   one row tile: the streams take alternate key tiles, and leave a partial result each.
// Warp roles (384 threads): warps 0-3 and 4-7 the streams' softmax (thread = row = TMEM lane), warp 8
// TMA producer, warp 9 TMEM allocator and MMA issuer, warps 10-11 the gates: log2 e (c_j - c_last) of
// a key tile's keys and the row tile's heads into shared memory, alternate key tiles.
//
// P V: P = hi + lo in bf16, two products (see fox_decode_mma.cu). A 32-column chunk of S, once read,
// takes its own 16 columns of hi and 16 of lo, so P needs no memory beside S; the row maximum is
// found in a pass of its own, because S is gone after the second.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_decode.h"

namespace fox {
namespace {

constexpr int kPrefixThreads = 384;
constexpr int kMaxHp = 16;
constexpr int kKapPitch = kTile + 4;  // floats: the heads' rows start in different banks
constexpr float kRaise = 8.0f;        // log2 units that a row may pass its running maximum by

template <int D>
struct PrefixLayout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;                    // two row tiles
  static constexpr int kK = 2 * kTileBytes;       // two stages
  static constexpr int kV = 4 * kTileBytes;
  static constexpr int kKap = 6 * kTileBytes;     // two stages of [hp][kKapPitch]
};

enum PBar {
  P_Q = 0,
  P_KFULL = 1,   // +stage
  P_KEMPTY = 3,
  P_VFULL = 5,
  P_VEMPTY = 7,
  P_GFULL = 9,   // +stage: the key tile's gate terms (and the tail of V) are in place
  P_GEMPTY = 11,
  P_SFULL = 13,  // +stream
  P_PFULL = 15,
  P_OFINAL = 17,
  P_DONE = 19,
  P_COUNT = 20,
};

// Row maximum of x_j = scale2 S_j - kap_j; columns from `lim` on are not keys.
template <bool kTail>
__device__ __forceinline__ float row_top(uint32_t tS, const float* kap, float scale2, int lim) {
  const float2 nsc = make_float2(-scale2, -scale2);
  float mn = INFINITY;  // min of kap_j - scale2 S_j
  uint32_t rawb[2][32];
  tmem_ld32(tS, rawb[0]);
#pragma unroll
  for (int qt = 0; qt < 4; ++qt) {
    tmem_ld_wait();
    if (qt + 1 < 4) tmem_ld32(tS + 32 * (qt + 1), rawb[(qt + 1) & 1]);
    const uint32_t* raw = rawb[qt & 1];
#pragma unroll
    for (int j4 = 0; j4 < 8; ++j4) {
      const int j = 32 * qt + 4 * j4;
      const float4 kk = lds_f4(kap + j);
      float2 a = ffma2(make_float2(__uint_as_float(raw[4 * j4]), __uint_as_float(raw[4 * j4 + 1])), nsc,
                       make_float2(kk.x, kk.y));
      float2 c = ffma2(make_float2(__uint_as_float(raw[4 * j4 + 2]), __uint_as_float(raw[4 * j4 + 3])), nsc,
                       make_float2(kk.z, kk.w));
      if (kTail) {
        if (j >= lim) a.x = INFINITY;
        if (j + 1 >= lim) a.y = INFINITY;
        if (j + 2 >= lim) c.x = INFINITY;
        if (j + 3 >= lim) c.y = INFINITY;
      }
      mn = fmin3(fmin3(mn, a.x, a.y), c.x, c.y);
    }
  }
  return -mn;
}

// P_j = 2^(x_j - off) over the row's S: chunk q's hi to columns 32 q .. 32 q + 15, lo to the next 16
// (two columns of P a 32-bit column). Returns the sum of the P_j, in fp32.
template <bool kTail>
__device__ __forceinline__ float row_exp(uint32_t tS, const float* kap, float scale2, float off, int lim) {
  const float2 nsc = make_float2(-scale2, -scale2), noff = make_float2(-off, -off);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int qt = 0; qt < 4; ++qt) {
    uint32_t raw[32];
    tmem_ld32(tS + 32 * qt, raw);
    tmem_ld_wait();
    uint32_t pk[32];
#pragma unroll
    for (int j4 = 0; j4 < 8; ++j4) {
      const int j = 32 * qt + 4 * j4;
      const float4 kk = lds_f4(kap + j);
      float2 wa = fsub2(noff, ffma2(make_float2(__uint_as_float(raw[4 * j4]), __uint_as_float(raw[4 * j4 + 1])), nsc,
                                    make_float2(kk.x, kk.y)));
      float2 wc = fsub2(noff, ffma2(make_float2(__uint_as_float(raw[4 * j4 + 2]), __uint_as_float(raw[4 * j4 + 3])),
                                    nsc, make_float2(kk.z, kk.w)));
      if (kTail) {
        if (j >= lim) wa.x = -INFINITY;
        if (j + 1 >= lim) wa.y = -INFINITY;
        if (j + 2 >= lim) wc.x = -INFINITY;
        if (j + 3 >= lim) wc.y = -INFINITY;
      }
      const float2 pa = make_float2(ex2_approx(wa.x), ex2_approx(wa.y));
      const float2 pc = make_float2(ex2_approx(wc.x), ex2_approx(wc.y));
      s = fadd2(s, fadd2(pa, pc));
      const uint32_t ha = pack_bf16x2(pa.x, pa.y), hc = pack_bf16x2(pc.x, pc.y);
      const float2 la = fsub2(pa, make_float2(__uint_as_float(ha << 16), __uint_as_float(ha & 0xFFFF0000u)));
      const float2 lc = fsub2(pc, make_float2(__uint_as_float(hc << 16), __uint_as_float(hc & 0xFFFF0000u)));
      pk[2 * j4] = ha;
      pk[2 * j4 + 1] = hc;
      pk[16 + 2 * j4] = pack_bf16x2(la.x, la.y);
      pk[16 + 2 * j4 + 1] = pack_bf16x2(lc.x, lc.y);
    }
    tmem_st32(tS + 32 * qt, pk);
  }
  return s.x + s.y;
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ DecodeParams p) {
  using L = PrefixLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[P_COUNT];
  __shared__ uint32_t tmem_word;
  __shared__ int abort_word;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &abort_word;
  const PagedArgs& a = p.a;
  const PrefixPlan& pp = p.pre;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.page_size, G = a.H / a.Hkv, P = a.prefix_len;
  const bool split_keys = pp.row_tiles == 1;  // the streams take alternate key tiles
  const int step = split_keys ? 2 : 1;        // key tiles from one of a stream's to its next

  grid_dep_trigger();  // the own keys' kernel may start where this one leaves room: it needs nothing from here
  if (threadIdx.x == 0) {
    for (int i = 0; i < P_COUNT; ++i)
      mbar_init(&bars[i], i == P_PFULL || i == P_PFULL + 1 ? 4
                          : i == P_GEMPTY || i == P_GEMPTY + 1 ? (split_keys ? 4 : 8)
                                                               : 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_word, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_word;

  const int total = a.Hkv * pp.items * pp.key_tiles, each = units_per_worker(total, pp.workers);
  const int u_end = min(total, static_cast<int>(blockIdx.x + 1) * each);
  int u = blockIdx.x * each;

  bool ok = true;              // of this thread's role
  int c0 = 0;                  // key tiles before this segment (ring position)
  int sc[2] = {0, 0};          // tiles of each stream before this segment
  int oc[2] = {0, 0};          // segments in which each stream had tiles
  int seg = 0;
  while (u < u_end) {
    // A segment: key tiles t1 - 1 down to t0 of item (hkv, it).
    const int item = u / pp.key_tiles, hkv = item / pp.items, it = item % pp.items;
    const int t0 = u % pp.key_tiles, t1 = min(pp.key_tiles, t0 + (u_end - u));
    const int nT = t1 - t0;
    const int T0 = split_keys ? 0 : 2 * it;  // row tile of stream 0; stream 1 has the next, or the same
    const bool has1 = split_keys ? nT > 1 : T0 + 1 < pp.row_tiles;
    const int n0 = split_keys ? (nT + 1) / 2 : nT, n1 = split_keys ? nT / 2 : (has1 ? nT : 0);
    const int npages = (P + S - 1) / S;

    if (warp == 8) {
      // --------------------------------------------------------- producer
      auto page_of = [&](int t) {  // lane i: page i of key tile t, or -1
        const int i = t * (kTile / S) + lane;
        if (lane >= kTile / S || i >= npages) return -1;
        int id = prefix_page(a, i * S);
        if (id < 0) {
          if (a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
          id = 0;
        }
        return id;
      };
      int id = ok ? page_of(t1 - 1) : -1;
      const bool began = ok;
      int issued = 0;
      if (ok && lane == 0) {
        const int rt1 = !split_keys && has1;
        mbar_arrive_expect_tx(&bars[P_Q], (1 + rt1) * pp.tpt * pp.hp * D * 2);
        for (int k = 0; k <= rt1; ++k) {
          const int T = T0 + k, tok = T / pp.head_chunks * pp.tpt, h = hkv * G + T % pp.head_chunks * pp.hp;
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(sm + L::kQ + k * L::kTileBytes + x * 16384, &tmap_q, &bars[P_Q], x * 64, h, tok);
        }
      }
      for (int s = 0; s < nT && ok; ++s) {
        const int c = c0 + s, st = c & 1, n = c >> 1;
        const int here = id;
        if (s + 1 < nT) id = page_of(t1 - 2 - s);
        const int loaded = __popc(__ballot_sync(0xffffffffu, here >= 0));
        ok = n == 0 || mbar_wait(&bars[P_KEMPTY + st], (n - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars[P_KFULL + st], loaded * S * D * 2);
        __syncwarp();
        if (here >= 0)
          for (int x = 0; x < D / 64; ++x)
            tma_load_4d(sm + L::kK + st * L::kTileBytes + x * 16384 + lane * S * 128, &tmap_k, &bars[P_KFULL + st],
                        x * 64, 0, hkv, here);
        ok = n == 0 || mbar_wait(&bars[P_VEMPTY + st], (n - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          mbar_wait_drain(&bars[P_KFULL + st], n & 1);
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[P_VFULL + st], loaded * S * D * 2);
        __syncwarp();
        if (here >= 0)
          for (int x = 0; x < D / 64; ++x)
            tma_load_4d(sm + L::kV + st * L::kTileBytes + x * 16384 + lane * S * 128, &tmap_v, &bars[P_VFULL + st],
                        x * 64, 0, hkv, here);
        ++issued;
      }
      // Every copy issued lands before the segment ends, also where a wait gave up.
      if (began) mbar_wait_drain(&bars[P_Q], seg & 1);
      for (int s = max(issued - 2, 0); s < issued; ++s) {
        const int c = c0 + s;
        mbar_wait_drain(&bars[P_KFULL + (c & 1)], (c >> 1) & 1);
        mbar_wait_drain(&bars[P_VFULL + (c & 1)], (c >> 1) & 1);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------- MMA issuer
      const uint32_t leader = elect_lane();
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = idesc_bf16(128, D, false, true);
      const uint32_t tS[2] = {tbase, tbase + 128};
      const uint32_t tO[2] = {tbase + 256, tbase + 256 + D};
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::kQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sm + L::kK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sm + L::kV), 16384, 1024);
      auto issue_s = [&](int k, int st) {
        const uint64_t q = desc_plus(dQ, split_keys ? 0 : k * L::kTileBytes), b = desc_plus(dK, st * L::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
          umma_ss_e(leader, tS[k], desc_plus(q, off), desc_plus(b, off), idS, ks > 0);
        }
        umma_commit_e(leader, &bars[P_SFULL + k]);
      };
      auto issue_pv = [&](int k, int st, bool acc) {
        const uint64_t v = desc_plus(dV, st * L::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
          const uint32_t pc = tS[k] + 32 * (ks >> 1) + 8 * (ks & 1);
          const uint64_t dv = desc_plus(v, ks * 2048);
          umma_ts_e(leader, tO[k], pc, dv, idO, (acc || ks > 0) ? 1u : 0u);
          umma_ts_e(leader, tO[k], pc + 16, dv, idO, 1u);
        }
      };
      auto wait_k = [&](int s) {
        const int c = c0 + s;
        if (!mbar_wait(&bars[P_KFULL + (c & 1)], (c >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA)) return false;
        tc_fence_after();
        return true;
      };
      auto takes = [&](int k, int s) { return split_keys ? (s & 1) == k : (k == 0 || has1); };
      ok = ok && mbar_wait(&bars[P_Q], seg & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
      for (int s = 0; s < step && s < nT && ok; ++s) {
        if (!(ok = wait_k(s))) break;
        for (int k = 0; k < 2; ++k)
          if (takes(k, s)) issue_s(k, (c0 + s) & 1);
        umma_commit_e(leader, &bars[P_KEMPTY + ((c0 + s) & 1)]);
      }
      int done[2] = {0, 0};
      for (int s = 0; s < nT && ok; ++s) {
        const int c = c0 + s, st = c & 1;
        ok = mbar_wait(&bars[P_VFULL + st], (c >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
        bool kready = false;
        for (int k = 0; k < 2 && ok; ++k) {
          if (!takes(k, s)) continue;
          ok = mbar_wait(&bars[P_PFULL + k], (sc[k] + done[k]) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
          if (!ok) break;
          tc_fence_after();
          issue_pv(k, st, done[k] > 0);
          ++done[k];
          if (s + step < nT) {
            if (!kready && !(ok = wait_k(s + step))) break;
            kready = true;
            issue_s(k, (c + step) & 1);
          } else {
            umma_commit_e(leader, &bars[P_OFINAL + k]);
          }
        }
        if (!ok) break;
        umma_commit_e(leader, &bars[P_VEMPTY + st]);
        if (kready) umma_commit_e(leader, &bars[P_KEMPTY + ((c + step) & 1)]);
      }
    } else if (warp >= 10) {
      // ------------------------------------------------------------ gates
      const int head0 = hkv * G;
      for (int s = 0; s < nT && ok; ++s) {
        const int c = c0 + s, st = c & 1, n = c >> 1;
        if ((c & 1) != warp - 10) continue;
        const int t = t1 - 1 - s, j0 = t * kTile, j = j0 + lane * 4;
        const bool in = j < P;
        const int page = in ? max(prefix_page(a, j), 0) : 0, slot = j % S;
        const int last = P - 1, lpage = max(prefix_page(a, last), 0);
        ok = n == 0 || mbar_wait(&bars[P_GEMPTY + st], (n - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        float* kap = reinterpret_cast<float*>(sm + L::kKap) + st * pp.hp * kKapPitch * pp.kap_tiles;
        for (int k = 0; k < pp.kap_tiles; ++k) {
          // the heads of row tile T0 + k; the same as T0's where a group is one chunk (kap_tiles 1)
          const int h0 = head0 + (T0 + k) % pp.head_chunks * pp.hp;
#pragma unroll 4
          for (int g = 0; g < pp.hp; ++g) {
            const int h = min(h0 + g, head0 + G - 1);
            const float2 cl = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, lpage, h));
            const float gl = a.g[g_offset(a, lpage, h, last % S)];
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            float2 base = make_float2(0.f, 0.f);
            if (in) {
              x = *reinterpret_cast<const float4*>(a.g + g_offset(a, page, h, slot));
              base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
            }
            if (p.bias_from_j) {
              const float before = __shfl_up_sync(0xffffffffu, x.w, 1);
              x = make_float4(slot == 0 ? 0.f : before, x.x, x.y, x.z);
            }
            // (base - c_last) in two parts each, then the sum within the page
            const float d = ((base.x - cl.x) + (base.y - cl.y)) - gl;
            *reinterpret_cast<float4*>(kap + (k * pp.hp + g) * kKapPitch + lane * 4) =
                make_float4((d + x.x) * kLog2e, (d + x.y) * kLog2e, (d + x.z) * kLog2e, (d + x.w) * kLog2e);
          }
        }
        if (j0 + kTile > P) {
          // Slots behind the prefix's end may hold anything: V there becomes 0 (its weights are 0).
          ok = mbar_wait(&bars[P_VFULL + st], n & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t sv = smem_u32(sm + L::kV + st * L::kTileBytes);
          for (int e = lane; e < (j0 + kTile - P) * (D / 8); e += 32) {
            const int row = P - j0 + e / (D / 8), x = e % (D / 8);
            sts_v4(sv + (x >> 3) * 16384 + row * 128 + (x & 7) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[P_GFULL + st]);
      }
    } else {
      // ----------------------------------------------- softmax, epilogue
      const int k = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
      const int mine = k ? n1 : n0;
      const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
      const uint32_t tS = tbase + k * 128 + lane_off, tO = tbase + 256 + k * D + lane_off;
      const int kap_row = (pp.kap_tiles > 1 ? k * pp.hp : 0) + r % pp.hp;
      float m = -INFINITY, l = 0.f;
      int q = 0;  // tiles of this stream so far
      for (int s = 0; s < nT && ok; ++s) {
        if (split_keys && (s & 1) != k) continue;
        const int c = c0 + s, st = c & 1, t = t1 - 1 - s;
        const bool work = mine > 0;
        ok = (!work || mbar_wait(&bars[P_SFULL + k], (sc[k] + q) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA)) &&
             mbar_wait(&bars[P_GFULL + st], (c >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (work) {
          tc_fence_after();
          const float* kap = reinterpret_cast<const float*>(sm + L::kKap) +
                             ((size_t)st * pp.hp * pp.kap_tiles + kap_row) * kKapPitch;
          const int lim = P - t * kTile;
          const float top = lim < kTile ? row_top<true>(tS, kap, p.scale2, lim) : row_top<false>(tS, kap, p.scale2, 0);
          const bool raise = top > m + kRaise;
          if (__any_sync(0xffffffffu, raise)) {
            const float alpha = raise ? ex2_approx(m - top) : 1.f;
            l *= alpha;
            if (q > 0) {  // O is settled: this S was committed after the previous P V
#pragma unroll 1
              for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                tmem_ld32(tO + x, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tO + x, o);
              }
            }
            if (raise) m = top;
          }
          const float off = m == -INFINITY ? 0.f : m;
          l += lim < kTile ? row_exp<true>(tS, kap, p.scale2, off, lim) : row_exp<false>(tS, kap, p.scale2, off, 0);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          if (work) mbar_arrive(&bars[P_PFULL + k]);
          mbar_arrive(&bars[P_GEMPTY + st]);
        }
        ++q;
      }
      const size_t slot = ((size_t)(blockIdx.x + item) * 2 + k) * kTile + r;
      if (mine > 0) {
        ok = ok && mbar_wait(&bars[P_OFINAL + k], oc[k] & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 32) {
            uint32_t o[32];
            tmem_ld32(tO + x, o);
            tmem_ld_wait();
            uint4* dst = reinterpret_cast<uint4*>(pp.po + slot * D + x);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          pp.ml[slot] = make_float2(m, l);
        }
      } else if (split_keys) {
        pp.ml[slot] = make_float2(-INFINITY, 0.f);  // one key tile: this stream had none
      }
    }
    // The segment ends for all roles at once: Q, S and O are free for the next.
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c0 += nT;
    sc[0] += n0;
    sc[1] += n1;
    oc[0] += n0 > 0;
    oc[1] += n1 > 0;
    ++seg;
    u += nT;
  }
  if (warp == 9) {
    // Every MMA issued must retire before tensor memory is freed.
    umma_commit_e(elect_lane(), &bars[P_DONE]);
    mbar_wait_drain(&bars[P_DONE], 0);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
cudaError_t launch(const DecodeParams& p, const CUtensorMap* maps, cudaStream_t s) {
  using L = PrefixLayout<D>;
  auto kernel = prefix_kernel<D>;
  // At least 116 KB, so that one CTA, which takes all of tensor memory, is ever resident on an SM.
  size_t smem = 1024 + L::kKap + sizeof(float) * 2 * p.pre.kap_tiles * p.pre.hp * kKapPitch;
  static_assert(1024 + PrefixLayout<128>::kKap + 4 * 2 * 2 * kMaxHp * kKapPitch <= 232448 - 512, "shared memory");
  if (smem < 118784) smem = 118784;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  TraceScope trace("prefix", s);
  kernel<<<kSMs, kPrefixThreads, smem, s>>>(maps[0], maps[1], maps[2], p);
  return cudaGetLastError();
}

}  // namespace

PrefixPlan prefix_plan(const PagedArgs& a) {
  PrefixPlan x = {};
  const int G = a.H / a.Hkv;
  x.hp = G < kMaxHp ? G : kMaxHp;
  x.head_chunks = ceil_div(G, x.hp);
  x.tpt = kTile / x.hp;
  if (x.tpt > a.rows) x.tpt = a.rows;
  x.row_tiles = ceil_div(a.rows, x.tpt) * x.head_chunks;
  x.items = x.row_tiles == 1 ? 1 : ceil_div(x.row_tiles, 2);
  // Two row tiles of an item have different heads where a group is several chunks.
  x.kap_tiles = x.head_chunks > 1 ? 2 : 1;
  x.key_tiles = ceil_div(a.prefix_len, kTile);
  x.workers = kSMs;
  return x;
}

cudaError_t launch_prefix(const DecodeParams& p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  CUtensorMap maps[3];
  if (!make_q_rows_map(&maps[0], p.q, a.d, a.H, a.rows, p.q_stride, p.pre.hp, p.pre.tpt) ||
      !make_page_map(&maps[1], a.k, a.d, a.page_size, a.Hkv, a.num_pages, a.page_size) ||
      !make_page_map(&maps[2], a.v, a.d, a.page_size, a.Hkv, a.num_pages, a.page_size))
    return cudaErrorInvalidValue;
  return a.d == 64 ? launch<64>(p, maps, s) : launch<128>(p, maps, s);
}

}  // namespace fox
