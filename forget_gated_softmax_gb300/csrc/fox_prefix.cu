// Attention of a batch to the prefix that its sequences share, computed once for all of them, bf16.
//
// c_i is constant along row i and cancels in the softmax, so against the prefix every query row of
// every sequence sees the same matrix of keys and the same bias c_last - c_j (c_last: the cumulative
// log gate of the prefix's last token). All rows of a key head therefore form one tall matrix: 128-row
// tiles against 128-key tiles on the tensor cores, K and V read from memory once for all sequences
// instead of once a sequence. The rows leave unnormalised partial results, which the merge joins with
// those of the sequences' own keys; the row's c_i - c_last enters there.
//
// A row tile is `hp` query heads of the key head's group x `tpt` tokens: row r is head r / tpt, token
// r % tpt, so that most warps' rows have one head and read its gate terms by one address. Key tiles of an
// item (key head, row tiles) run from the last to the first: the bias falls with distance, so the first
// tile nearly always holds the row maximum. Work is split like the own keys' (fox_paged.h): the items' key
// tiles on one line, equal ranges of it to the CTAs, one CTA an SM.
//
// Two streams of softmax warps share the tensor core, each with its S and O in tensor memory:
//   more than one row tile a key head: an item is two row tiles, one a stream, on the same key tiles;
//   one row tile (kSplit): the streams take alternate key tiles, and leave a partial result each.
// A tile passes between softmax and tensor core in two halves of 64 keys: once a half's P V is issued, S of
// the same half of the next tile is, into the columns that P leaves. So the softmax of one half runs while
// the other is multiplied (S of whole tiles: 162 against 150 us at 32768 keys and 1024 rows a key head,
// although MMAs 64 columns wide read Q twice).
// Warp roles (512 threads): warps 0-3 and 4-7 the streams' softmax (thread = row = TMEM lane), warp 8
// loads Q and K, warps 9 and 14 issue the streams' MMAs (one warp for both spent 1.7 us a key tile on
// waits, fences and commits that two have side by side), warps 10-11 load V and make the gate terms
// log2 e (c_j - c_last) of a key tile's keys and the row tile's heads, a stage each, and warps 12, 13 and 15
// turn each V tile from bf16 to fp16 in place (kV16: only clear what is behind the prefix's end).
//
// P V runs in fp16, as in fox_attn_fwd_kernel and for its reason: with bf16 P its 8 significant bits add an
// error as large as O's own rounding. Two bf16 terms a weight (as in fox_decode_mma.cu, where products
// cost nothing) made the tensor core the bound: 2.8 us a pair of 128 x 128 tiles, against 2.2 now. A magnitude
// of 65536 or more in V (outside fp16) sets DEV_ERR_RANGE. A 32-column chunk of S, once read, holds its P.
//
// 32768 keys, 256 sequences x 4 heads a key head, 8 of these, d = 128: 133 us, 1030 TFLOP/s, 53 % of
// cuBLAS's burst bf16 rate. What bounds it is the chain of each stream, S -> softmax -> P V, and no unit: the tensor pipe is 48 %
// active, issue slots 54 %. Of the time between two instructions of a warp a third goes on what it waits to be loaded (S from
// tensor memory), then fixed latencies (15 %), the scheduler's other warps (13 %) and instruction fetch (8 %): two softmax
// warps a scheduler cannot cover them. Without the conversion of V it took 5 us less; 168 registers for the softmax (88 for the others) took no less.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_decode.h"

namespace fox {
namespace {

constexpr int kPrefixThreads = 512;
constexpr int kConverters = 3;  // two: 142 us where three take 137
constexpr int kMaxHp = 16;
constexpr int kOpening = 4;  // key tiles' time
constexpr int kKapPitch = kTile + 4;  // floats: the heads' rows start in different banks
constexpr float kRaise = 4.0f;        // log2 units that a row may pass its running maximum by
// P is 2^kLift times the weight against the running maximum (and below 2^15 with what that may be passed by): fp16
// then holds weights down to 2^-25 with all its bits and the least 2^-35, where a long prefix's many small ones count.
constexpr float kLift = 11.0f;

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
  P_VFULL = 5,    // +V stage
  P_VEMPTY = 8,
  P_VREADY = 11,  // V in fp16, and 0 behind the prefix's end
  P_GFULL = 14,   // +stage: the key tile's gate terms are in place
  P_GEMPTY = 16,
  P_SFULL = 18,   // +2 stream + half of the tile's keys
  P_PFULL = 22,   // +2 stream + half
  P_PVDONE = 26,  // +2 stream + half: that P V is through
  P_OFINAL = 30,  // +stream
  P_DONE = 32,
  P_COUNT = 33,
};

__host__ __device__ constexpr int e_bar(int stream, int half) { return 2 * stream + half; }

template <int D, bool kSplit, bool kV16>  // kV16: V comes in fp16
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
  constexpr int step = kSplit ? 2 : 1;  // key tiles from one of a stream's to its next

  grid_dep_wait();     // before tensor memory is taken, which what is ahead may still have to take itself
  grid_dep_trigger();  // the own keys' kernel may start where this one leaves room: it needs nothing from here
  if (threadIdx.x < P_COUNT) {
    const int i = threadIdx.x;
    mbar_init(&bars[i], i >= P_PFULL && i < P_PFULL + 4 ? 4
                        : i >= P_GEMPTY && i < P_GEMPTY + 2 ? (kSplit ? 4 : 8)
                        : i >= P_VREADY && i < P_VREADY + 3 ? kConverters
                        : i == P_KEMPTY || i == P_KEMPTY + 1 || (i >= P_VEMPTY && i < P_VEMPTY + 3)
                            ? (kSplit ? 1 : 2)  // the streams that use a key tile
                        : i == P_DONE ? 2
                                      : 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_word = 0;
  if (warp == 9) {
    tmem_alloc(&tmem_word, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_word;

  const int u_end = min(a.Hkv * pp.items * pp.line, static_cast<int>(blockIdx.x + 1) * pp.each);
  int u = blockIdx.x * pp.each;

  // V's stages: with one row tile three, the third in the place of a second row tile's Q, since a stream then has
  // every other tile and would wait for its next V from the end of its last P V on (52.3 -> 50.1 us at 32 sequences behind 16384 tokens,
  // 75.0 -> 68.5 at 30 behind 50000).
  auto v_round = [](int c) { return kSplit ? c / 3 : c >> 1; };  // of key tile c, and its stage
  auto v_stage = [](int c) { return kSplit ? c % 3 : c & 1; };
  auto v_at = [](int st) { return kSplit && st == 2 ? L::kQ + L::kTileBytes : L::kV + st * L::kTileBytes; };

  bool ok = true;              // of this thread's role
  uint32_t vmax = 0u;          // converters: largest |v| bit pattern seen, per bf16 half
  int c0 = 0;                  // key tiles before this segment (ring position)
  int sc[2] = {0, 0};          // tiles of each stream before this segment
  int oc[2] = {0, 0};          // segments in which each stream had tiles
  int seg = 0;
  while (u < u_end) {
    // A segment: key tiles t1 - 1 down to t0 of item (hkv, it).
    const int item = u / pp.line, hkv = item / pp.items, it = item % pp.items;
    const int t0 = u % pp.line, t1 = min(pp.key_tiles, t0 + (u_end - u));
    if (t0 >= t1) {  // an item's empty units
      u = (item + 1) * pp.line;
      continue;
    }
    const int nT = t1 - t0;
    const int T0 = kSplit ? 0 : 2 * it;  // row tile of stream 0; stream 1 has the next, or the same
    const bool has1 = kSplit ? nT > 1 : T0 + 1 < pp.row_tiles;
    const int n0 = kSplit ? (nT + 1) / 2 : nT, n1 = kSplit ? nT / 2 : (has1 ? nT : 0);
    const int npages = ceil_div(P, S);
    // Lane i: page i of key tile t, -1 where the prefix has ended.
    auto page_of = [&](int t) {
      const int i = t * (kTile >> a.page_shift) + lane;
      return t >= 0 && lane < kTile >> a.page_shift && i < npages ? checked_page(a, a.prefix[i]) : -1;
    };
    if (warp == 8) {
      // -------------------------------------------------------- Q and K
      const uint64_t policy = stream_policy();
      int id = ok ? page_of(t1 - 1) : -1, issued = 0;
      const bool began = ok;
      if (ok) {
        const int rt1 = !kSplit && has1;
        if (lane == 0) mbar_arrive_expect_tx(&bars[P_Q], (1 + rt1) * pp.tpt * pp.hp * D * 2);
        __syncwarp();
        if (lane < pp.hp)  // a head a lane
#pragma unroll 1
          for (int k = 0; k <= rt1; ++k) {
            const int T = T0 + k, tok = T / pp.head_chunks * pp.tpt, h = hkv * G + T % pp.head_chunks * pp.hp + lane;
#pragma unroll 1
            for (int x = 0; x < D / 64; ++x)
              tma_load_3d(sm + L::kQ + k * L::kTileBytes + x * 16384 + lane * pp.tpt * 128, &tmap_q, &bars[P_Q], x * 64, h,
                          tok);
          }
        __syncwarp();
      }
#pragma unroll 1
      for (int s = 0; s < nT && ok; ++s) {
        const int c = c0 + s, st = c & 1, n = c >> 1, here = id;
        if (s + 1 < nT) id = page_of(t1 - 2 - s);
        const int loaded = __popc(__ballot_sync(0xffffffffu, here >= 0));
        ok = n == 0 || mbar_wait(&bars[P_KEMPTY + st], (n - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars[P_KFULL + st], loaded * S * D * 2);
        __syncwarp();
        if (here >= 0)
#pragma unroll 1
          for (int x = 0; x < D / 64; ++x)
            tma_load_4d_by(policy, sm + L::kK + st * L::kTileBytes + x * 16384 + lane * S * 128, &tmap_k, &bars[P_KFULL + st],
                        x * 64, 0, hkv, here);
        ++issued;
      }
      // Every copy issued lands before the segment ends, also where a wait gave up.
      if (began) mbar_wait_drain(&bars[P_Q], seg & 1);
#pragma unroll 1
      for (int s = max(issued - 2, 0); s < issued; ++s)
        mbar_wait_drain(&bars[P_KFULL + ((c0 + s) & 1)], ((c0 + s) >> 1) & 1);
    } else if (warp == 9 || warp == 14) {
      // ------------------------------------------------------ MMA issuers
      const int k = warp == 14;  // the stream
      const int mine = k ? n1 : n0;
      const uint32_t leader = elect_lane();
      constexpr uint32_t idS = idesc_bf16(128, 64, false, false);
      constexpr uint32_t idO = idesc_f16(128, D, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::kQ + (kSplit ? 0 : k * L::kTileBytes)), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sm + L::kK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sm + L::kV), 16384, 1024);
      const uint32_t tS = tbase + k * 128, tO = tbase + 256 + k * D;
      ok = ok && mbar_wait(&bars[P_Q], seg & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
      // Step s: P V of the stream's key tile s, and S of its next; the step before the first only has the S.
#pragma unroll 1
      for (int s = kSplit ? k - 2 : -1, q = -1; s < nT && ok; s += step, ++q) {
        const int c = c0 + s, cn = c + step;
        const bool pv = q >= 0, next = s + step < nT;
        const int vn = v_round(c), vs = v_stage(c);
        if (mine == 0) {  // an item's missing second row tile: the stages are let go as they come
          if (next) {
            ok = mbar_wait(&bars[P_KFULL + (cn & 1)], (cn >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
            if (ok && lane == 0) mbar_arrive(&bars[P_KEMPTY + (cn & 1)]);
          }
          if (ok && pv) {
            ok = mbar_wait(&bars[P_VREADY + vs], vn & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
            if (ok && lane == 0) mbar_arrive(&bars[P_VEMPTY + vs]);
          }
          continue;
        }
        const uint64_t vd = dV + static_cast<int64_t>((v_at(vs) - L::kV) >> 4), kd = dK + ((cn & 1) ? L::kTileBytes >> 4 : 0);
        if (pv) ok = mbar_wait(&bars[P_VREADY + vs], vn & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
#pragma unroll 1
        for (int h = 0; h < 2 && ok; ++h) {
          if (pv) {
            ok = mbar_wait(&bars[P_PFULL + e_bar(k, h)], (sc[k] + q) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
            if (!ok) break;
            tc_fence_after();
            // O += P V over 64 keys: rows 64 h on of V
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_ts_e(leader, tO, tS + h * 64 + 32 * (ks >> 1) + 8 * (ks & 1),
                        vd + static_cast<uint64_t>((h * 8192 + ks * 2048) >> 4), idO, q > 0 || h > 0 || ks > 0);
            umma_commit_e(leader, &bars[P_PVDONE + e_bar(k, h)]);
            if (h == 1) umma_commit_e(leader, &bars[P_VEMPTY + vs]);
          }
          if (next) {
            if (h == 0) ok = mbar_wait(&bars[P_KFULL + (cn & 1)], (cn >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
            if (!ok) break;
            if (!pv) tc_fence_after();
            // S of the same 64 columns, whose P is read by then (MMAs run in order)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_ss_e(leader, tS + h * 64, dQ + static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                        kd + static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32 + h * 8192) >> 4), idS, ks > 0);
            umma_commit_e(leader, &bars[P_SFULL + e_bar(k, h)]);
            if (h == 1) umma_commit_e(leader, &bars[P_KEMPTY + (cn & 1)]);
          } else if (h == 1) {
            umma_commit_e(leader, &bars[P_OFINAL + k]);
          }
        }
      }
    } else if (warp >= 12) {
      // --------------------------------------------- V from bf16 to fp16
      // The warps take 16-byte pieces of the swizzled layout TMA wrote in turn; the conversion is per element,
      // so the layout is unchanged. Slots behind the prefix's end may hold anything: V there becomes 0 (its
      // weights are 0).
      const int first = (warp == 15 ? kConverters - 1 : warp - 12) * 32 + lane;
#pragma unroll 1
      for (int s = 0; s < nT && ok; ++s) {
        const int c = c0 + s, vn = v_round(c), vs = v_stage(c), keys = P - (t1 - 1 - s) * kTile;
        ok = mbar_wait(&bars[P_VFULL + vs], vn & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4* tile = reinterpret_cast<uint4*>(sm + v_at(vs));
        if (keys < kTile)
#pragma unroll 1
          for (int e = first; e < L::kTileBytes / 16; e += 32 * kConverters)  // eight pieces a row of 64 channels
            if (((e >> 3) & (kTile - 1)) >= keys) tile[e] = make_uint4(0, 0, 0, 0);
        // No further unrolled: in bursts the softmax waits for its loads of shared memory (by 2 137 us, by 4 153,
        // by 8 171 at 32768 keys and 1024 rows a key head).
#pragma unroll 2
        for (int e = first; !kV16 && e < L::kTileBytes / 16; e += 32 * kConverters) {
          const uint4 w = tile[e];
          const uint32_t in[4] = {w.x, w.y, w.z, w.w};
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = in[i];
            out[i] = pack_f16x2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
            asm("max.u16x2 %0, %0, %1;" : "+r"(vmax) : "r"(x & 0x7FFF7FFFu));
          }
          tile[e] = make_uint4(out[0], out[1], out[2], out[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[P_VREADY + vs]);
      }
    } else if (warp >= 10) {
      // ------------------------------------------------------ V and gates
      const int head0 = hkv * G, mine = warp - 10;  // the stage of this warp
      const int s0 = (c0 & 1) == mine ? 0 : 1;
      const int last = P - 1, lpage = checked_page(a, a.prefix[last >> a.page_shift]);
      const uint64_t policy = stream_policy();
      int id = ok ? page_of(t1 - 1 - s0) : -1, issued = 0;
#pragma unroll 1
      for (int s = s0; s < nT && ok; s += 2) {
        const int c = c0 + s, st = c & 1, n = c >> 1, vn = v_round(c), vs = v_stage(c), here = id;
        const int t = t1 - 1 - s, j0 = t * kTile, j = j0 + lane * 4;
        const bool in = j < P;
        id = page_of(s + 2 < nT ? t - 2 : -1);
        const int loaded = __popc(__ballot_sync(0xffffffffu, here >= 0));
        const int page = max(__shfl_sync(0xffffffffu, here, (lane * 4) >> a.page_shift), 0), slot = j & (S - 1);
        float* kap = reinterpret_cast<float*>(sm + L::kKap) + st * pp.hp * kKapPitch * pp.kap_tiles;
        bool first = true;
#pragma unroll 1
        for (int g0 = 0; g0 < pp.hp * pp.kap_tiles && ok; g0 += 4) {
          // Four heads at a time, their loads on the way before anything is waited for.
          float4 x[4];
          float2 base[4], cl[4];
          float gl[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // of row tile T0 + k, or of either where a group is one chunk (kap_tiles 1)
            const int g = min(g0 + i, pp.hp * pp.kap_tiles - 1), k = g / pp.hp;
            const int h = min(head0 + (T0 + k) % pp.head_chunks * pp.hp + g - k * pp.hp, head0 + G - 1);
            cl[i] = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, lpage, h));
            gl[i] = a.g[g_offset(a, lpage, h, last & (S - 1))];
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            base[i] = make_float2(0.f, 0.f);
            if (in) {
              x[i] = *reinterpret_cast<const float4*>(a.g + g_offset(a, page, h, slot));
              base[i] = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
            }
          }
          if (first) {
            first = false;
            ok = vn == 0 || mbar_wait(&bars[P_VEMPTY + vs], (vn - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars[P_VFULL + vs], loaded * S * D * 2);
            __syncwarp();
            if (here >= 0)
#pragma unroll 1
              for (int y = 0; y < D / 64; ++y)
                tma_load_4d_by(policy, sm + v_at(vs) + y * 16384 + lane * S * 128, &tmap_v, &bars[P_VFULL + vs],
                            y * 64, 0, hkv, here);
            ++issued;
            ok = n == 0 || mbar_wait(&bars[P_GEMPTY + st], (n - 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (g0 + i >= pp.hp * pp.kap_tiles) break;
            float4 y = x[i];
            if (p.bias_from_j) {
              const float before = __shfl_up_sync(0xffffffffu, y.w, 1);
              y = make_float4(slot == 0 ? 0.f : before, y.x, y.y, y.z);
            }
            // A slot behind the prefix's end may hold anything: some finite value instead (its S is masked).
            if (j >= P) y.x = 0.f;
            if (j + 1 >= P) y.y = 0.f;
            if (j + 2 >= P) y.z = 0.f;
            if (j + 3 >= P) y.w = 0.f;
            // (base - c_last) in two parts each, then the sum within the page
            const float d = ((base[i].x - cl[i].x) + (base[i].y - cl[i].y)) - gl[i];
            *reinterpret_cast<float4*>(kap + (g0 + i) * kKapPitch + lane * 4) =
                make_float4((d + y.x) * kLog2e, (d + y.y) * kLog2e, (d + y.z) * kLog2e, (d + y.w) * kLog2e);
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[P_GFULL + st]);
      }
      // Every copy issued lands before the segment ends, also where a wait gave up (of this warp's last two, one
      // may be through and its stage taken by the other warp's next: then the wait only runs out). Where none did, the conversion has seen them all.
      if (!ok || *abort_flag)
#pragma unroll 1
        for (int i = max(issued - 2, 0); i < issued; ++i) {
          const int c = c0 + s0 + 2 * i;
          mbar_wait_drain(&bars[P_VFULL + v_stage(c)], v_round(c) & 1);
        }
    } else {
      // ----------------------------------------------- softmax, epilogue
      const int k = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
      const int mine = k ? n1 : n0;
      const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
      const uint32_t tO = tbase + 256 + k * D + lane_off;
      const int kap_row = (pp.kap_tiles > 1 ? k * pp.hp : 0) + min(r / pp.tpt, pp.hp - 1);
      const float2 nsc = make_float2(-p.scale2, -p.scale2);
      float m = -INFINITY, l = 0.f;
      int q = 0;  // tiles of this stream so far
#pragma unroll 1
      for (int s = 0; s < nT && ok; ++s) {
        if (kSplit && (s & 1) != k) continue;
        const int c = c0 + s, st = c & 1;
        ok = mbar_wait(&bars[P_GFULL + st], (c >> 1) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_SYNC);
#pragma unroll 1
        for (int h = 0; h < 2 && mine > 0 && ok; ++h) {
          ok = mbar_wait(&bars[P_SFULL + e_bar(k, h)], (sc[k] + q) & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
          ok = __all_sync(0xffffffffu, ok);  // the tcgen05 loads below are warp-collective
          if (!ok) break;
          tc_fence_after();
          const uint32_t tS = tbase + k * 128 + h * 64 + lane_off;
          const float* kap = reinterpret_cast<const float*>(sm + L::kKap) +
                             (st * pp.hp * pp.kap_tiles + kap_row) * kKapPitch + h * 64;
          const int lim = P - (t1 - 1 - s) * kTile - h * 64;  // columns from lim on are not keys
          // P and the row's maximum in one pass, with the running maximum; where a row has passed that by more
          // than 2^4 (rare after the first tile), once more with the new one: S is still there.
          uint32_t pk[32];
          float2 sum;
#pragma unroll 1
          for (int again = 0;; ++again) {
            const float off = m == -INFINITY ? 0.f : m - kLift;
            const float2 noff = make_float2(-off, -off);
            float mn = INFINITY;  // of tn_j = kap_j - scale2 S_j = -x_j
            sum = make_float2(0.f, 0.f);
            uint32_t rawb[2][32];
            tmem_ld32(tS, rawb[0]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              tmem_ld_wait();
              if (x == 0) tmem_ld32(tS + 32, rawb[1]);
              float2* tn = reinterpret_cast<float2*>(rawb[x]);
              if (lim < 64) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {  // S of no key is the least there is
                  if (32 * x + 2 * j >= lim) tn[j].x = -INFINITY;
                  if (32 * x + 2 * j + 1 >= lim) tn[j].y = -INFINITY;
                }
              }
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float4 kk = lds_f4(kap + 32 * x + 2 * j);
                const float2 ta = ffma2(tn[j], nsc, make_float2(kk.x, kk.y));
                const float2 tc = ffma2(tn[j + 1], nsc, make_float2(kk.z, kk.w));
                mn = fmin3(fmin3(mn, ta.x, ta.y), tc.x, tc.y);
                const float2 wa = fsub2(noff, ta), wc = fsub2(noff, tc);
                const float2 pa = make_float2(ex2_approx(wa.x), ex2_approx(wa.y));
                const float2 pc = make_float2(ex2_approx(wc.x), ex2_approx(wc.y));
                sum = fadd2(sum, fadd2(pa, pc));
                pk[16 * x + j] = pack_f16x2(pa.x, pa.y);
                pk[16 * x + j + 1] = pack_f16x2(pc.x, pc.y);
              }
            }
            const bool raise = again == 0 && -mn > m + kRaise;
            if (!__any_sync(0xffffffffu, raise)) break;
            const float alpha = raise ? ex2_approx(m + mn) : 1.f;
            l *= alpha;
            if (q > 0 || h > 0) {
              // O has to be settled: the P V before this half's, issued after its S, through.
              ok = mbar_wait(&bars[P_PVDONE + e_bar(k, h ^ 1)], (sc[k] + q - (h == 0)) & 1, abort_flag, a.err,
                             DEV_ERR_TIMEOUT_MMA);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < D; x += 16) {
                uint32_t o[16];
                tmem_ld16(tO + x, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(tO + x, o);
              }
            }
            if (raise) m = -mn;
          }
          if (!ok) break;
          tmem_st16(tS, pk);
          tmem_st16(tS + 32, pk + 16);
          l += sum.x + sum.y;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[P_PFULL + e_bar(k, h)]);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bars[P_GEMPTY + st]);
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
          pp.ml[slot] = make_float2(m - kLift, l);
        }
      } else if (kSplit) {
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
  if (warp >= 12 && warp != 14) {
    // |v| >= 65536 (bf16 pattern 0x4780 and above, infinities included) is outside fp16.
    const bool over = (vmax & 0xFFFFu) >= 0x4780u || (vmax >> 16) >= 0x4780u;
    if (__any_sync(0xffffffffu, over) && lane == 0 && a.err) atomicOr(a.err, DEV_ERR_RANGE);
  }
  if (warp == 9 || warp == 14) {
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

template <int D, bool kSplit, bool kV16>
cudaError_t launch(const DecodeParams& p, const CUtensorMap* maps, cudaStream_t s) {
  using L = PrefixLayout<D>;
  auto kernel = prefix_kernel<D, kSplit, kV16>;
  // At least 116 KB, so that one CTA, which takes all of tensor memory, is ever resident on an SM.
  constexpr size_t kLeast = 118784;
  size_t smem = 1024 + L::kKap + sizeof(float) * 2 * p.pre.kap_tiles * p.pre.hp * kKapPitch;
  if (smem < kLeast) smem = kLeast;
  // One limit for every call (launch in fox_decode_mma.cu has the reason).
  constexpr size_t kMost = 1024 + L::kKap + sizeof(float) * 2 * 2 * kMaxHp * kKapPitch;
  constexpr size_t kLimit = kMost < kLeast ? kLeast : kMost;
  static_assert(kLimit <= 232448 - 512, "shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLimit));
  if (e != cudaSuccess) return e;
  TraceScope trace("prefix", s);
  const cudaError_t f =
      launch_dependent(kernel, dim3(kSMs), dim3(kPrefixThreads), smem, s, maps[0], maps[1], maps[2], p);
  return f != cudaSuccess ? f : cudaGetLastError();
}

}  // namespace

PrefixPlan prefix_plan(const PagedArgs& a) {
  PrefixPlan x = {};
  const int G = a.H / a.Hkv;
  x.hp = G < kMaxHp ? G : kMaxHp;
  x.head_chunks = ceil_div(G, x.hp);
  x.tpt = kTile / x.hp / 8 * 8;  // each head's rows start at a whole swizzle block of shared memory
  x.row_tiles = ceil_div(a.rows, x.tpt) * x.head_chunks;
  x.items = x.row_tiles == 1 ? 1 : ceil_div(x.row_tiles, 2);
  // Two row tiles of an item have different heads where a group is several chunks.
  x.kap_tiles = x.head_chunks > 1 ? 2 : 1;
  x.key_tiles = ceil_div(a.prefix_len, kTile);
  x.workers = kSMs;
  // Equal ranges of all items' key tiles and of kOpening empty units behind each item, the time that beginning
  // a second item costs a CTA (its pipeline runs empty and fills again); or, where that leaves the longest range
  // no longer, a whole number of CTAs an item, none of which begins a second. (Four such units or ten: 133 to 135 us
  // at 32768 keys and 4 items a key head, without them 137.)
  const int n = a.Hkv * x.items;
  x.line = x.key_tiles + kOpening;
  x.each = units_per_worker(n * x.line, x.workers);
  const int ctas = x.workers / n;
  if (ctas > 0) {
    const int whole = ceil_div(x.key_tiles, ctas);
    if (whole <= x.each) {
      x.each = whole;
      x.line = whole * ceil_div(x.key_tiles, whole);
    }
  }
  return x;
}

namespace {
template <bool kV16>
cudaError_t launch_as(const DecodeParams& p, const CUtensorMap* maps, cudaStream_t s) {
  if (p.pre.row_tiles == 1) return p.a.d == 64 ? launch<64, true, kV16>(p, maps, s) : launch<128, true, kV16>(p, maps, s);
  return p.a.d == 64 ? launch<64, false, kV16>(p, maps, s) : launch<128, false, kV16>(p, maps, s);
}
}  // namespace

cudaError_t launch_prefix(const DecodeParams& p, bool v16, cudaStream_t s) {
  const PagedArgs& a = p.a;
  CUtensorMap maps[3];
  if (!make_q_rows_map(&maps[0], p.q, a.d, a.H, a.rows, p.q_stride, 1, p.pre.tpt) ||
      !make_page_map(&maps[1], a.k, a.d, a.page_size, a.Hkv, a.num_pages, a.page_size) ||
      !make_page_map(&maps[2], a.v, a.d, a.page_size, a.Hkv, a.num_pages, a.page_size))
    return cudaErrorInvalidValue;
  return v16 ? launch_as<true>(p, maps, s) : launch_as<false>(p, maps, s);
}

}  // namespace fox
