// Attention of the newest tokens over the 4-bit paged cache, on the tensor cores.
//
// The plan is fox_decode_mma.cu's: one warp a worker of the work line (fox_paged.h) with a ring of key tiles of its own, transposed
// products S^T = K Q^T and O^T += V^T P^T by the register MMAs (16 x 8 x 16), so that the few query rows are the 8-wide side. Bytes
// are a quarter; what a key costs in instructions is more, so the codes' layout (fox_four.h) is made for this kernel:
//
// K. A lane's part of an MMA operand (a token's channels 8 t .. 8 t + 7 of every block) lies side by side. A nibble u + 8 = n at bits 9..6
//   of an fp16 of exponent 0 is 1 + n / 16, at bits 5..2 it is 1 + n / 256: two masks on the word and two on the word rotated by 8 make
//   the eight values of two MMA steps. With q' = 16 q and 256 q in their places the products sum to sum q u plus sums of q alone,
//   which the accumulator begins with (negated; one a block and row). So a block costs 5 instructions and no subtraction, and fp32
//   sums keep 2^-24 of 264 sum |q|. The block's scale multiplies its sum.
// V. ldmatrix.trans turns 16-bit units (four channels of a token) so that a register has the same four channels of two
//   neighbouring tokens: what the V^T operand wants, nibble by nibble. The masks give 1 + n / 1024 and 1 + n / 64, an fma n - 8, exactly.
//   The scales, which vary along the sum, go to P: P s in fp16 (P and s in fp16, so rounded twice by 2^-12), once a block of 32 channels.
// Weights are P = 2^(x - r), with r = the running maximum less `lift`: as fp16 holds 2^15 down to 2^-24, weights down to
//   2^-25 of the largest keep all bits at lift 11. lift falls where scales above 1 are met, so that P s stays below 2^15 too;
//   r moves when a score passes it by lift + 4, or a scale its bound, which one vote finds.
// q in fp16: each row times a power of two so that its largest |q| is in [32, 64); what a bf16 holds is then exact down to 2^-24 of that.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fox_decode_ring.h"
#include "fox_four.h"

namespace fox {
namespace {

constexpr int kRoom = 4;   // log2 units that a score may pass the running maximum by
constexpr int kLift = 11;  // log2 of a weight's largest value against the running maximum, while scales are below 1

template <int D, int NT>
struct Layout4 {
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kStages = 2;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocks = D / kFourBlock;
  static constexpr int kTileBytes = kKeyTile * D / 2;          // codes of K or V of a stage
  static constexpr int kScaleBytes = kKeyTile * kBlocks;       // scales of K or V of a stage
  static constexpr int kStageBytes = 2 * (kTileBytes + kScaleBytes);
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kOutStride = D + 4;
  static_assert(8 * kOutStride * 4 <= kStageBytes, "eight rows pass through a stage that was read");
  static_assert(kRows * kOutStride * 4 <= kStages * kStageBytes, "rows are kept in a ring that was read");
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (w & mask) | 1.0 in both halves, one instruction.
__device__ __forceinline__ uint32_t over_one(uint32_t w, uint32_t mask) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x3C003C00u));
  return d;
}
// The values u of two tokens' channel pairs: nibbles 0 and 1 (of w >> 8: 2 and 3) of both halves.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t w) {  // 1024 (1 + n / 1024) - 1032
  return hfma2(over_one(w, 0x000F000Fu), 0x64006400u, 0xE408E408u);
}
__device__ __forceinline__ uint32_t high_nibbles(uint32_t w) {  // 64 (1 + n / 64) - 72
  return hfma2(over_one(w, 0x00F000F0u), 0x54005400u, 0xD480D480u);
}
__device__ __forceinline__ void bulk_load_by(uint64_t policy, void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// kMany: sequences may bring more than one token, so that rows of a tile may end at different keys.
template <int D, int NT, bool kMany>
__global__ void __launch_bounds__(32 * Layout4<D, NT>::kWarps, 1)
    decode4_kernel(const __grid_constant__ CUtensorMap tmap_g, const __grid_constant__ DecodeParams p, const MmaShape x) {
  using L = Layout4<D, NT>;
  constexpr int W = L::kWarps, NB = L::kBlocks, RowB = D / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int scratch[W];
  __shared__ __align__(8) uint64_t bars[W][L::kStages];
  __shared__ int abort_word;
  __shared__ Kept<L::kRows, W> kept;
  __shared__ int ids[W][2][64];
  __shared__ BlockEnds ends;
  __shared__ ItemRows<L::kRows> rows_of[W];
  __shared__ int offs[kSMs + 1];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &abort_word;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ItemRows<L::kRows>& it = rows_of[warp];
  constexpr int stages = L::kStages;
  uint8_t* ring = sm + warp * stages * L::kStageBytes;
  uint8_t* all_gates = sm + W * stages * L::kStageBytes;
  uint8_t* gates = all_gates + warp * stages * x.gstage;
  uint8_t* q_of = all_gates + W * stages * x.gstage + warp * L::kQBytes;
  SeqEntry* seqs = reinterpret_cast<SeqEntry*>(all_gates + W * (stages * x.gstage + L::kQBytes));

  const bool shared = p.pre.key_tiles > 0;
  if (threadIdx.x == 0) abort_word = 0;
  if (lane == 0) {
    kept.i0[warp] = -1;
    for (int s = 0; s < stages; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
  }
  // Behind a shared prefix's kernels the wait comes last (fox_decode_mma.cu).
  if (!shared) grid_dep_wait();
  grid_dep_trigger();
  scan_sequences(p, seqs, scratch);  // ends with a block barrier
  if (shared && blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += blockDim.x) p.cum[b] = seqs[b].u0;

  const int G = a.H / a.Hkv, Gp = p.Gp, S = a.page_size;
  const int KS = S < kKeyTile ? S : kKeyTile;      // tokens of a sub-page
  const int heads = x.heads, gpitch = x.gpitch;
  const int base_off = (S == 16 ? 2 : 1) * x.gsub;
  const int P = a.prefix_len, tp = p.walk_prefix ? ceil_div(P, kKeyTile) : 0;  // the prefix's tiles come first
  const int total = seqs[a.B].u0 * a.Hkv, each = units_per_worker(total, p.workers);
  const int w = blockIdx.x * W + warp;
  const int u0 = min(total, w * each), count = min(total, u0 + each) - u0;

  const int g8 = lane >> 2, t4 = lane & 3;
  uint32_t qf[NB][NT][4];       // Q^T operand: of block b, its lane's channels 0 1, 2 3, 6 7, 4 5
  float start[NB][NT][2];       // what a block's sum begins with
  float unit[NT][2];            // log2 units of a row's S
  float acc[2 * NB][NT][4];     // O^T: of block b channels 4 g8 + 0, + 1 and + 2, + 3
  float r[NT][2], l[NT][2];     // the reference that weights are taken against, their sum
  int top_e = 0;                // exponent bits of the largest scale of V so far
  Gate2 ci[NT][2];
  int pos[NT][2], gidx[NT][2];
  int last = 0;  // with kMany: own position of the item's last row
  const uint64_t policy = stream_policy();
  const uint32_t vplace = lane * RowB, vturn = NB == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1;

  Place cur = {}, pro = {};
  int since = -stages, asked = 0, filled = 0, ahead = 0;
  if (count > 0) cur = pro = place_of(p, seqs, u0);
  Window now = {}, next = {};
  int left = count, at = 0, buf = 0;
  bool fresh = true, opened = false, ok = true;
  int stage = 0;
  uint32_t phase = 0;

  // Step n consumes tile n and then issues the copies of tile n + stages; the first `stages` only issue.
#pragma unroll 1
  for (int n = -stages; n < count; ++n) {
    if (n == 0 && warp == 0) find_ends<W>(p, seqs, total, each, ends);  // while the first copies are on their way
    if (n >= 0) {
      if (!opened) {
        opened = true;
        if (n - since > 1)
          cp_async_wait<1>();  // asked for before the last step
        else
          cp_async_wait<0>();
        __syncwarp();
        since = n;
        fresh = true;
        top_e = 0;
        const int r0 = cur.rt * p.Rt;
        if (kMany) last = cur.s.own - cur.s.n + min(token_of(p, r0 + p.Rt - 1), cur.s.n - 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // Row nt * 8 + g8: this lane's channels of every block, in fp16 at a power of two.
          const uint8_t* qr = q_of + (nt * 8 + g8) * (D * 2);
          float f[NB][8], most = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 y = *reinterpret_cast<const uint4*>(qr + (((b * 4 + t4) ^ (g8 & 7)) << 4));
            const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[b][2 * i] = __uint_as_float(v[i] << 16);
              f[b][2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
              most = fmaxf(most, fmaxf(fabsf(f[b][2 * i]), fabsf(f[b][2 * i + 1])));
            }
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          // 2^-e brings `most` to [32, 64); in two factors, both of them normal numbers
          const int e = most > 0.f ? min(static_cast<int>(__float_as_uint(most) >> 23), 254) - 127 - 5 : 0;
          const float down0 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23),
                      down1 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
          const float row_unit = p.scale2 / down0 / down1;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // pairs 0 and 3 stand at bits 9..6, pairs 1 and 2 at bits 5..2
              const bool low = i == 1 || i == 2;
              const float up = low ? 256.f : 16.f;
              const uint32_t h = pack_f16x2(f[b][2 * i] * down0 * down1 * up, f[b][2 * i + 1] * down0 * down1 * up);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
              sum -= (back.x + back.y) * (low ? 264.f / 256.f : 24.f / 16.f);
              qf[b][nt][i == 0 ? 0 : i == 1 ? 1 : i == 3 ? 2 : 3] = h;
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            start[b][nt][0] = __shfl_sync(0xffffffffu, sum, t4 * 8);
            start[b][nt][1] = __shfl_sync(0xffffffffu, sum, t4 * 8 + 4);
          }
          unit[nt][0] = __shfl_sync(0xffffffffu, row_unit, t4 * 8);
          unit[nt][1] = __shfl_sync(0xffffffffu, row_unit, t4 * 8 + 4);
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const int rl = nt * 8 + 2 * t4 + e2, rr = r0 + rl, t = token_of(p, rr), g = rr - t * Gp;
            const bool here = t < cur.s.n && g < G;
            pos[nt][e2] = cur.s.own - cur.s.n + t;
            gidx[nt][e2] = here ? (G > L::kRows ? g - r0 % Gp : g) : 0;
            ci[nt][e2] = {-INFINITY, 0.f};  // an empty row's scores are -inf
            if (here) ci[nt][e2] = gate_sum(it.base[rl], it.g[rl]);
            r[nt][e2] = -INFINITY;
            l[nt][e2] = 0.f;
          }
        }
#pragma unroll
        for (int dt = 0; dt < 2 * NB; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[dt][nt][e] = 0.f;
      }
      uint8_t* st = ring + stage * L::kStageBytes;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[warp][stage], phase, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA));
      if (!ok) break;
      cp_async_wait<L::kStages - 1>();  // the stage's bases: so many groups were committed after theirs
      __syncwarp();

      const bool pre = cur.tile < tp;
      const int j0 = (pre ? cur.tile : cur.tile - tp) * kKeyTile, have = pre ? P : cur.s.own, end = pre ? P : kMany ? last + 1 : cur.s.own;
      const uint8_t* sk = st;
      const uint8_t* sv = st + L::kTileBytes;
      const uint8_t* sks = sv + L::kTileBytes;
      uint8_t* svs = st + 2 * L::kTileBytes + L::kScaleBytes;
      if (j0 + kKeyTile > have) {
        // Slots behind the end may hold anything, NaN scales among them: V's scales there become 0 (K's scores are left out).
        if (lane >= have - j0)
#pragma unroll
          for (int b = 0; b < NB; ++b) svs[(lane & 16) * NB + four_v_scale(b, lane, NB)] = 0;
        fence_proxy_async_smem();  // before the next copy into this stage
        __syncwarp();
      }
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
        // Keys mt * 16 + g8 and + 8: this lane's words of every block, and the blocks' scales (2^-112 s in fp32: their bits).
        uint32_t kw[2][NB], ksw[2];
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {
          const int row = mt * 16 + k8 * 8 + g8;
          if (NB == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(sk + row * RowB + t4 * 16);
            kw[k8][0] = y.x;
            kw[k8][1] = y.y;
            kw[k8][NB - 2] = y.z;
            kw[k8][NB - 1] = y.w;
            ksw[k8] = *reinterpret_cast<const uint32_t*>(sks + row * 4);
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(sk + row * RowB + t4 * 8);
            kw[k8][0] = y.x;
            kw[k8][1] = y.y;
            ksw[k8] = *reinterpret_cast<const uint16_t*>(sks + row * 2);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t x0 = kw[0][b], x1 = kw[1][b], y0 = __funnelshift_r(x0, x0, 8), y1 = __funnelshift_r(x1, x1, 8);
          const uint32_t k0[4] = {over_one(x0, 0x03C003C0u), over_one(x1, 0x03C003C0u), over_one(x0, 0x003C003Cu),
                                  over_one(x1, 0x003C003Cu)};
          const uint32_t k1[4] = {over_one(y0, 0x03C003C0u), over_one(y1, 0x03C003C0u), over_one(y0, 0x003C003Cu),
                                  over_one(y1, 0x003C003Cu)};
          const float s0 = __uint_as_float((b < 3 ? ksw[0] << (20 - 8 * b) : ksw[0] >> 4) & 0x0FF00000u);
          const float s1 = __uint_as_float((b < 3 ? ksw[1] << (20 - 8 * b) : ksw[1] >> 4) & 0x0FF00000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float c[4] = {start[b][nt][0], start[b][nt][1], start[b][nt][0], start[b][nt][1]};
            mma_f16(c, k0, qf[b][nt][0], qf[b][nt][1]);
            mma_f16(c, k1, qf[b][nt][2], qf[b][nt][3]);
            s[mt][nt][0] = fmaf(c[0], s0, s[mt][nt][0]);
            s[mt][nt][1] = fmaf(c[1], s0, s[mt][nt][1]);
            s[mt][nt][2] = fmaf(c[2], s1, s[mt][nt][2]);
            s[mt][nt][3] = fmaf(c[3], s1, s[mt][nt][3]);
          }
        }
      }
      // Scores of keys mt * 16 + g8 (+ 8) and rows 2 t4 (+ 1), in log2 units.
      const uint8_t* sg = gates + stage * x.gstage;
      const float2* bs = reinterpret_cast<const float2*>(sg + base_off);
      const bool edge = j0 + kKeyTile > (pre ? P : cur.s.own - cur.s.n);  // some slot is no key of some row
      // the largest scale: a lane's four (two) tokens and blocks
      uint32_t wide = NB == 4 ? *reinterpret_cast<const uint32_t*>(svs + lane * 4)
                              : *reinterpret_cast<const uint16_t*>(svs + lane * 2);
      const uint32_t cap = static_cast<uint32_t>(top_e << 3 | 7) * 0x01010101u;
      bool grow = __vmaxu4(wide, cap) != cap;
      const float lim = static_cast<float>(min(kLift, 25 - top_e) + kRoom);
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nt][e] = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const int sub = S == 16 ? mt : 0;
            const float2 base = bs[sub * heads + gidx[nt][e]];
            const float beta = (ci[nt][e].hi - base.x) + (ci[nt][e].lo - base.y);
            const float* gr = reinterpret_cast<const float*>(sg + sub * x.gsub) + gidx[nt][e] * gpitch + 4 -
                              p.bias_from_j + (S == 16 ? 0 : mt * 16);
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8) {
              const int key = g8 + k8 * 8;
              float y = fmaf(beta - gr[key], kLog2e, s[mt][nt][k8 * 2 + e] * 0x1p112f * unit[nt][e]);
              if (edge && j0 + mt * 16 + key > (pre ? P - 1 : pos[nt][e])) y = -INFINITY;
              s[mt][nt][k8 * 2 + e] = y;
              top[nt][e] = fmaxf(top[nt][e], y);
            }
          }
          grow |= top[nt][e] > r[nt][e] + lim;
        }
      if (__any_sync(0xffffffffu, grow)) {
        const float was = static_cast<float>(min(kLift, 25 - top_e));
        uint32_t most = max(max(wide & 255u, wide >> 8 & 255u), max(wide >> 16 & 255u, wide >> 24));
        most = __reduce_max_sync(0xffffffffu, most);
        top_e = max(top_e, static_cast<int>(most >> 3));
        const float lift = static_cast<float>(min(kLift, 25 - top_e));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = top[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            const float rn = fmaxf(r[nt][e] + was, y) - lift;
            const float alpha = rn == -INFINITY ? 1.f : ex2_approx(r[nt][e] - rn);
            r[nt][e] = rn;
            l[nt][e] *= alpha;
#pragma unroll
            for (int dt = 0; dt < 2 * NB; ++dt) {
              acc[dt][nt][e] *= alpha;
              acc[dt][nt][e + 2] *= alpha;
            }
          }
      }
      if (!kMany || j0 < end) {  // not where no row sees a key of the tile
        uint32_t ph[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float o0 = r[nt][0] == -INFINITY ? 0.f : r[nt][0], o1 = r[nt][1] == -INFINITY ? 0.f : r[nt][1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8) {
              const float p0 = ex2_approx(s[mt][nt][k8 * 2] - o0), p1 = ex2_approx(s[mt][nt][k8 * 2 + 1] - o1);
              l[nt][0] += p0;
              l[nt][1] += p1;
              ph[mt][nt][k8] = turn8x8(pack_f16x2(p0, p1));
            }
        }
        uint32_t vsw[2][NB];  // scales of tokens 2 t4, 2 t4 + 1 (+ 8) of each 16
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
          if (NB == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(svs + mt * 64 + t4 * 16);
            vsw[mt][0] = y.x;
            vsw[mt][1] = y.y;
            vsw[mt][NB - 2] = y.z;
            vsw[mt][NB - 1] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(svs + mt * 32 + t4 * 8);
            vsw[mt][0] = y.x;
            vsw[mt][1] = y.y;
          }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t v[4];
          ldsm4_t(smem_u32(sv) + vplace + ((b ^ vturn) << 4), v);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint32_t x0 = v[2 * mt], x1 = v[2 * mt + 1], y0 = x0 >> 8, y1 = x1 >> 8;
            const uint32_t v0[4] = {low_nibbles(x0), high_nibbles(x0), low_nibbles(x1), high_nibbles(x1)};
            const uint32_t v1[4] = {low_nibbles(y0), high_nibbles(y0), low_nibbles(y1), high_nibbles(y1)};
            const uint32_t sa = (vsw[mt][b] & 0x00FF00FFu) << 7, sb = (vsw[mt][b] >> 1) & 0x7F807F80u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t pa = hmul2(ph[mt][nt][0], sa), pb = hmul2(ph[mt][nt][1], sb);
              mma_f16(acc[2 * b][nt], v0, pa, pb);
              mma_f16(acc[2 * b + 1][nt], v1, pa, pb);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage

      if (cur.tile + 1 == cur.tiles || n + 1 == count) {
        // Results, eight rows at a time through the stage just read; or, for the block to join with its neighbours', kept at the
        // ring's start (all copies were read).
        const bool alone = cur.i0 >= u0 && cur.i0 + cur.tiles <= u0 + count, keep = !alone && n + 1 == count;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float* out = keep ? reinterpret_cast<float*>(ring) + nt * 8 * L::kOutStride : reinterpret_cast<float*>(st);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = l[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            const int rl = 2 * t4 + e;
#pragma unroll
            for (int b = 0; b < NB; ++b)
              *reinterpret_cast<float4*>(out + rl * L::kOutStride + b * 32 + g8 * 4) =
                  make_float4(acc[2 * b][nt][e], acc[2 * b][nt][e + 2], acc[2 * b + 1][nt][e], acc[2 * b + 1][nt][e + 2]);
            if (g8 == 0) {
              kept.m[warp][nt * 8 + rl] = r[nt][e];
              kept.l[warp][nt * 8 + rl] = y;
            }
          }
          __syncwarp();
          if (!keep) {
            leave_rows<__nv_bfloat16, D>(p, cur, w, alone && !shared, out - nt * 8 * L::kOutStride, L::kOutStride, kept.m[warp],
                                         kept.l[warp], nt * 8, nt * 8 + 8);
            __syncwarp();
          }
        }
        if (keep && lane == 0) {
          kept.i0[warp] = cur.i0;
          kept.at[warp] = cur;
        }
        fence_proxy_async_smem();  // before the next copy into this stage
        __syncwarp();
        opened = false;
      }
      if (++cur.tile == cur.tiles && n + 1 < count) next_item(p, seqs, cur);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    }

    if (fresh) {
      // Table entries of the rows of the item after the next.
      __syncwarp();
#pragma unroll 1
      while (asked < filled + 2 && ahead < count) {
        Place at_item = cur;
        if (asked > 0) {
          at_item = it.at[(asked - 1) & 1];
          next_item(p, seqs, at_item);
        }
        const int slot = asked & 1;
        ahead += at_item.tiles - at_item.tile;
        ++asked;
        if (lane == 0) it.at[slot] = at_item;
        const int rr = at_item.rt * p.Rt + lane, t = token_of(p, rr), g = rr - t * Gp;
        if (lane < L::kRows && t < at_item.s.n && g < G) {
          const int j = at_item.s.own - at_item.s.n + t;
          cp_async4(smem_u32(&it.page[slot][lane]), a.table + (size_t)at_item.b * a.table_stride + (j >> a.page_shift));
        }
        __syncwarp();
      }
    }
    if (n + stages < count) {
      // A window of the producer's next tiles, whose pages are read long before they are needed.
      if (at == now.n) {
        at = 0;
#pragma unroll 1
        do {
          now = next;
          buf ^= 1;
          if (n < 0) cp_async_commit();
          cp_async_wait<0>();  // now's ids; they were asked for a window ago
          __syncwarp();
          next.n = 0;
          if (left > 0) {
            next.hkv = pro.hkv;
            next.rt = pro.rt;
            next.tile = pro.tile;
            next.n = min(min(32, pro.tiles - pro.tile), left);
            next.own = pro.s.own;
            if (lane < next.n) {
              const int t = pro.tile + lane, j = (t < tp ? t : t - tp) * kKeyTile;
              const int* row = t < tp ? a.prefix : a.table + (size_t)pro.b * a.table_stride;
              cp_async4(smem_u32(&ids[warp][buf ^ 1][lane]), row + (j >> a.page_shift));
              if (S == 16 && j + 16 < (t < tp ? P : pro.s.own))
                cp_async4(smem_u32(&ids[warp][buf ^ 1][32 + lane]), row + (j >> 4) + 1);
            }
            left -= next.n;
            pro.tile += next.n;
            if (pro.tile == pro.tiles && left > 0) next_item(p, seqs, pro);
          }
        } while (now.n == 0);
      }
    }
    if (fresh) {
      // Q and gates of the rows of the next item, at the start of the first.
      fresh = false;
      if (n < 0) cp_async_commit();
      cp_async_wait<0>();  // the entries, asked for in an earlier step (but the first item's)
      __syncwarp();
      if (filled < asked) {
        const int slot = filled & 1;
        const Place at_item = it.at[slot];
        const int r0 = at_item.rt * p.Rt;
        {
          const int rr = r0 + lane, t = token_of(p, rr), g = rr - t * Gp, h = at_item.hkv * G + g;
          if (lane < L::kRows && t < at_item.s.n && g < G) {
            const int page = checked_page(a, it.page[slot][lane]);
            cp_async8(smem_u32(&it.base[lane]), a.gbase + gbase_offset(a, page, h));
            cp_async4(smem_u32(&it.g[lane]), a.g + g_offset(a, page, h, (at_item.s.own - at_item.s.n + t) & (S - 1)));
          }
        }
#pragma unroll 1
        for (int e = lane; e < L::kRows * (D / 8); e += 32) {
          const int rl = e / (D / 8), chunk = e % (D / 8), rr = r0 + rl, t = token_of(p, rr), g = rr - t * Gp;
          const bool in = t < at_item.s.n && g < G;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                                     (size_t)(at_item.s.row0 + (in ? t : 0)) * p.q_stride +
                                     (size_t)(at_item.hkv * G + (in ? g : 0)) * D + chunk * 8;
          cp_async16_or_0(smem_u32(q_of + rl * (D * 2) + ((chunk ^ (rl & 7)) << 4)), src, in);
        }
        ++filled;
      }
    }
    if (n + stages < count) {
      // Copies of the producer's next tile; the stage is the one just read, and in the first steps the n-th.
      const int to = n < 0 ? n + stages : (stage == 0 ? stages : stage) - 1;
      uint8_t* dst = ring + to * L::kStageBytes;
      uint8_t* sg = gates + to * x.gstage;
      const int h0 = now.hkv * G + (G > L::kRows ? now.rt * p.Rt % Gp : 0);
      const int t = now.tile + at, j = (t < tp ? t : t - tp) * kKeyTile, slot = j & (S - 1);
      const int subs = S == 16 && j + 16 < (t < tp ? P : now.own) ? 2 : 1;  // pages of 16: the second may be none
      if (lane == 0)
        mbar_arrive_expect_tx(&bars[warp][to], subs * (2 * KS * (RowB + NB) + heads * gpitch * 4));
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < subs; ++i) {
        const int id = checked_page(a, ids[warp][buf][32 * i + at]);
        // One lane a copy: codes and scales of K and V, whose tokens lie side by side in a page, and the gates.
        if (lane < 4) {
          const bool is_v = lane & 1, scales = lane & 2;
          const int row = scales ? NB : RowB;
          const uint8_t* src = scales ? (is_v ? p.vs : p.ks) : static_cast<const uint8_t*>(is_v ? a.v : a.k);
          bulk_load_by(policy, dst + (scales ? 2 * L::kTileBytes + (is_v ? L::kScaleBytes : 0) : is_v ? L::kTileBytes : 0) + i * 16 * row,
                       src + (((size_t)id * a.Hkv + now.hkv) * S + slot) * row, KS * row, &bars[warp][to]);
        } else if (lane == 31) {
          tma_load_3d(sg + i * x.gsub, &tmap_g, &bars[warp][to], slot - 4, h0, id);
        }
        if (lane < heads && h0 + lane < a.H)
          cp_async8(smem_u32(sg + base_off) + (i * heads + lane) * 8, a.gbase + gbase_offset(a, id, h0 + lane));
      }
      ++at;
    }
    cp_async_commit();
  }
  if (!ok) {
    // A wait gave up: every copy issued must still land before shared memory is used or released.
    for (int s = 0; s < stages; ++s) mbar_wait_drain(&bars[warp][s], s < stage ? phase ^ 1 : phase);
    cp_async_wait_all();
  }
  clear_idle_rows<__nv_bfloat16, D>(p, seqs);
  // The threads' sums stand in the queries' place.
  static_assert(32 * sizeof(Column) <= L::kQBytes, "they fit there");
  join_items<__nv_bfloat16, D, L::kRows, W>(p, seqs, total, each, kept, ends, reinterpret_cast<const float*>(sm),
                                            stages * L::kStageBytes / 4, L::kOutStride, offs, reinterpret_cast<Column*>(all_gates + W * stages * x.gstage));
  if (shared) grid_dep_wait();  // as fox_decode_mma.cu's kernel
}

template <int D, int NT, bool kMany>
cudaError_t launch_as(const DecodeParams& p, const CUtensorMap& gates, cudaStream_t s) {
  using L = Layout4<D, NT>;
  auto kernel = decode4_kernel<D, NT, kMany>;
  const MmaShape x = mma_shape(p.a, L::kRows);
  constexpr size_t kMost = 232448 - 16384;  // of an SM's shared memory, less the static part
  const size_t smem = 1024 + sizeof(SeqEntry) * ((size_t)p.a.B + 1) +
                      (size_t)L::kWarps * (L::kQBytes + L::kStages * (L::kStageBytes + x.gstage));
  // One limit for every call (launch_as in fox_decode_mma.cu has the reason).
  constexpr size_t kLimit = 1024 + sizeof(SeqEntry) * (kMaxSeqs + 1) +
                            L::kWarps * (L::kQBytes + L::kStages * (L::kStageBytes + most_gates(L::kRows)));
  static_assert(kLimit <= kMost, "shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLimit));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode4", s);
  const cudaError_t f = launch_dependent(kernel, dim3(kSMs), dim3(32 * L::kWarps), smem, s, gates, p, x);
  return f != cudaSuccess ? f : cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch(const DecodeParams& p, const CUtensorMap& gates, cudaStream_t s) {
  return p.a.max_new > 1 ? launch_as<D, NT, true>(p, gates, s) : launch_as<D, NT, false>(p, gates, s);
}

}  // namespace

int decode4_rows(int rows) { return rows <= 8 ? 8 : 16; }
int decode4_warps(int, int Rt) { return Rt == 8 ? Layout4<128, 1>::kWarps : Layout4<128, 2>::kWarps; }

cudaError_t launch_decode4(const DecodeParams& p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  const int KS = a.page_size < kKeyTile ? a.page_size : kKeyTile, G = a.H / a.Hkv;
  CUtensorMap gates;
  if (!make_f32_3d_map(&gates, a.g, a.page_size, a.H, a.num_pages, (uint64_t)a.page_size * 4, (uint64_t)a.page_size * a.H * 4,
                       KS + 4, G < p.Rt ? G : p.Rt))
    return cudaErrorInvalidValue;
  if (a.d == 64) return p.Rt == 8 ? launch<64, 1>(p, gates, s) : launch<64, 2>(p, gates, s);
  return p.Rt == 8 ? launch<128, 1>(p, gates, s) : launch<128, 2>(p, gates, s);
}

}  // namespace fox
