// Attention of the newest tokens over the 4-bit paged cache, on the tensor cores.
//
// The plan is fox_decode_mma.cu's: one warp a worker of the work line (fox_paged.h) with a ring of key tiles of its own, transposed
// products S^T = K Q^T and O^T += V^T P^T by the register MMAs (16 x 8 x 16), so that the few query rows are the 8-wide side. Bytes
// are a quarter; what a key costs in instructions is more, so the codes' layout (fox_four.h) is made for this kernel:
//
// K. A lane's part of an MMA operand (a token's channels 8 t .. 8 t + 7 of every block) lies side by side. A nibble u + 8 = n at bits 9..6
//   of an fp16 whose other bits are 0 is n 2^-18, at bits 5..2 it is n 2^-22, both exactly: two masks on the word and two on the word rotated
//   by 8 make the eight values of two MMA steps. With 2^8 q and 2^12 q in their places the products sum to 2^-10 sum q u plus sums of q alone
//   (one a block and row), whose products with the scales one more MMA takes off: scales as they are, the sums in three fp16. So a block costs 5
//   instructions a word and no subtraction of its own. An MMA aligns its terms by their operands' exponents, here as 256 |q|, cuts each
//   at 2^-25 of the largest, and the sum to fp32 (measured); with 1 + n / 16 and 1 + n / 256 for values, whose sums stand 264 sum |q| high,
//   LSE came out four to six times further off at the same time. The block's scale multiplies its sum.
// V. ldmatrix.trans turns 16-bit units (four channels of a token) so that a register has the same four channels of two
//   neighbouring tokens: what the V^T operand wants, nibble by nibble. The masks give 1 + n / 1024 and 1 + n / 64, an fma n - 8, exactly.
//   The scales, which vary along the sum, go to P, once a block of 32 channels: P s f in fp16, with f the power of two that brings the largest
//   scale met so far in the block's channels to [1, 2), so that neither small nor large values leave fp16's range. P is rounded to fp16,
//   and the product again, by 2^-11 of itself at most each while the product is 2^-14 or more; f is taken off when the sums leave. A lane
//   spreads s f out for the warp, a word of four, over the stage's scales (by every lane for itself, 8 more instructions a tile: 176 us below).
// Weights are P = 2^(x - r), with r = the running maximum less kLift: as fp16 holds 2^-24 and above, in full from 2^-14 on, weights down to
//   2^-25 of the largest keep all bits, and so do their products with scales of the largest's size (of 2^-k of it, from 2^(k - 25) on);
//   r moves when a weight passes 2^(kLift + kRoom), f when a scale passes its bound, which one vote finds: the weights are then formed again.
// q in fp16: each row times a power of two so that its largest |q| is in [4, 8); what a bf16 holds is then exact down to 2^-27 of that,
//   and off by 2^-35 of it at most.
// Up to four rows a tile (kRows 4) stand twice among the eight columns, so that scores and weights of half the keys fall to each half of the
//   lanes: columns 0..3 then sum the first 16 keys of a tile, columns 4..7 the others, and are added at the end.
//
// Bound by instructions: 798 a key tile of 128 channels and 4 rows, some 180 of them to spread K out, 200 V, 95 the copies (all lanes' own: by
// bulk copies of a loading warp, which has a lane a worker, 301 us against 235 then). 64 sequences of up to 16384 tokens, 32 heads on 8, 725 MB:
// 171 us, 4.2 TB/s, issue slots 58 % used and the ALU's pipe 52 %; the copies alone took 130, the rest without them 135 when both took 169 (15 of
// either are launch, look-ups and join). V as subnormals, their offset of 8 taken off by two more products: 4 % fewer instructions, 177 for 172 us. One sequence of 65536, 80 MB: 34 us, of which launch and first
// look-ups are 13 and the join of the workers' parts 6; one of 1000, 16 heads of 64 channels: 14.5, all but 3 of them launch, look-ups and join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fox_decode_ring.h"
#include "fox_four.h"

namespace fox {
namespace {

// A weight of the running maximum is 2^kLift at least, and 2^(kLift + kRoom) before the reference moves: 2^15 times 1.875, the largest scale
// times f, is below fp16's end.
constexpr int kLift = 11, kRoom = 4;
constexpr uint32_t kWeightRoom = (0x7FFFu - (kLift + kRoom + 15 << 10)) * 0x00010001u;  // added to a weight above 2^(kLift + kRoom): a sign bit
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

template <int D, int kRows_>  // rows of a row tile: 4, 8 or 16
struct Layout4 {
  static constexpr int kStages = 2;
  static constexpr int kRows = kRows_;
  static constexpr int kBlocks = D / kFourBlock;
  static constexpr int kTileBytes = kKeyTile * D / 2;          // codes of K or V of a stage
  static constexpr int kScaleBytes = kKeyTile * kBlocks;       // scales of K or V of a stage
  static constexpr int kStageBytes = 2 * (kTileBytes + kScaleBytes);
  static constexpr int kGateSub = kRows * 20 * 4;                // gates of 16 slots: [heads][4 before, 16] sums
  static constexpr int kGateBytes = 2 * (kGateSub + kRows * 8);  // of a stage: of two halves, and the halves' [heads] bases
  static constexpr int kQPitch = D * 2 + 16;                     // bytes from one query row to the next
  static constexpr int kQBytes = kRows * kQPitch;
  static constexpr int kOutStride = D + 4;
  static_assert((kRows < 8 ? kRows : 8) * kOutStride * 4 <= kStageBytes, "eight rows pass through a stage that was read");
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
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t majority(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xe8;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
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

// The rows of an item that a warp will need next, besides their Q.
template <int kRows>
struct RowGates {
  float2 base[kRows];
  float g[kRows];
};

// 16 bytes on their way to shared memory, or zeros where there are none to copy (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy16_or_0(uint32_t dst, const void* src, bool copy, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0), "l"(policy)
               : "memory");
}

// What a warp has on its way: the copies of its worker's key tiles, in the order of the line, `kStages` ahead of their use. Pages are
// looked up for up to 32 tiles of an item at a time, a lane a tile, one such window ahead.
template <int D, int kRows>
struct Loader {
  using L = Layout4<D, kRows>;
  static constexpr int NB = L::kBlocks, RowB = D / 2;
  Place pro;                 // behind the last window's last tile
  Window now, next;
  int at, left;              // the next tile of `now`; units that no window holds yet
  uint32_t gates_to;         // this lane's place in a stage's gates
  int h0, most;              // first head of `now`'s rows, and how many
  int id0, id1, nid0, nid1;  // this lane's tile of `now` and `next`: its page, and with pages of 16 tokens the second one

  __device__ __forceinline__ void look_ahead(const DecodeParams& p, const SeqEntry* seqs, int tp) {
    const PagedArgs& a = p.a;
    next.n = 0;
    if (left == 0) return;
    next.hkv = pro.hkv;
    next.rt = pro.rt;
    next.tile = pro.tile;
    next.n = min(min(32, pro.tiles - pro.tile), left);
    next.own = pro.s.own;
    const int lane = threadIdx.x & 31;
    if (lane < next.n) {
      const int t = pro.tile + lane, j = (t < tp ? t : t - tp) * kKeyTile;
      const int* row = t < tp ? a.prefix : a.table + (size_t)pro.b * a.table_stride;
      nid0 = row[j >> a.page_shift];
      nid1 = a.page_shift == 4 && j + 16 < (t < tp ? a.prefix_len : pro.s.own) ? row[(j >> 4) + 1] : 0;
    }
    left -= next.n;
    pro.tile += next.n;
    if (pro.tile == pro.tiles && left > 0) next_item(p, seqs, pro);
  }
  __device__ __forceinline__ void begin(const DecodeParams& p, const SeqEntry* seqs, int tp, const Place& first, int count) {
    const int lane = threadIdx.x & 31;
    gates_to = (lane >> 2 & 1) * L::kGateSub + (4 + (lane & 3) * 4) * 4 + (lane >> 3) * 80;
    pro = first;
    left = count;
    at = now.n = 0;
    id0 = id1 = nid0 = nid1 = 0;
    next.n = 0;
    if (count > 0) look_ahead(p, seqs, tp);
  }
  // Asks for the next tile of the line; there is one. `dst`, `sg`: where its codes and scales, and its gates, go in shared memory.
  __device__ __forceinline__ void ask(const DecodeParams& p, int G, const SeqEntry* seqs, int tp, uint32_t dst, uint32_t sg,
                                      uint64_t policy) {
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, S = 1 << a.page_shift;
    if (at == now.n) {
      at = 0;
      now = next;
      id0 = lane < now.n ? checked_page(a, nid0) : 0;
      id1 = lane < now.n ? checked_page(a, nid1) : 0;
      look_ahead(p, seqs, tp);
      h0 = now.hkv * G + (G > kRows ? now.rt * p.Rt % p.Gp : 0);
      most = min(min(G, kRows), a.H - h0);
    }
    const int t = now.tile + at, j = (t < tp ? t : t - tp) * kKeyTile, slot = j & (S - 1);
    const int page0 = __shfl_sync(0xffffffffu, id0, at);
    // Tokens of a head counted through the pool: 32 bits hold them (check_four). Those of a page lie side by side, in halves of
    // 16 that are two pages' with pages of 16: NB lanes a half of K's or V's scales, four lanes a half of a head's gates.
    const uint32_t token0 = (static_cast<uint32_t>(page0) * a.Hkv + now.hkv << a.page_shift) + slot;
    const uint32_t row0 = static_cast<uint32_t>(page0) * a.H + h0;
    const uint32_t l16 = lane * 16, mine = dst + l16;
    const uint8_t* scales = (lane < 2 * NB ? p.ks : p.vs - 32 * NB) + l16;
    const int h4 = lane >> 3;
    if (S != 16) {
      const uint64_t codes = (uint64_t)token0 * RowB + l16;
      const uint8_t* k = static_cast<const uint8_t*>(a.k) + codes;
      const uint8_t* v = static_cast<const uint8_t*>(a.v) + codes;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) copy16(mine + i * 512, k + i * 512, policy);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) copy16(mine + L::kTileBytes + i * 512, v + i * 512, policy);
      if (lane < 4 * NB) copy16(mine + 2 * L::kTileBytes, scales + (uint64_t)token0 * NB, policy);
      const float* g = a.g + ((size_t)(row0 + h4) * S + (slot + (lane & 7) * 4));
      const uint32_t to = sg + gates_to;
#pragma unroll
      for (int h = 0; h < kRows; h += 4)
        if (h + h4 < most) copy16(to + h * 80, g + (size_t)h * S, policy);
      if (lane < 2 * kRows && lane % kRows < most) {
        const size_t row = row0 + lane % kRows;
        cp_async8(sg + 2 * L::kGateSub + lane * 8, a.gbase + 2 * row);
        if (p.bias_from_j) {  // the four slots before, 0 before a page's first
          const int before = slot + lane / kRows * 16 - 4;
          copy16_or_0(sg + lane / kRows * L::kGateSub + lane % kRows * 80, a.g + ((row << a.page_shift) + max(before, 0)), before >= 0, policy);
        }
      }
    } else {
      const bool two = j + 16 < (t < tp ? a.prefix_len : now.own);  // the second half's page may be none
      const int page1 = __shfl_sync(0xffffffffu, id1, at);
      const uint32_t row1 = static_cast<uint32_t>(page1) * a.H + h0;
      const uint32_t token1 = (static_cast<uint32_t>(page1) * a.Hkv + now.hkv) * 16;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* pool = static_cast<const uint8_t*>(x ? a.v : a.k) + lane * 16;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          copy16(mine + x * L::kTileBytes + i * 512, pool + (uint64_t)token0 * RowB + i * 512, policy);
          copy16_or_0(mine + x * L::kTileBytes + (D / 64 + i) * 512, pool + (uint64_t)token1 * RowB + i * 512, two, policy);
        }
      }
      if (lane < 4 * NB) {
        const bool second = lane / NB & 1;
        copy16_or_0(mine + 2 * L::kTileBytes, scales - (second ? 16 * NB : 0) + (uint64_t)(second ? token1 : token0) * NB, !second || two,
                    policy);
      }
      const bool other = lane >> 2 & 1;
      const uint32_t to = sg + gates_to;
      for (int h = h4; h < most; h += 4)
        copy16_or_0(to + (h - h4) * 80, a.g + ((size_t)((other ? row1 : row0) + h) * 16 + (lane & 3) * 4), !other || two, policy);
      if (lane < 2 * kRows && lane % kRows < most) {
        cp_async8(sg + 2 * L::kGateSub + lane * 8, a.gbase + 2 * (size_t)((lane < kRows ? row0 : row1) + lane % kRows));
        if (p.bias_from_j) copy16_or_0(sg + lane / kRows * L::kGateSub + lane % kRows * 80, a.g, false, policy);
      }
    }
    ++at;
  }
};

// kMany: sequences may bring more than one token, so that rows of a tile may end at different keys.
template <int D, int kRows, int W, bool kMany>
__global__ void __launch_bounds__(32 * W, 1) decode4_kernel(const __grid_constant__ DecodeParams p, const int G) {
  using L = Layout4<D, kRows>;
  constexpr int NB = L::kBlocks, RowB = D / 2, stages = L::kStages, NT = kRows == 16 ? 2 : 1;
  constexpr bool kTwice = kRows == 4;        // rows stand twice among the columns
  constexpr int MT = kTwice ? 1 : 2;         // of a tile's two halves of 16 keys, how many a lane forms weights of
  extern __shared__ uint8_t smem_raw[];
  __shared__ int scratch[W];
  __shared__ Kept<L::kRows, W> kept;
  __shared__ BlockEnds ends;
  __shared__ RowGates<L::kRows> row_gates[W];
  __shared__ Place places[W][2];
  __shared__ int offs[kSMs + 1];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* all_gates = sm + W * stages * L::kStageBytes;
  uint8_t* all_q = all_gates + W * stages * L::kGateBytes;
  uint8_t* ring = sm + warp * stages * L::kStageBytes;
  uint8_t* gates = all_gates + warp * stages * L::kGateBytes;
  uint8_t* q_of = all_q + warp * L::kQBytes;
  RowGates<L::kRows>* rows = &row_gates[warp];
  SeqEntry* seqs = reinterpret_cast<SeqEntry*>(all_q + W * L::kQBytes);

  const bool shared = p.pre.key_tiles > 0;
  if (lane == 0) kept.i0[warp] = -1;
  // Behind a shared prefix's kernels the wait comes last (fox_decode_mma.cu).
  if (!shared) grid_dep_wait();
  grid_dep_trigger();
  scan_sequences(p, seqs, scratch);  // ends with a block barrier
  if (shared && blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += blockDim.x) p.cum[b] = seqs[b].u0;

  const int total = seqs[a.B].u0 * a.Hkv, each = units_per_worker(total, p.workers);
  const int w = blockIdx.x * W + warp;
  const int u0 = min(total, w * each), count = min(total, u0 + each) - u0;
  const int Gp = p.Gp, S = a.page_size;
  const int P = a.prefix_len, tp = p.walk_prefix ? ceil_div(P, kKeyTile) : 0;  // the prefix's tiles come first
  const int g8 = lane >> 2, t4 = lane & 3;
  const int half = kTwice ? t4 >> 1 : 0;  // where rows stand twice, the half of a tile's keys that this lane weighs
  const uint32_t vplace = lane * RowB, vturn = NB == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1;
  const uint64_t policy = stream_policy();

  // An item's rows come in three steps, each while an item before it is computed: its place and this lane's row's page (places[k & 1],
  // row_page) two items ahead, Q and the gates at the rows' places one item ahead.
  int units_placed = 0, placed = 0, row_page = 0;
  auto place_item = [&]() {
    if (units_placed >= count) return;
    Place y;
    if (placed == 0) {
      y = place_of(p, seqs, u0);
    } else {
      y = places[warp][(placed - 1) & 1];
      next_item(p, seqs, y);
    }
    __syncwarp();
    if (lane == 0) places[warp][placed & 1] = y;
    __syncwarp();
    units_placed += y.tiles - y.tile;
    ++placed;
    const int rr = y.rt * p.Rt + lane, t = token_of(p, rr), g = rr - t * Gp;
    if (lane < L::kRows && t < y.s.n && g < G)
      row_page = a.table[(size_t)y.b * a.table_stride + ((y.s.own - y.s.n + t) >> a.page_shift)];
  };
  auto ask_rows = [&](int k) {  // of item k, the last one placed
    const Place& y = places[warp][k & 1];
    const int r0 = y.rt * p.Rt, new0 = y.s.own - y.s.n, n = y.s.n, hkv = y.hkv;
    {
      const int rr = r0 + lane, t = token_of(p, rr), g = rr - t * Gp, h = hkv * G + g;
      if (lane < L::kRows && t < n && g < G) {
        const int page = checked_page(a, row_page);
        cp_async8(smem_u32(&rows->base[lane]), a.gbase + gbase_offset(a, page, h));
        cp_async4(smem_u32(&rows->g[lane]), a.g + g_offset(a, page, h, (new0 + t) & (S - 1)));
      }
    }
    const int row_of = y.s.row0;
#pragma unroll 1
    for (int e = lane; e < L::kRows * (D / 8); e += 32) {
      const int rl = e / (D / 8), chunk = e % (D / 8), rr = r0 + rl, t = token_of(p, rr), g = rr - t * Gp;
      const bool in = t < n && g < G;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (size_t)(row_of + (in ? t : 0)) * p.q_stride +
                                 (size_t)(hkv * G + (in ? g : 0)) * D + chunk * 8;
      cp_async16_or_0(smem_u32(q_of + rl * L::kQPitch + chunk * 16), src, in);
    }
  };

  Loader<D, kRows> load;
  int asked = 0;  // tiles
  place_item();
  {
    Place y = {};
    if (count > 0) y = places[warp][0];
    load.begin(p, seqs, tp, y, count);
  }
  if (count > 0) ask_rows(0);
#pragma unroll 1
  for (; asked < stages; ++asked) {
    if (asked < count)
      load.ask(p, G, seqs, tp, smem_u32(ring + asked * L::kStageBytes), smem_u32(gates + asked * L::kGateBytes), policy);
    cp_async_commit();
  }
  place_item();
  if (warp == 0) find_ends<W>(p, seqs, total, each, ends);  // while the first copies are on their way

  int done = 0, stage = 0, segment = 0;  // `segment`: where the latest item began
  Place cur = {};
#pragma unroll 1
  for (int item = 0; done < count; ++item) {
    // A segment: key tiles cur.tile .. tile1 - 1 of an item.
    if (item == 0)
      cur = places[warp][0];
    else
      next_item(p, seqs, cur);
    const int tile0 = cur.tile, tile1 = min(cur.tiles, tile0 + (count - done));
    const int r0 = cur.rt * p.Rt, own = cur.s.own, new0 = own - cur.s.n;
    // with kMany: own position of the item's last row
    const int last = kMany ? new0 + min(token_of(p, r0 + p.Rt - 1), cur.s.n - 1) : own - 1;
    // The rows were asked for with the tile that was asked for after the first one of the item before was read, the first item's
    // with its own first tile.
    if (item == 0 || done - segment > 1)
      cp_async_wait<stages - 1>();
    else
      cp_async_wait<0>();
    segment = done;
    __syncwarp();
    uint32_t qf[NB][NT][4];     // Q^T operand: of block b, its lane's channels 0 1, 2 3, 6 7, 4 5
    uint32_t start[NT][2];      // what the blocks' sums have too much, negated, in three fp16 each: an operand beside the scales
    float unit[NT][2];          // log2 units of a row's S
    float acc[2 * NB][NT][4];   // O^T: of block b channels 4 g8 + 0, + 1 and + 2, + 3
    float r[NT][2], l[NT][2];   // the reference that weights are taken against, their sum
    // Of the block of channels whose scales this lane spreads out, lane % NB: exponent bits of the largest scale of V so far, its bound
    // (`over` below), and f, 2^(15 - exponent bits), twice.
    int top_e = 0;
    uint32_t scale_room = 0, scale_low = 0, f2 = 0;
    Gate2 ci[NT][2];
    int pos[NT][2], head[NT][2];  // a row's own place, its head of the row tile's
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // Row nt * 8 + g8: this lane's channels of every block, in fp16 at a power of two.
      const uint8_t* qr = q_of + (nt * 8 + g8) % kRows * L::kQPitch;
      float f[NB][8], most = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 y = *reinterpret_cast<const uint4*>(qr + (b * 4 + t4) * 16);
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
      // 2^-e brings `most` to [4, 8); in two factors, both of them normal numbers
      const int e = most > 0.f ? min(static_cast<int>(__float_as_uint(most) >> 23), 254) - 127 - 2 : 0;
      const float down0 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23),
                  down1 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
      const float row_unit = p.scale2 / down0 * 0x1p10f / down1;
      uint32_t piece[3][NB / 2];  // the sums of two blocks, in three parts
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // pairs 0 and 3 stand at bits 9..6, pairs 1 and 2 at bits 5..2
          const bool low = i == 1 || i == 2;
          const float up = low ? 4096.f : 256.f;
          const uint32_t h = pack_f16x2(f[b][2 * i] * down0 * down1 * up, f[b][2 * i + 1] * down0 * down1 * up);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
          sum -= (back.x + back.y) * (8.f / 1024.f / up);  // 32 channels of 8 times less than 8, 2^-10: at most 2
          qf[b][nt][i == 0 ? 0 : i == 1 ? 1 : i == 3 ? 2 : 3] = h;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t h = pack_f16x2(sum, 0.f) & 0xFFFFu;
          sum -= __half2float(*reinterpret_cast<const __half*>(&h));
          piece[i][b / 2] = b % 2 ? piece[i][b / 2] | h << 16 : h;
        }
      }
      // The operand's rows 2 t4, 2 t4 + 1 and + 8, + 9 (blocks b, b + 1 of a part), beside which scales() puts the blocks' scales.
      if (NB == 4) {
        start[nt][0] = t4 == 0 ? piece[0][0] : t4 == 1 ? piece[0][NB / 2 - 1] : t4 == 2 ? piece[1][0] : piece[1][NB / 2 - 1];
        start[nt][1] = t4 == 0 ? piece[2][0] : t4 == 1 ? piece[2][NB / 2 - 1] : 0u;
      } else {
        start[nt][0] = t4 == 0 ? piece[0][0] : t4 == 1 ? piece[1][0] : t4 == 2 ? piece[2][0] : 0u;
        start[nt][1] = 0u;
      }
      unit[nt][0] = __shfl_sync(0xffffffffu, row_unit, t4 * 8);
      unit[nt][1] = __shfl_sync(0xffffffffu, row_unit, t4 * 8 + 4);
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const int rl = (nt * 8 + 2 * t4 + e2) % kRows, rr = r0 + rl, t = token_of(p, rr), g = rr - t * Gp;
        const bool here = t < cur.s.n && g < G;
        pos[nt][e2] = new0 + t;
        head[nt][e2] = here ? (G > kRows ? g - r0 % Gp : g) : 0;
        ci[nt][e2] = {-INFINITY, 0.f};  // an empty row's scores are -inf
        if (here) ci[nt][e2] = gate_sum(rows->base[rl], rows->g[rl]);
        r[nt][e2] = 0.f;
        l[nt][e2] = 0.f;
      }
    }
    __syncwarp();
    if (item + 1 < placed) {  // into the places just read, with the next commit
      ask_rows(item + 1);
      place_item();
    }
#pragma unroll
    for (int dt = 0; dt < 2 * NB; ++dt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[dt][nt][e] = 0.f;

#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      cp_async_wait<stages - 1>();
      __syncwarp();
      const bool pre = tile < tp;
      const int j0 = (pre ? tile : tile - tp) * kKeyTile;
      uint8_t* st = ring + stage * L::kStageBytes;
      const uint8_t* sk = st;
      const uint8_t* sv = st + L::kTileBytes;
      uint8_t* sks = st + 2 * L::kTileBytes;
      uint8_t* svs = st + 2 * L::kTileBytes + L::kScaleBytes;
      const uint8_t* sg = gates + stage * L::kGateBytes;
      // The tile's keys are those of the prefix, or of the sequence's own, which end for each row with its own.
      const bool edge = j0 + kKeyTile > (pre ? P : new0);  // some slot is no key of some row
      if (edge && j0 + kKeyTile > (pre ? P : own)) {
        // Slots behind the end may hold anything, NaN scales among them: V's scales there become 0 (K's scores are left out).
        if (lane >= (pre ? P : own) - j0)
#pragma unroll
          for (int b = 0; b < NB; ++b) svs[(lane & 16) * NB + four_v_scale(b, lane, NB)] = 0;
        __syncwarp();
      }
      if (!kMany || pre || j0 <= last) {  // not where no row sees a key of the tile
        float s[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // Keys mt * 16 + g8 and + 8: this lane's words of every block, and the blocks' scales.
          uint32_t kw[2][NB], kh[2];
          float ks[2][NB];
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            const int row = mt * 16 + k8 * 8 + g8;
            uint32_t ksw;
            if (NB == 4) {
              const uint4 y = *reinterpret_cast<const uint4*>(sk + row * RowB + t4 * 16);
              kw[k8][0] = y.x;
              kw[k8][1] = y.y;
              kw[k8][NB - 2] = y.z;
              kw[k8][NB - 1] = y.w;
              ksw = *reinterpret_cast<const uint32_t*>(sks + row * 4);
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(sk + row * RowB + t4 * 8);
              kw[k8][0] = y.x;
              kw[k8][1] = y.y;
              ksw = *reinterpret_cast<const uint16_t*>(sks + row * 2);
            }
#pragma unroll
            for (int b = 0; b < NB; b += 2) {
              // bytes b and b + 1 to bits 14..7 of two halves: fp16
              const uint32_t h = __byte_perm(ksw, 0, b ? 0x3424 : 0x1404) >> 1;
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
              ks[k8][b] = f.x;
              ks[k8][b + 1] = f.y;
              kh[k8] = b && !(t4 & 1) ? kh[k8] : h;  // blocks 0, 1 or, in odd lanes, 2, 3
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
            const uint32_t both[4] = {kh[0], kh[1], kh[0], kh[1]};
            mma_f16(s[mt][nt], both, start[nt][0], start[nt][1]);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t x0 = kw[0][b], x1 = kw[1][b], y0 = __funnelshift_r(x0, x0, 8), y1 = __funnelshift_r(x1, x1, 8);
            const uint32_t k0[4] = {x0 & 0x03C003C0u, x1 & 0x03C003C0u, x0 & 0x003C003Cu, x1 & 0x003C003Cu};
            const uint32_t k1[4] = {y0 & 0x03C003C0u, y1 & 0x03C003C0u, y0 & 0x003C003Cu, y1 & 0x003C003Cu};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(c, k0, qf[b][nt][0], qf[b][nt][1]);
              mma_f16(c, k1, qf[b][nt][2], qf[b][nt][3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][nt][e] = fmaf(c[e], ks[e >> 1][b], s[mt][nt][e]);
            }
          }
        }
        // Scores less the reference, of keys m * 16 + g8 (+ 8) and rows 2 t4 (+ 1), in log2 units; m: mt, or this lane's half.
        float y[MT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* gr = reinterpret_cast<const float*>(sg) + (head[nt][e] * 20 + 4 + g8 - p.bias_from_j) + half * (L::kGateSub / 4);
            const float2* bs = reinterpret_cast<const float2*>(sg + 2 * L::kGateSub) + head[nt][e] + half * kRows;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const float2 base = bs[mt * kRows];
              const float beta = (ci[nt][e].hi - base.x) + (ci[nt][e].lo - base.y);
#pragma unroll
              for (int k8 = 0; k8 < 2; ++k8) {
                const float x = kTwice && half ? s[1][nt][k8 * 2 + e] : s[mt][nt][k8 * 2 + e];
                y[mt][nt][k8 * 2 + e] =
                    fmaf(beta - gr[mt * (L::kGateSub / 4) + k8 * 8], kLog2e, fmaf(x, unit[nt][e], -r[nt][e]));
              }
            }
          }
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                if (j0 + (mt + half) * 16 + (e >> 1) * 8 + g8 > (pre ? P - 1 : pos[nt][e & 1])) y[mt][nt][e] = -INFINITY;
        }
        // Weights, two rows to an fp16 pair.
        uint32_t ph[2][NT][2];
        float wt[MT][NT][4];
        auto weigh = [&]() {
          uint32_t most = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int k8 = 0; k8 < 2; ++k8) {
                wt[mt][nt][k8 * 2] = ex2_approx(y[mt][nt][k8 * 2]);
                wt[mt][nt][k8 * 2 + 1] = ex2_approx(y[mt][nt][k8 * 2 + 1]);
                ph[mt][nt][k8] = pack_f16x2(wt[mt][nt][k8 * 2], wt[mt][nt][k8 * 2 + 1]);
                most = hmax2(most, ph[mt][nt][k8]);
              }
          return most;
        };
        const uint32_t most = weigh();
        // A weight above 2^(kLift + kRoom), or a scale byte above top_e's (a lane's four of the tile's, all of one block): sums of
        // the lower bits that reach a sign bit, for bytes with or without the sign bits. And where nothing was weighed before.
        const uint32_t wide = *reinterpret_cast<const uint32_t*>(svs + lane % (8 * NB) * 4);
        const uint32_t over = ((most + kWeightRoom) & 0x80008000u) | (majority(wide, (wide & 0x7F7F7F7Fu) + scale_room, scale_low) & 0x80808080u);
        if (__any_sync(0xffffffffu, over != 0 || tile == tile0)) {
          uint32_t top_s = max(max(wide & 255u, wide >> 8 & 255u), max(wide >> 16 & 255u, wide >> 24));
#pragma unroll
          for (int k = NB; k < 8 * NB; k <<= 1) top_s = max(top_s, __shfl_xor_sync(0xffffffffu, top_s, k));
          const int was_e = top_e;
          top_e = max(top_e, static_cast<int>(top_s >> 3));
          const uint32_t bound = static_cast<uint32_t>(top_e << 3 | 7);
          scale_room = (0x7Fu - (bound & 0x7Fu)) * 0x01010101u;
          scale_low = bound < 0x80u ? 0xFFFFFFFFu : 0u;
          const float f = power_of_2(15 - top_e), fell = power_of_2(was_e - top_e);
          f2 = pack_f16x2(f, f);
          float down[NB];  // of the sums so far
#pragma unroll
          for (int b = 0; b < NB; ++b) down[b] = __shfl_sync(0xffffffffu, fell, b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // the largest score less the reference; a row that weighed something had one of kLift there
              float z = l[nt][e] > 0.f ? static_cast<float>(kLift) : -INFINITY;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) z = fmaxf(z, fmaxf(y[mt][nt][e], y[mt][nt][e + 2]));
#pragma unroll
              for (int k = kTwice ? 2 : 4; k < 32; k <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, k));
              const float up = z == -INFINITY ? 0.f : z - kLift, alpha = up > 0.f ? ex2_approx(-up) : 1.f;  // below 0 only where nothing is summed yet
              r[nt][e] += up;
              l[nt][e] *= alpha;
#pragma unroll
              for (int dt = 0; dt < 2 * NB; ++dt) {
                acc[dt][nt][e] *= alpha * down[dt / 2];
                acc[dt][nt][e + 2] *= alpha * down[dt / 2];
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                y[mt][nt][e] -= up;
                y[mt][nt][e + 2] -= up;
              }
            }
          weigh();
        }
        // Scales of V times f, in fp16, in the place of the stage's scales, all of which were read: of each word of four those of tokens 2 t, 2 t + 1
        // and of + 8, + 9, as the weights' operands have them.
        *reinterpret_cast<uint2*>(sks + lane % (8 * NB) * 8) =
            make_uint2(hmul2((wide & 0x00FF00FFu) * 128u, f2), hmul2((wide >> 1) & 0x7F807F80u, f2));
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8) {
              l[nt][0] += wt[mt][nt][k8 * 2];
              l[nt][1] += wt[mt][nt][k8 * 2 + 1];
              ph[mt][nt][k8] = turn8x8(ph[mt][nt][k8]);
              if (kTwice) {  // a column has no weights of the other half's keys
                ph[1][nt][k8] = g8 < 4 ? 0u : ph[0][nt][k8];
                ph[0][nt][k8] = g8 < 4 ? ph[0][nt][k8] : 0u;
              }
            }
        // Scales of tokens 2 t4, 2 t4 + 1 (+ 8) of each 16, where rows stand twice of those whose weights this lane's column has.
        uint2 vsw[MT][NB];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int b = 0; b < NB; b += 2) {
            const uint4 x = *reinterpret_cast<const uint4*>(sks + (((kTwice ? g8 >> 2 : mt) * 4 + t4) * NB + b) * 8);
            vsw[mt][b] = make_uint2(x.x, x.y);
            vsw[mt][b + 1] = make_uint2(x.z, x.w);
          }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t v[4];
          ldsm4_t(smem_u32(sv) + vplace + ((b ^ vturn) << 4), v);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint2 sw = vsw[kTwice ? 0 : mt][b];
            const uint32_t x0 = v[2 * mt], x1 = v[2 * mt + 1], y0 = x0 >> 8, y1 = x1 >> 8;
            const uint32_t v0[4] = {low_nibbles(x0), high_nibbles(x0), low_nibbles(x1), high_nibbles(x1)};
            const uint32_t v1[4] = {low_nibbles(y0), high_nibbles(y0), low_nibbles(y1), high_nibbles(y1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t pa = hmul2(ph[mt][nt][0], sw.x), pb = hmul2(ph[mt][nt][1], sw.y);
              mma_f16(acc[2 * b][nt], v0, pa, pb);
              mma_f16(acc[2 * b + 1][nt], v1, pa, pb);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (tile + 1 == tile1) {
        done += tile1 - tile0;
        // Results, eight rows at a time through the stage just read; or, for the block to join with its neighbours', kept at the
        // ring's start (all copies were read).
        const bool alone = cur.i0 >= u0 && cur.i0 + cur.tiles <= u0 + count, keep = !alone && done == count;
        cur.tile = tile1;
        float up[NB];  // takes f off
#pragma unroll
        for (int b = 0; b < NB; ++b) up[b] = power_of_2(__shfl_sync(0xffffffffu, top_e, b) - 15);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float* out = reinterpret_cast<float*>(keep ? ring : st) + (keep ? nt * 8 * L::kOutStride : 0);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = l[nt][e];
#pragma unroll
            for (int k = kTwice ? 2 : 4; k < 32; k <<= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
            const int rl = 2 * t4 + e;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              float4 x = make_float4(acc[2 * b][nt][e] * up[b], acc[2 * b][nt][e + 2] * up[b], acc[2 * b + 1][nt][e] * up[b],
                                     acc[2 * b + 1][nt][e + 2] * up[b]);
              if (kTwice) {
                x.x += __shfl_xor_sync(0xffffffffu, x.x, 2);
                x.y += __shfl_xor_sync(0xffffffffu, x.y, 2);
                x.z += __shfl_xor_sync(0xffffffffu, x.z, 2);
                x.w += __shfl_xor_sync(0xffffffffu, x.w, 2);
              }
              if (rl < kRows) *reinterpret_cast<float4*>(out + rl * L::kOutStride + b * 32 + g8 * 4) = x;
            }
            if (g8 == 0 && rl < kRows) {
              kept.m[warp][nt * 8 + rl] = y > 0.f ? r[nt][e] : -INFINITY;
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
      }
      if (asked < count) {
        load.ask(p, G, seqs, tp, smem_u32(st), smem_u32(sg), policy);
        ++asked;
      }
      cp_async_commit();
      stage = stage + 1 == stages ? 0 : stage + 1;
    }
  }
  clear_idle_rows<__nv_bfloat16, D>(p, seqs);
  // The threads' sums stand in the gates' place.
  static_assert(32 * sizeof(Column) <= stages * L::kGateBytes, "they fit there");
  join_items<__nv_bfloat16, D, L::kRows, W>(p, seqs, total, each, kept, ends, reinterpret_cast<const float*>(sm),
                                            stages * L::kStageBytes / 4, L::kOutStride, offs, reinterpret_cast<Column*>(all_gates));
  if (shared) grid_dep_wait();  // as fox_decode_mma.cu's kernel
}

// The prefix's K in bf16 and V in fp16, as the prefix kernel multiplies them; V of 65536 and above is reported.
// Blocks of kSpreadUnits units of a page's K, then of its V, and one more a page for its gates and table entry. A unit is 16 channels of one
// token and head, a chunk of each half of the head: stores are contiguous over lanes. Bound by memory: 32768 tokens of 8 heads of 128 channels, 34 MB
// to 134, 30 us, 5.5 TB/s (a chunk a thread, blocks of one head 45).
constexpr int kSpreadThreads = 256, kSpreadUnits = 8 * kSpreadThreads;
inline int spread_blocks(const PagedArgs& a) { return ceil_div(a.Hkv * a.page_size * (a.d / 16), kSpreadUnits); }
__device__ __forceinline__ uint32_t four_largest(const uint4& w) {
  return __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
}
template <int D>
__global__ void __launch_bounds__(kSpreadThreads) spread4_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ PagedArgs to,
                                                                 int blocks) {
  constexpr int kBlocks = D / kFourBlock, kHalf = kBlocks / 2, kUnits = D / 16;
  const PagedArgs& a = p.a;
  const int S = a.page_size, per = 2 * blocks + 1, at = blockIdx.x / per, part = blockIdx.x - at * per, tid = threadIdx.x;
  grid_dep_wait();
  grid_dep_trigger();
  const int page = checked_page(a, a.prefix[at]), live = min(S, a.prefix_len - at * S);
  if (part == 2 * blocks) {
    const size_t n = (size_t)a.H * S / 4;
    const float4* g = reinterpret_cast<const float4*>(a.g) + (size_t)page * n;
    float4* out = reinterpret_cast<float4*>(to.g) + (size_t)at * n;
    for (size_t i = tid; i < n; i += kSpreadThreads) out[i] = g[i];
    for (int h = tid; h < a.H; h += kSpreadThreads)
      reinterpret_cast<float2*>(to.gbase)[(size_t)at * a.H + h] = reinterpret_cast<const float2*>(a.gbase)[(size_t)page * a.H + h];
    if (tid == 0) const_cast<int32_t*>(to.prefix)[at] = at;
    return;
  }
  const bool is_v = part >= blocks;
  const int begin = (is_v ? part - blocks : part) * kSpreadUnits, end = min(begin + kSpreadUnits, a.Hkv * S * kUnits);
  const int j = tid % kUnits, b = j >> 2, t = j & 3;
  uint32_t most = 0;  // magnitudes of V, as bits
  const uint8_t* from = static_cast<const uint8_t*>(is_v ? a.v : a.k) + four_row(a, page, 0, 0);
  const uint8_t* scales = (is_v ? p.vs : p.ks) + four_scale_row(a, page, 0, 0);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_v ? to.v : to.k) + kv_offset(to, at, 0, 0) + j * 8;
#pragma unroll 4
  for (int i = begin + tid; i < end; i += kSpreadThreads) {
    const int row = i / kUnits, slot = row & (S - 1);
    const int word = is_v ? four_v_word(b, t, slot, kBlocks) : four_k_word(b, t, kBlocks);
    const uint8_t* codes = from + (size_t)row * (D / 2);
    const uint8_t* scale = scales + (is_v ? (row & ~15) * kBlocks + four_v_scale(b, slot, kBlocks) : row * kBlocks + b);
    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(codes + word);
    const uint32_t w1 = *reinterpret_cast<const uint32_t*>(codes + (is_v ? word ^ kHalf * 16 : word + kHalf * 4));
    const uint32_t s0 = scale[0], s1 = scale[is_v ? 4 * kHalf : kHalf];
    uint4* to_row = reinterpret_cast<uint4*>(out + (size_t)row * D);
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (slot < live) {
      x0 = is_v ? four_v16(w0, s0) : four_values(w0, s0, false);
      x1 = is_v ? four_v16(w1, s1) : four_values(w1, s1, false);
      if (is_v) most = __vmaxu2(most, __vmaxu2(four_largest(x0), four_largest(x1)));
    }
    to_row[0] = x0;
    to_row[D / 16] = x1;
  }
  if (((most & 0xFFFFu) >= 0x7C00u || most >= 0x7C000000u) && a.err) atomicOr(a.err, DEV_ERR_RANGE);
}

constexpr size_t smem_bytes(int D, int rows, int W, size_t B) {
  const size_t stage = 2 * (kKeyTile * D / 2 + kKeyTile * D / kFourBlock), q = rows * (D * 2 + 16), gates = rows * 176;
  return 128 + sizeof(SeqEntry) * (B + 1) + W * (q + 2 * (stage + gates));
}
constexpr size_t kMost = 232448 - 8192;  // of an SM's shared memory, less the static part

template <int D, int kRows, int W, bool kMany>
cudaError_t launch_as(const DecodeParams& p, cudaStream_t s) {
  using L = Layout4<D, kRows>;
  static_assert(smem_bytes(D, kRows, W, 0) == 128 + sizeof(SeqEntry) + W * (L::kQBytes + L::kStages * (L::kStageBytes + L::kGateBytes)), "");
  auto kernel = decode4_kernel<D, kRows, W, kMany>;
  // One limit for every call (launch_as in fox_decode_mma.cu has the reason).
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode4", s);
  const cudaError_t f = launch_dependent(kernel, dim3(kSMs), dim3(32 * W), smem_bytes(D, kRows, W, p.a.B), s, p, p.a.H / p.a.Hkv);
  return f != cudaSuccess ? f : cudaGetLastError();
}

// Workers of a CTA: three a scheduler, as registers allow, or two where a worker's rings and rows leave no room for three in shared memory.
// 64 sequences of up to 16384 tokens, 4 rows: 12 workers 172 us, 10 199, 14 and 16 (128 registers, some of them spilled) 190 and 178 (64 channels,
// up to 8192: 130, 151, 138 and 126); a third stage of the ring 171 where two took 169. 16 rows of 128 channels, up to 8192: 8 workers 163, 10 279.
constexpr int warps_of(int D, int rows) { return rows < 16 || D == 64 ? 12 : 8; }

template <int D, int kRows>
cudaError_t launch(const DecodeParams& p, cudaStream_t s) {
  constexpr int W = warps_of(D, kRows);
  static_assert(smem_bytes(D, kRows, W, kMaxSeqs) <= kMost, "shared memory");
  return p.a.max_new > 1 ? launch_as<D, kRows, W, true>(p, s) : launch_as<D, kRows, W, false>(p, s);
}

}  // namespace

// The smallest tile that holds them: 4 rows a key head, 64 sequences of up to 16384 tokens, 172 us in tiles of 4 and 179 of 8; 8 rows, up
// to 8192, 105 of 8 and 153 of 16 (64 channels: 4 rows 130 and 137, 8 rows 140 and 190).
int decode4_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
int decode4_warps(const PagedArgs& a, int Rt) { return warps_of(a.d, Rt); }

cudaError_t launch_spread4(const DecodeParams& p, const PagedArgs& to, cudaStream_t s) {
  TraceScope trace("prefix_spread", s);
  const int blocks = spread_blocks(p.a);
  const cudaError_t e = launch_dependent(p.a.d == 64 ? spread4_kernel<64> : spread4_kernel<128>,
                                         dim3(static_cast<unsigned>(to.num_pages) * (2 * blocks + 1)), dim3(kSpreadThreads), 0, s, p, to, blocks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_decode4(const DecodeParams& p, cudaStream_t s) {
  if (p.a.d == 64) return p.Rt == 4 ? launch<64, 4>(p, s) : p.Rt == 8 ? launch<64, 8>(p, s) : launch<64, 16>(p, s);
  return p.Rt == 4 ? launch<128, 4>(p, s) : p.Rt == 8 ? launch<128, 8>(p, s) : launch<128, 16>(p, s);
}

}  // namespace fox
