// Attention of the newest tokens over the paged cache, bf16, on the tensor cores.
//
// Bound by memory: K and V of every key are read once, 2 bytes an element, for at most 16 query rows
// of work each: 64 sequences of up to 16384 tokens on 8 key heads (2.5 GB) take 381 us, 97 % of a copy's rate, one of
// 65536 (277 MB) 53 us, 12 of them launch, first look-ups and join; one of 1000 is these alone, 13 us. So the kernel
// is built to keep copies in flight, and uses the small register MMAs
// (16 x 8 x 16), of which it needs too few to matter: 128-row tensor-memory tiles would be 8 to
// 128 times padding here.
//
// One warp is one worker of the work line (fox_paged.h), with a ring of key tiles of its own that TMA
// fills: no barrier joins the warps, and each has the next tiles on their way while it computes.
// A stage holds 32 keys: K, V (128-byte swizzled, 64 channels a block) and the gates' sums g of the
// row tile's heads, from four slots before the first key, so that the exclusive sums of bias_from_j
// are there too (0 before a page's first slot, which is what TMA fills in).
//
// Transposed products, so that the few query rows are the 8-wide side and K and V the 16-high one:
//   S^T (keys x rows) = K Q^T     K as it lies (ldmatrix), Q in registers
//   O^T (d x rows)   += V^T P^T   V transposed on the way (ldmatrix.trans), P^T turned in registers
// x = scale2 S + log2e ((c_i - base of the page) - g_j), the difference of the cumulative sums in
// two fp32 each. The running maximum moves only when a score passes it by 2^8, which one vote finds.
// P is split into two bf16 terms (P = hi + lo, both multiplied): with one, its 8 significant bits
// would add to O an error as large as O's own rounding; V keeps its full bf16 range.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_decode_ring.h"

namespace fox {
namespace {

constexpr float kGrow = 8.0f;  // log2 units that a score may pass the running maximum by

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Sets the values of keys [from, to) of a tile of V that are infinite or no number to 0; true if there were any.
template <int D>
static __device__ __noinline__ bool take_out(uint8_t* v, int from, int to) {
  bool odd = false;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < (to - from) * (D / 8); e += 32) {
    const int row = from + e / (D / 8), c = e % (D / 8);
    uint4* at = reinterpret_cast<uint4*>(v + (c >> 3) * (kKeyTile * 128) + row * 128 + ((c ^ row) & 7) * 16);
    uint32_t w[4] = {at->x, at->y, at->z, at->w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
      any |= lo || hi;
      w[i] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
    }
    if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
    odd |= any;
  }
  fence_proxy_async_smem();  // before the next copy into the stage
  __syncwarp();
  return odd;
}
// What take_out took from keys that some of a segment's rows see, to the sums of those (rows + r * pitch), once more
// from the cache. Key tiles from tile0 to tile1.
template <int D>
static __device__ __noinline__ void put_back(const DecodeParams& p, const Place& at, int tile0, int tile1, int tp,
                                             float* rows, int pitch) {
  const PagedArgs& a = p.a;
  const int lane = threadIdx.x & 31, r0 = at.rt * p.Rt, R = rows_of(p, at), new0 = at.s.own - at.s.n;
  const int lo = max((tile0 - tp) * kKeyTile, new0 + token_of(p, r0) + 1);
  const int hi = min((tile1 - tp + 1) * kKeyTile, new0 + token_of(p, r0 + R - 1) + 1);
#pragma unroll 1
  for (int j = lo; j < hi; ++j) {
    const int page = own_page_or_0(a, at.b, j);
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + kv_offset(a, page, at.hkv, j & (a.page_size - 1));
#pragma unroll 1
    for (int ch = lane; ch < D; ch += 32) {
      const float f = __bfloat162float(v[ch]);
      if (fabsf(f) < INFINITY) continue;
#pragma unroll 1
      for (int r = 0; r < R; ++r)
        if (j <= new0 + token_of(p, r0 + r)) rows[r * pitch + ch] += f;
    }
  }
  __syncwarp();
}
// Shared memory: K and V of every (warp, stage), then its gates, then the sequences' work offsets.
// Gates of a stage: per sub-page (32 slots, or two of 16) [heads][slots + 4] sums, then [heads] bases.
struct MmaShape {
  int heads, gpitch;          // heads of a row tile; floats from one head's sums to the next's
  int gsub, gstage;           // bytes of a sub-page's sums (a TMA destination: 128-byte steps); of a stage's gates
};
inline MmaShape mma_shape(const PagedArgs& a, int rows) {
  const int G = a.H / a.Hkv, subs = a.page_size == 16 ? 2 : 1;
  MmaShape x;
  x.heads = G < rows ? G : rows;
  x.gpitch = (subs == 2 ? 16 : kKeyTile) + 4;
  x.gsub = (x.heads * x.gpitch * 4 + 127) / 128 * 128;
  x.gstage = subs * x.gsub + (subs * x.heads * 8 + 127) / 128 * 128;
  return x;
}
constexpr int most_gates(int rows) { return 2 * ((rows * 20 * 4 + 127) / 128 * 128) + rows * 16; }  // gstage at most

// An item's rows are asked for by asynchronous copies while the item before is computed: Q and the gates when
// that one begins, for which the table's entries for the rows' own tokens are there, asked for an item earlier.
// Against loads when the item begins: 256 sequences of up to 500 86.5 -> 80.6 us, one of 65536 59.1 -> 57.3, 16 of up to 4096
// with four tokens each 70.0 -> 68.7; 128 of up to 200 with 64 channels 29.7 -> 30.6.
template <int kRows>
struct ItemRows {
  Place at[2];         // by the item's number & 1, as the entries are
  int page[2][kRows];
  float g[kRows];
  float2 base[kRows];
};

// kMany: sequences may bring more than one token, so that a tile may hold keys that some of an item's rows do not see
// (a kernel of its own: one token a sequence took 0.5 to 4 % longer with that code in it, several tokens take up to 2 %).
template <int D, int NT, bool kMany>
__global__ void __launch_bounds__(32 * MmaLayout<D, NT>::kWarps, 1)
    decode_mma_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                      const __grid_constant__ CUtensorMap tmap_g, const __grid_constant__ DecodeParams p,
                      const MmaShape x) {
  using L = MmaLayout<D, NT>;
  constexpr int W = L::kWarps;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int scratch[W];
  __shared__ __align__(8) uint64_t bars[W][L::kStages];
  __shared__ int abort_word;
  __shared__ Kept<L::kRows, W> kept;
  __shared__ int ids[W][2][64];  // two windows' table entries, by asynchronous copies: no instruction waits for them before their use
  __shared__ BlockEnds ends;
  __shared__ ItemRows<L::kRows> rows_of[W];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &abort_word;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ItemRows<L::kRows>& it = rows_of[warp];
  constexpr int stages = L::kStages;
  uint8_t* ring = sm + warp * stages * (2 * L::kTileBytes);
  uint8_t* gates = sm + W * stages * (2 * L::kTileBytes) + warp * stages * x.gstage;
  uint8_t* q_of = sm + W * stages * (2 * L::kTileBytes + x.gstage) + warp * L::kQBytes;
  SeqEntry* seqs = reinterpret_cast<SeqEntry*>(sm + W * (stages * (2 * L::kTileBytes + x.gstage) + L::kQBytes));

  const bool shared = p.pre.key_tiles > 0;
  if (threadIdx.x == 0) abort_word = 0;
  if (lane == 0) {
    kept.i0[warp] = -1;
    for (int s = 0; s < stages; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
  }
  // Behind a shared prefix's kernel, which nothing here needs and which let this one start once all before it
  // were through, the wait comes last.
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
  uint32_t qf[D / 16][NT][2];
  float acc[D / 16][NT][4];
  float m[NT][2], l[NT][2];
  Gate2 ci[NT][2];
  int pos[NT][2], gidx[NT][2];
  int first = 0, last = 0;  // with kMany: own positions of the item's first and last row
  bool odd = false;         // with kMany: an infinity or a NaN was taken out of the item's V
  // ldmatrix addresses of this lane: K rows (keys) x 16-byte channel chunks, V the same, transposed.
  const uint64_t policy = stream_policy();
  const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kchunk = lane >> 4;
  const int vrow = (lane & 7) + (lane >> 4) * 8, vchunk = (lane >> 3) & 1;

  // The consumer's place, and the producer's, which runs ahead by a window or two.
  Place cur = {}, pro = {};
  // The step that opened the item; items whose entries, and whose Q and gates, were asked for;
  // the units of the first `asked` ones.
  int since = -stages, asked = 0, filled = 0, ahead = 0;
  if (count > 0) cur = pro = place_of(p, seqs, u0);
  Window now = {}, next = {};
  int left = count, at = 0, buf = 0;  // units that no window holds yet; the producer's next tile of `now`; now's ids
  bool fresh = true, opened = false, ok = true;
  int stage = 0;
  uint32_t phase = 0;

  // Step n consumes tile n and then issues the copies of tile n + stages; the first `stages` only issue.
#pragma unroll 1
  for (int n = -stages; n < count; ++n) {
    if (n == 0 && warp == 0) find_ends<W>(p, seqs, total, each, ends);  // while the first copies are on their way
    if (n >= 0) {
      if (!opened) {
        // The item's rows: Q fragments, and places and cumulative gates of this thread's columns of S^T, rows
        // 2 t4 and 2 t4 + 1; nothing summed yet.
        opened = true;
        if (n - since > 1)
          cp_async_wait<1>();  // asked for before the last step
        else
          cp_async_wait<0>();
        __syncwarp();
        since = n;
        fresh = true;
        const uint32_t qa = smem_u32(q_of);
        const int r0 = cur.rt * p.Rt;
        if (kMany) {
          first = cur.s.own - cur.s.n + token_of(p, r0);
          last = cur.s.own - cur.s.n + min(token_of(p, r0 + p.Rt - 1), cur.s.n - 1);
          odd = false;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ks += 2) {
            uint32_t f[4];
            const int row = nt * 8 + (lane & 7), chunk = ks * 2 + (lane >> 3);
            ldsm4(qa + row * (D * 2) + ((chunk ^ (row & 7)) << 4), f);
            qf[ks][nt][0] = f[0];
            qf[ks][nt][1] = f[1];
            qf[ks + 1][nt][0] = f[2];
            qf[ks + 1][nt][1] = f[3];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rl = nt * 8 + 2 * t4 + e, r = r0 + rl, t = token_of(p, r), g = r - t * Gp;
            const bool here = t < cur.s.n && g < G;
            pos[nt][e] = cur.s.own - cur.s.n + t;
            gidx[nt][e] = here ? (G > L::kRows ? g - r0 % Gp : g) : 0;
            ci[nt][e] = {-INFINITY, 0.f};  // an empty row's scores are -inf
            if (here) ci[nt][e] = gate_sum(it.base[rl], it.g[rl]);
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
          }
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[dt][nt][e] = 0.f;
      }
      uint8_t* st = ring + stage * (2 * L::kTileBytes);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[warp][stage], phase, abort_flag, a.err, DEV_ERR_TIMEOUT_TMA));
      if (!ok) break;
      cp_async_wait<L::kStages - 1>();  // the stage's bases: so many groups were committed after theirs
      __syncwarp();

      // The tile's keys are those of the prefix, or of the sequence's own, which end for each row with its own: every
      // row sees the keys before `seen`, no row those from `end` on.
      const bool pre = cur.tile < tp;
      const int j0 = (pre ? cur.tile : cur.tile - tp) * kKeyTile, seen = pre ? P : kMany ? first + 1 : cur.s.own,
                end = pre ? P : kMany ? last + 1 : cur.s.own;
      const uint32_t sk = smem_u32(st), sv = sk + L::kTileBytes;
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t kf[4];
          const int row = mt * 16 + krow, chunk = (ks & 3) * 2 + kchunk;
          ldsm4(sk + (ks >> 2) * (kKeyTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), kf);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], kf, qf[ks][nt][0], qf[ks][nt][1]);
        }
      }
      // Scores of keys mt * 16 + g8 (+ 8) and rows 2 t4 (+ 1), in log2 units.
      const uint8_t* sg = gates + stage * x.gstage;
      const float2* bs = reinterpret_cast<const float2*>(sg + base_off);
      const bool edge = j0 + kKeyTile > (pre ? P : cur.s.own - cur.s.n);  // some slot is no key of some row
      bool grow = false;
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
              float x = fmaf(beta - gr[key], kLog2e, s[mt][nt][k8 * 2 + e] * p.scale2);
              if (edge && j0 + mt * 16 + key > (pre ? P - 1 : pos[nt][e])) x = -INFINITY;
              s[mt][nt][k8 * 2 + e] = x;
              top[nt][e] = fmaxf(top[nt][e], x);
            }
          }
          grow |= top[nt][e] > m[nt][e] + kGrow;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float mn = fmaxf(m[nt][e], x);
            const float alpha = mn == -INFINITY ? 1.f : ex2_approx(m[nt][e] - mn);
            m[nt][e] = mn;
            l[nt][e] *= alpha;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
              acc[dt][nt][e] *= alpha;
              acc[dt][nt][e + 2] *= alpha;
            }
          }
      }
      if (j0 + kKeyTile > end && (!kMany || j0 < end)) {
        // Slots behind the end may hold anything: V there becomes 0 (its weights are 0).
        for (int e = lane; e < (j0 + kKeyTile - end) * (D / 8); e += 32) {
          const int row = end - j0 + e / (D / 8), c = e % (D / 8);
          sts_v4(sv + (c >> 3) * (kKeyTile * 128) + row * 128 + (c & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before the next copy into this stage
        __syncwarp();
      }
      // So does what is no number in the values of a key that only some of the rows see: times the others' weights of 0
      // it would be a NaN.
      if (kMany && j0 < end && j0 + kKeyTile > seen && seen < end)
        odd |= take_out<D>(st + L::kTileBytes, max(seen - j0, 0), min(end - j0, kKeyTile));
      if (!kMany || j0 < end) {  // not where no row sees a key of the tile
        // P^T fragments, hi and lo.
        uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float o0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], o1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8) {
              const float p0 = ex2_approx(s[mt][nt][k8 * 2] - o0), p1 = ex2_approx(s[mt][nt][k8 * 2 + 1] - o1);
              l[nt][0] += p0;
              l[nt][1] += p1;
              const uint32_t hi = pack_bf16x2(p0, p1);
              ph[mt][nt][k8] = turn8x8(hi);
              pl[mt][nt][k8] = turn8x8(pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u)));
            }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t vf[4];
            const int row = mt * 16 + vrow, chunk = (dt & 3) * 2 + vchunk;
            ldsm4_t(sv + (dt >> 2) * (kKeyTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), vf);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(acc[dt][nt], vf, ph[mt][nt][0], ph[mt][nt][1]);
              mma16816(acc[dt][nt], vf, pl[mt][nt][0], pl[mt][nt][1]);
            }
          }
      }
      __syncwarp();  // every lane has read the stage

      if (cur.tile + 1 == cur.tiles || n + 1 == count) {
        // Results: O^T through shared memory to rows, finished or the worker's part of them: by the stage just
        // read, or, for the block to join with its neighbours', kept at the ring's start (all copies were read).
        const bool alone = cur.i0 >= u0 && cur.i0 + cur.tiles <= u0 + count, keep = !alone && n + 1 == count;
        float* out = reinterpret_cast<float*>(keep ? ring : st);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = l[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            const int rl = nt * 8 + 2 * t4 + e;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
              out[rl * L::kOutStride + dt * 16 + g8] = acc[dt][nt][e];
              out[rl * L::kOutStride + dt * 16 + g8 + 8] = acc[dt][nt][e + 2];
            }
            if (g8 == 0) {
              kept.m[warp][rl] = m[nt][e];
              kept.l[warp][rl] = y;
            }
          }
        if (kMany && __any_sync(0xffffffffu, odd)) {
          __syncwarp();
          put_back<D>(p, cur, max(u0 - cur.i0, 0), cur.tile, tp, out, L::kOutStride);
        }
        if (keep && lane == 0) {
          kept.i0[warp] = cur.i0;
          kept.at[warp] = cur;
        }
        __syncwarp();
        if (!keep)
          leave_rows<__nv_bfloat16, D>(p, cur, w, alone && !shared, out, L::kOutStride, kept.m[warp], kept.l[warp]);
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
        const int r = at_item.rt * p.Rt + lane, t = token_of(p, r), g = r - t * Gp;
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
          const int r = r0 + lane, t = token_of(p, r), g = r - t * Gp, h = at_item.hkv * G + g;
          if (lane < L::kRows && t < at_item.s.n && g < G) {
            const int page = checked_page(a, it.page[slot][lane]);
            cp_async8(smem_u32(&it.base[lane]), a.gbase + gbase_offset(a, page, h));
            cp_async4(smem_u32(&it.g[lane]), a.g + g_offset(a, page, h, (at_item.s.own - at_item.s.n + t) & (S - 1)));
          }
        }
#pragma unroll 1
        for (int e = lane; e < L::kRows * (D / 8); e += 32) {
          const int rl = e / (D / 8), chunk = e % (D / 8), r = r0 + rl, t = token_of(p, r), g = r - t * Gp;
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
      uint8_t* dst = ring + to * (2 * L::kTileBytes);
      uint8_t* sg = gates + to * x.gstage;
      const int h0 = now.hkv * G + (G > L::kRows ? now.rt * p.Rt % Gp : 0);
      const int t = now.tile + at, j = (t < tp ? t : t - tp) * kKeyTile, slot = j & (S - 1);
      const int subs = S == 16 && j + 16 < (t < tp ? P : now.own) ? 2 : 1;  // pages of 16: the second may be none
      if (lane == 0) mbar_arrive_expect_tx(&bars[warp][to], subs * (2 * KS * D * 2 + heads * gpitch * 4));
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < subs; ++i) {
        const int id = checked_page(a, ids[warp][buf][32 * i + at]);
        // One lane a copy: K and V of 64 channels each, and the gates.
        if (lane < D / 32) {
          const int y = lane >> 1;
          tma_load_4d_by(policy, dst + (lane & 1) * L::kTileBytes + y * (kKeyTile * 128) + i * (16 * 128), lane & 1 ? &tmap_v : &tmap_k,
                      &bars[warp][to], y * 64, slot, now.hkv, id);
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
  // Sums and offsets stand in the first and the second warp's second stage.
  const int warp_bytes = stages * (2 * L::kTileBytes);
  static_assert(32 * W * sizeof(Column) <= 2 * L::kTileBytes && (kSMs + 1) * 4 <= 2 * L::kTileBytes, "they fit there");
  join_items<__nv_bfloat16, D, L::kRows, W>(p, seqs, total, each, kept, ends, reinterpret_cast<const float*>(sm),
                                            warp_bytes / 4, L::kOutStride,
                                            reinterpret_cast<int*>(sm + warp_bytes + 2 * L::kTileBytes),
                                            reinterpret_cast<Column*>(sm + 2 * L::kTileBytes));
  // With a shared prefix a merge follows, launched as a dependent of this kernel as this one is of the
  // prefix's; it needs both grids to be through, so this one ends after that one.
  if (shared) grid_dep_wait();
}

template <int D, int NT, bool kMany>
cudaError_t launch_as(const DecodeParams& p, const CUtensorMap* maps, cudaStream_t s) {
  using L = MmaLayout<D, NT>;
  auto kernel = decode_mma_kernel<D, NT, kMany>;
  const MmaShape x = mma_shape(p.a, L::kRows);
  constexpr int kMostGates = most_gates(L::kRows);
  constexpr size_t kMost = 232448 - 12288;  // of an SM's shared memory, less the static part
  const size_t fixed = 1024 + (size_t)L::kWarps * L::kQBytes + sizeof(SeqEntry) * ((size_t)p.a.B + 1);
  const size_t one = (size_t)L::kWarps * (2 * L::kTileBytes + x.gstage);
  const size_t smem = fixed + L::kStages * one;
  // The limit is the function's, not the call's: always the same value, the most that any call takes, so that host
  // threads with different batches do not lower it between each other's calls here and launches.
  constexpr size_t kLimit = 1024 + sizeof(SeqEntry) * (kMaxSeqs + 1) +
                            L::kWarps * (L::kQBytes + L::kStages * (2 * L::kTileBytes + kMostGates));
  static_assert(kLimit <= kMost, "shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLimit));
  if (e != cudaSuccess) return e;
  TraceScope trace("decode", s);
  const cudaError_t f =
      launch_dependent(kernel, dim3(kSMs), dim3(32 * L::kWarps), smem, s, maps[0], maps[1], maps[2], p, x);
  return f != cudaSuccess ? f : cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch(const DecodeParams& p, const CUtensorMap* maps, cudaStream_t s) {
  return p.a.max_new > 1 ? launch_as<D, NT, true>(p, maps, s) : launch_as<D, NT, false>(p, maps, s);
}

}  // namespace

int decode_mma_warps(int d) { return d == 128 ? MmaLayout<128, 1>::kWarps : MmaLayout<64, 1>::kWarps; }
int decode_mma_rows(int rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_decode_mma(const DecodeParams& p, cudaStream_t s) {
  const PagedArgs& a = p.a;
  const int KS = a.page_size < kKeyTile ? a.page_size : kKeyTile, G = a.H / a.Hkv;
  CUtensorMap maps[3];
  if (!make_page_map(&maps[0], a.k, a.d, a.page_size, a.Hkv, a.num_pages, KS) ||
      !make_page_map(&maps[1], a.v, a.d, a.page_size, a.Hkv, a.num_pages, KS) ||
      !make_f32_3d_map(&maps[2], a.g, a.page_size, a.H, a.num_pages, (uint64_t)a.page_size * 4,
                       (uint64_t)a.page_size * a.H * 4, KS + 4, G < p.Rt ? G : p.Rt))
    return cudaErrorInvalidValue;
  if (a.d == 64) return p.Rt == 8 ? launch<64, 1>(p, maps, s) : launch<64, 2>(p, maps, s);
  return p.Rt == 8 ? launch<128, 1>(p, maps, s) : launch<128, 2>(p, maps, s);
}

}  // namespace fox
