// Attention of the newest tokens of every sequence over the paged cache in fp32, on CUDA cores, and
// the merge of partial results (of this kernel's and of the bf16 one's, fox_decode_mma.cu).
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
__global__ void __launch_bounds__(32 * kSimtWarps) decode_simt_kernel(const DecodeParams p) {
  constexpr int E = D / 32;
  extern __shared__ long long cum[];  // [B + 1]
  __shared__ long long scratch[kSimtWarps];
  __shared__ float qs[kSimtWarps][kSimtRows][D];
  __shared__ double ci[kSimtWarps][kSimtRows];
  grid_dep_trigger();
  const PagedArgs& a = p.a;
  scan_units(p, cum, scratch);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += blockDim.x) p.cum[b] = cum[b];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv, Gp = p.Gp, S = a.page_size;
  const long long per_head = cum[a.B], total = per_head * a.Hkv;
  const long long each = units_per_worker(total, p.workers);
  const long long w = (long long)blockIdx.x * kSimtWarps + warp;
  long long u = w * each;
  const long long u_end = min(total, u + each);
  while (u < u_end) {
    const int hkv = static_cast<int>(u / per_head);
    const long long in_head = u - hkv * per_head;
    const int b = find_seq(cum, a.B, in_head);
    bool bad;
    const SeqInfo s = seq_info(a, b, &bad);
    const int P = p.walk_prefix ? a.prefix_len : 0;
    const int keys = walk_keys(a, s, p.walk_prefix), tiles = ceil_div(keys, kKeyTile);
    const int rt = static_cast<int>((in_head - cum[b]) / tiles);
    const int tile0 = static_cast<int>((in_head - cum[b]) % tiles);
    const int tile1 = static_cast<int>(min(static_cast<long long>(tiles), tile0 + (u_end - u)));
    const int R = min(p.Rt, s.n * Gp - rt * p.Rt);

    __syncwarp();
    for (int r = 0; r < R; ++r) {
      const int rr = rt * p.Rt + r, t = rr / Gp, h = hkv * G + min(rr % Gp, G - 1);
      const float* src = static_cast<const float*>(p.q) + (size_t)(s.row0 + t) * p.q_stride + (size_t)h * D;
      for (int c = lane * 4; c < D; c += 128) {
        float f[4];
        load4(src + c, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) qs[warp][r][c + e] = f[e] * p.scale2;
      }
      if (lane == 0) ci[warp][r] = gate_at(a, b, s.own - s.n + t, h);
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
        const int at = j < P ? j : j - P;
        page = j < P ? prefix_page(a, j) : own_page(a, b, at);
        slot = at % S;
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
          const int rr = rt * p.Rt + r, t = rr / Gp, h = hkv * G + min(rr % Gp, G - 1);
          if (j <= P + s.own - s.n + t) {
            const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
            const float beta = static_cast<float>(ci[warp][r] - base.x - base.y);
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
    // The item's first and last unit say whether this worker has all of it.
    const long long i0 = hkv * per_head + cum[b] + (long long)rt * tiles, i1 = i0 + tiles - 1;
    const bool whole = i0 / each == i1 / each;
    const size_t slot0 = (size_t)(w + ((long long)hkv * a.B + b) * p.RTmax + rt) * p.Rs;
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      if (r >= R) continue;
      float sum = l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int rr = rt * p.Rt + r, t = rr / Gp, h = hkv * G + min(rr % Gp, G - 1);
      if (rr % Gp >= G) continue;  // an empty row
      if (whole) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= inv;
        const size_t row = (size_t)(s.row0 + t) * a.H + h;
        put_out<float>(static_cast<float*>(p.o) + row * D + lane * E, acc[r], E);
        if (lane == 0) p.lse[row] = sum > 0.f ? (m[r] + log2f(sum)) * kLn2 : -INFINITY;
      } else {
        if (lane == 0) p.ml[slot0 + r] = make_float2(m[r], sum);
        put_out<float>(p.po + (slot0 + r) * D + lane * E, acc[r], E);
      }
    }
    u += tile1 - tile0;
  }
}

// One warp a (row, query head): the partial results of the row's item joined, in the workers' order.
// Rows of idle sequences get O = 0 and LSE = -inf.
constexpr int kMergeWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) decode_merge_kernel(const DecodeParams p) {
  constexpr int E = D / 32;
  grid_dep_wait();
  const PagedArgs& a = p.a;
  const long long id = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(id / a.H), h = static_cast<int>(id % a.H);
  if (row >= a.rows) return;
  const int b = seq_of_row(a, row);
  if (b < 0) return;
  bool bad;
  const SeqInfo s = seq_info(a, b, &bad);
  if (bad || row < s.row0 || row >= s.row0 + s.n) return;
  T* o = static_cast<T*>(p.o) + ((size_t)row * a.H + h) * D + lane * E;
  float* lse = p.lse + (size_t)row * a.H + h;
  float acc[E] = {};
  if (s.own < 0) {
    put_out<T>(o, acc, E);
    if (lane == 0) *lse = -INFINITY;
    return;
  }
  const int G = a.H / a.Hkv, hkv = h / G, r = (row - s.row0) * p.Gp + h % G;
  const int rt = r / p.Rt, tiles = ceil_div(walk_keys(a, s, p.walk_prefix), kKeyTile);
  const long long per_head = p.cum[a.B], each = units_per_worker(per_head * a.Hkv, p.workers);
  const long long i0 = hkv * per_head + p.cum[b] + (long long)rt * tiles, i1 = i0 + tiles - 1;
  const long long w0 = i0 / each, w1 = i1 / each;
  const bool shared = p.pre.key_tiles > 0;
  if (w0 == w1 && !shared) return;  // finished by its one worker
  // Partial results: the own item's, then the prefix's. Of result i, ml and po lie `step` rows further on.
  const int n_own = static_cast<int>(w1 - w0) + 1;
  const size_t own0 = (size_t)(w0 + ((long long)hkv * a.B + b) * p.RTmax + rt) * p.Rs + r % p.Rt;
  int n = n_own, step = 0;
  size_t pre0 = 0;
  float shift = 0.f;  // log2 e (c_i - c_last): what the row's prefix scores lack
  if (shared) {
    const PrefixPlan& x = p.pre;
    const int hl = h % G, tile = row / x.tpt * x.head_chunks + hl / x.hp;
    const int item = hkv * x.items + (x.row_tiles == 1 ? 0 : tile / 2);
    const long long pe = units_per_worker((long long)a.Hkv * x.items * x.key_tiles, x.workers);
    const long long v0 = (long long)item * x.key_tiles / pe, v1 = ((long long)(item + 1) * x.key_tiles - 1) / pe;
    const bool both = x.row_tiles == 1;  // the streams are two results, else this row is one stream's
    n += static_cast<int>(v1 - v0 + 1) * (both ? 2 : 1);
    step = both ? kTile : 2 * kTile;
    pre0 = ((size_t)(v0 + item) * 2 + (both ? 0 : tile & 1)) * kTile + row % x.tpt * x.hp + hl % x.hp;
    const int last = a.prefix_len - 1, page = max(prefix_page(a, last), 0);
    shift = static_cast<float>(gate_at(a, b, s.own - s.n + (row - s.row0), h) - gate_sum(a, page, last % a.page_size, h)) *
            kLog2e;
  }
  auto ml_of = [&](int i) {
    if (i < n_own) return p.ml[own0 + (size_t)i * p.Rs];
    float2 x = p.pre.ml[pre0 + (size_t)(i - n_own) * step];
    x.x += shift;
    return x;
  };
  auto po_of = [&](int i) {
    return i < n_own ? p.po + (own0 + (size_t)i * p.Rs) * D : p.pre.po + (pre0 + (size_t)(i - n_own) * step) * D;
  };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, ml_of(i).x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float safe = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int first = 0; first < n; first += 32) {
    float wgt = 0.f;
    if (first + lane < n) {
      const float2 ml = ml_of(first + lane);
      wgt = ex2_approx(ml.x - safe);
      l += ml.y * wgt;
    }
    const int c = min(32, n - first);
#pragma unroll 8
    for (int i = 0; i < c; ++i) {
      const float f = __shfl_sync(0xffffffffu, wgt, i);
      if (f == 0.f) continue;  // nothing of it counts (a stream without keys wrote no sums of V)
      const float* src = po_of(first + i) + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + e);
        acc[e] = fmaf(f, x.x, acc[e]);
        acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= inv;
  put_out<T>(o, acc, E);
  if (lane == 0) *lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

struct DecodeLayout {
  int Rt, Gp, Rs, RTmax, workers;
  size_t cum, ml, po, pml, ppo, end;
  PrefixPlan pre;
};

DecodeLayout decode_layout(const PagedArgs& a, bool f32) {
  DecodeLayout L;
  const int G = a.H / a.Hkv;
  L.Rt = f32 ? kSimtRows : decode_mma_rows(a.max_new * G);
  L.Gp = padded_group(G, L.Rt);
  const int most = a.max_new * L.Gp;
  L.Rs = most < L.Rt ? most : L.Rt;
  L.RTmax = ceil_div(most, L.Rt);
  L.workers = f32 ? kSMs * kSimtCtas * kSimtWarps : decode_mma_workers(a.d);
  const size_t slots = (size_t)L.workers + (size_t)a.B * a.Hkv * L.RTmax;
  L.cum = kErrWordBytes;
  L.ml = align_up(L.cum + sizeof(long long) * ((size_t)a.B + 1), 256);
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
  TraceScope trace("decode", s);
  decode_simt_kernel<D>
      <<<kSMs * kSimtCtas, 32 * kSimtWarps, sizeof(long long) * (p.a.B + 1), s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_merge(const DecodeParams& p, cudaStream_t s) {
  const long long blocks = ((long long)p.a.rows * p.a.H + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  TraceScope trace("decode_merge", s);
  const cudaError_t e = launch_dependent(decode_merge_kernel<T, D>, dim3(static_cast<unsigned>(blocks)),
                                         dim3(32 * kMergeWarps), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

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
  p.workers = L.workers;
  p.cum = reinterpret_cast<long long*>(ws + L.cum);
  p.ml = reinterpret_cast<float2*>(ws + L.ml);
  p.po = reinterpret_cast<float*>(ws + L.po);
  p.pre = L.pre;
  p.pre.ml = reinterpret_cast<float2*>(ws + L.pml);
  p.pre.po = reinterpret_cast<float*>(ws + L.ppo);
  cudaError_t e = p.pre.key_tiles > 0 ? launch_prefix(p, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  e = !f32 ? launch_decode_mma(p, s) : x.a.d == 64 ? launch_simt<64>(p, s) : launch_simt<128>(p, s);
  if (e != cudaSuccess) return e;
  if (f32) return x.a.d == 64 ? launch_merge<float, 64>(p, s) : launch_merge<float, 128>(p, s);
  return x.a.d == 64 ? launch_merge<__nv_bfloat16, 64>(p, s) : launch_merge<__nv_bfloat16, 128>(p, s);
}

}  // namespace fox
