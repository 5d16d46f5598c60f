// Appending new tokens to the 4-bit cache, and reading tokens back.
//
// Q is rotated as in fox_append.cu. K is too, but to the nearest bf16 of the exact a cos - b sin: the 4-bit form has borders everywhere, and a
// value on the other side of one is a whole step away. Kahan's difference of products (one product's rounding error by a fused
// multiply-add, taken off the fused difference) is within 1.5 units of the last place of fp32; where that leaves open on which side of
// a border of bf16 a value lies (1 of 8000), 64 bits decide, in which the products are exact.
//
// A thread has 16 channels of up to eight rows: a chunk of 8 and its partner's in the rotation, or two neighbouring chunks. A block of 32
// channels is two threads' neighbouring chunks (K that was rotated with a partner passes through shared memory for that): its largest
// magnitude by a shuffle, its scale by the first of them, two words of codes by each (fox_four.h).
//
// Bound by memory, as far as rows are on their way (6 prompts of up to 16384 tokens, 32 + 2 * 8 heads of 128, rotation in pairs: 1.27 GB in
// 242 us, 5.2 TB/s; 18 % fewer instructions, with q in a loop of its own, took as long). What that took: the rows of a thread in turn by
// the same code (unrolled, the warps waited for instructions: 427 us, in turn 297), a row's loads one row ahead of its use and 64
// registers, so that 8 blocks are on an SM
// (four rows ahead and 6 blocks 289, two and 8 blocks 258, one and 10 blocks with spills 311), and eight rows a thread, before which a block looks up
// where its rows stand (four 266, sixteen 250 but 62 for 57 where they are read back).
// One token of each of 128 sequences: 12 us by itself, most of it the launch and dependent trips to memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_append.cuh"
#include "fox_four.h"

namespace fox {
namespace {

struct Append4Params : AppendParams {
  uint8_t* ks;
  uint8_t* vs;
  int thread_rows;
};
constexpr int kResident = 8;                           // blocks of an SM
constexpr int kMostRows = 8;                           // rows of a thread
constexpr int kMostPlaces = kMostRows * kThreads / 8;  // of a block
using Bf16 = Vec<__nv_bfloat16>;

// a c - b s: rounded to fp32 twice, or within 1.5 units of the last place.
template <bool kExact>
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  if (!kExact) return a * c - b * s;
  const float p = __fmul_rn(b, s), e = __fmaf_rn(b, s, -p);
  return __fsub_rn(__fmaf_rn(a, c, -p), e);
}
// The same through 64 bits, in which the products are exact, but not the difference of two that lie far apart: rounded down and up, to 64 bits
// and then to fp32, which leaves the fp32 value itself, or its two neighbours. Of these the odd one then rounds to bf16 as the exact one does.
__device__ __forceinline__ float turned_exactly(float a, float c, float b, float s) {
  const double q = -(static_cast<double>(b) * s);
  const float below = __double2float_rd(__fma_rd(a, c, q)), above = __double2float_ru(__fma_ru(a, c, q));
  return __float_as_uint(below) & 1u ? below : above;
}
// `least` so far and two values' lower halves less 0x7FFD, modulo 2^16, where a border of bf16 is 3 (a carry may add 1 to the upper):
// up to 7 the side of the border is open (1.5 units, 2.5 where products are subnormal).
__device__ __forceinline__ uint32_t border(uint32_t least, float x, float y) {
  return __vminu2(least, __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x5410) + 0x80038003u);
}
__device__ __forceinline__ bool at_border(uint32_t least) { return (least & 0xFFFFu) <= 7u || (least >> 16) <= 7u; }

// Sixteen channels, x and y, turned by eight angles: channel i of x with i of y, or neighbours of either.
struct Sixteen {
  uint4 x, y;
};
template <bool kNeighbours, typename F>
__device__ __forceinline__ Sixteen turn_with(const Sixteen& w, const float* cs, const float* sn, F turn) {
  float x[8], y[8], co[8], si[8];
  Bf16::unpack(w.x, x);
  Bf16::unpack(w.y, y);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const float4 c = *reinterpret_cast<const float4*>(cs + k), s = *reinterpret_cast<const float4*>(sn + k);
    co[k] = c.x, co[k + 1] = c.y, co[k + 2] = c.z, co[k + 3] = c.w;
    si[k] = s.x, si[k + 1] = s.y, si[k + 2] = s.z, si[k + 3] = s.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& p = kNeighbours ? (i < 4 ? x[2 * i] : y[2 * i - 8]) : x[i];
    float& q = kNeighbours ? (i < 4 ? x[2 * i + 1] : y[2 * i - 7]) : y[i];
    const float a = p, b = q;
    p = turn(a, co[i], b, si[i]);
    q = turn(b, co[i], -a, si[i]);
  }
  return {Bf16::pack(x), Bf16::pack(y)};
}
template <bool kNeighbours>
__device__ __noinline__ Sixteen turn16_exactly(Sixteen w, const float* cs, const float* sn) {
  return turn_with<kNeighbours>(w, cs, sn, turned_exactly);
}
template <bool kNeighbours>
__device__ __forceinline__ Sixteen turn16(const Sixteen& w, const float* cs, const float* sn, bool exact) {
  if (!exact) return turn_with<kNeighbours>(w, cs, sn, turned<false>);
  uint32_t least = 0xFFFFFFFFu;
  float last = 0.f;
  int n = 0;
  const Sixteen z = turn_with<kNeighbours>(w, cs, sn, [&](float a, float c, float b, float s) {
    const float x = turned<true>(a, c, b, s);
    if (n++ & 1) least = border(least, last, x);
    last = x;
    return x;
  });
  return at_border(least) ? turn16_exactly<kNeighbours>(w, cs, sn) : z;
}

// Codes of eight of a block's values. Where the block has an infinity, a NaN or what is too large (its scale is then the largest) each is
// held as the nearest there is.
__device__ __forceinline__ uint32_t block_codes(const uint4& w, float inv, bool odd) {
  float f[8];
  Bf16::unpack(w, f);
  if (odd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] == f[e] ? fminf(fmaxf(f[e], -430080.f), 430080.f) : 0.f;
  }
  return four_codes(f, inv);
}

// Where a row's tokens stand: of head 0, counted through the pool (check_four); kNoRow: the row is not appended.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
struct RowToken {
  uint32_t token;
  int slot, pos;
};
__device__ __forceinline__ RowToken row_token(const AppendParams& p, int row) {
  const RowPlace x = row_place(p, row);
  return {x.page < 0 ? kNoRow : static_cast<uint32_t>(x.page) * p.a.Hkv * p.a.page_size + x.slot, x.slot, x.pos};
}

enum Turn { kNone, kHalves, kPairs };  // channel i with i + rot / 2; 2 i with 2 i + 1

template <Turn kTurn>
__device__ __forceinline__ void copy_rows4(const Append4Params& p, RowToken* places, uint4* exchange) {
  const PagedArgs& a = p.a;
  const int hs = a.d == 128 ? 3 : 2, hp = 1 << hs, blocks = a.d / kFourBlock;  // units of a head
  const int nk = a.Hkv << hs;
  const CopyShape x = copy_shape(2 * nk + (p.qn ? a.H << hs : 0));
  const int tid = threadIdx.x, lane = tid & 31, block = blockIdx.x - p.gate_blocks;
  const int chunk = block % x.chunks, row0 = block / x.chunks * (p.thread_rows * x.side);
  const int sub = x.side > 1 ? tid / x.per_row : 0, at = x.side > 1 ? tid - sub * x.per_row : chunk * kThreads + tid;
  // Units of a row are a multiple of 4 (8 with 128 channels) and so are a block's: a head's lie in neighbouring lanes.
  const bool live = at < x.per_row && sub < x.side, is_v = at >= nk && at < 2 * nk, is_q = at >= 2 * nk;
  const int w = is_q ? at - 2 * nk : is_v ? at - nk : at, h = w >> hs, j = w & (hp - 1);
  const int half = p.rot / 2;
  const bool apart = kTurn == kHalves && !is_v && j * 8 < half;
  const int c0 = (apart ? j : 2 * j) * 8, c1 = apart ? c0 + half : c0 + 8;
  const bool turns = kTurn != kNone && !is_v && c0 < p.rot;
  const long long stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_q ? p.qn : is_v ? p.vn : p.kn) +
                             (size_t)(row0 + sub) * stride + h * a.d;
  const int rows = min(p.thread_rows * x.side, a.rows - row0);
  Sixteen next;
  auto fetch = [&](int r) {
    if (r < rows) next = {__ldcs(reinterpret_cast<const uint4*>(src + c0)), __ldcs(reinterpret_cast<const uint4*>(src + c1))};
    src += x.side * stride;
  };
  if (live) fetch(sub);
  for (int r = tid; r < rows; r += kThreads) places[r] = row_token(p, row0 + r);
  __syncthreads();
  if (!live) return;  // a head's lanes live or not together
  const uint32_t head_lanes = (hp == 8 ? 0xFFu : 0xFu) << (lane & ~(hp - 1));
  const int b = j >> 1, t = 2 * j & 3, head = h * a.page_size;  // of the two neighbouring chunks that are held
  const float* cs = p.cos + (kTurn == kPairs ? c0 / 2 : c0);
  const float* sn = p.sin + (kTurn == kPairs ? c0 / 2 : c0);
  __nv_bfloat16* q_out = static_cast<__nv_bfloat16*>(p.qo) + ((size_t)(row0 + sub) * a.H + h) * a.d;
  uint4* mine = exchange + (tid & ~(hp - 1)) * 2;  // a head's channels
#pragma unroll 1
  for (int r = sub; r < rows; r += x.side) {
    Sixteen y = next;
    fetch(r + x.side);
    const RowToken g = places[r];  // of the row: the same for all of its lanes
    if (g.token == kNoRow) continue;
    if (turns) y = turn16<kTurn == kPairs>(y, cs + (size_t)g.pos * half, sn + (size_t)g.pos * half, !is_q);
    if (is_q) {
      __nv_bfloat16* dst = q_out + (size_t)(r - sub) * a.H * a.d;
      __stcs(reinterpret_cast<uint4*>(dst + c0), y.x);
      __stcs(reinterpret_cast<uint4*>(dst + c1), y.y);
      continue;
    }
    if (kTurn == kHalves && !is_v) {
      mine[c0 >> 3] = y.x;
      mine[c1 >> 3] = y.y;
      __syncwarp(head_lanes);
      y = {mine[2 * j], mine[2 * j + 1]};
      __syncwarp(head_lanes);
    }
    uint32_t most = four_larger(four_larger(y.x), four_larger(y.y));
    most = four_larger(most, __shfl_xor_sync(0x3u << (lane & ~1), most, 1));
    const float top = fabsf(__uint_as_float(four_larger(most, most << 16) & 0xFFFF0000u));
    const uint32_t byte = four_scale_byte(top);
    const float inv = byte ? __fdividef(1.f, four_scale(byte)) : 0.f;  // 2 units of the last place are enough (four_code_bits)
    const bool odd = !(top <= 430080.f);
    if (odd && a.err) atomicOr(a.err, DEV_ERR_RANGE);
    const uint32_t w0 = block_codes(y.x, inv, odd), w1 = block_codes(y.y, inv, odd);
    const uint32_t token = g.token + head;
    uint8_t* row = static_cast<uint8_t*>(is_v ? a.v : a.k) + (uint64_t)token * (a.d / 2);
    if (is_v) {
      *reinterpret_cast<uint2*>(row + four_v_word(b, t, g.slot, blocks)) = make_uint2(w0, w1);
      if (t == 0) p.vs[(uint64_t)(token - (g.slot & 15)) * blocks + four_v_scale(b, g.slot, blocks)] = static_cast<uint8_t>(byte);
    } else {
      *reinterpret_cast<uint32_t*>(row + four_k_word(b, t, blocks)) = four_k_order(w0);
      *reinterpret_cast<uint32_t*>(row + four_k_word(b, t + 1, blocks)) = four_k_order(w1);
      if (t == 0) p.ks[(uint64_t)token * blocks + b] = static_cast<uint8_t>(byte);
    }
  }
}

template <Turn kTurn>
__global__ void __launch_bounds__(kThreads, kResident) cache_append4_kernel(const Append4Params p) {
  __shared__ __align__(16) union {
    float zs[128][kGateHeads + 1];
    struct {
      uint4 exchange[kTurn == kHalves ? 2 * kThreads : 1];
      RowToken places[kMostPlaces];
    } rows;
  } sh;
  grid_dep_wait();
  grid_dep_trigger();
  if (static_cast<int>(blockIdx.x) < p.gate_blocks)
    gate_block(p, sh.zs);
  else
    copy_rows4<kTurn>(p, sh.rows.places, sh.rows.exchange);
}

// The values of rows, 16 channels a thread: a chunk of each half of a head, so that stores are contiguous over lanes. s u has 7
// significant bits, so bf16 has it exactly. Bound by memory, what is written above all (the tokens of 6 prompts: 0.3 GB in 57 us, 5.2 TB/s; a chunk
// and four rows a thread, so that blocks are short and look-ups many: 86).
struct Read4Params : AppendParams {
  const uint8_t* ks;
  const uint8_t* vs;
  __nv_bfloat16* ko;
  __nv_bfloat16* vo;
  int thread_rows;
};
__global__ void __launch_bounds__(kThreads, 10) cache_read4_kernel(const Read4Params p) {
  __shared__ RowToken places[kMostPlaces];
  grid_dep_wait();
  grid_dep_trigger();
  const PagedArgs& a = p.a;
  const int hs = a.d == 128 ? 3 : 2, blocks = a.d / kFourBlock, half = blocks / 2, nk = a.Hkv << hs;
  const CopyShape x = copy_shape(2 * nk);
  const int tid = threadIdx.x, chunk = blockIdx.x % x.chunks, row0 = blockIdx.x / x.chunks * (p.thread_rows * x.side);
  const int sub = x.side > 1 ? tid / x.per_row : 0, at = x.side > 1 ? tid - sub * x.per_row : chunk * kThreads + tid;
  const bool live = at < x.per_row && sub < x.side, is_v = at >= nk;
  const int w = is_v ? at - nk : at, h = w >> hs, j = w & ((1 << hs) - 1), b = j >> 2, t = j & 3, head = h * a.page_size;
  const int rows = min(p.thread_rows * x.side, a.rows - row0);
  for (int r = tid; r < rows; r += kThreads) places[r] = row_token(p, row0 + r);
  __syncthreads();
  if (!live) return;
  const long long stride = (is_v ? p.v_stride : p.k_stride) * x.side;
  __nv_bfloat16* out = (is_v ? p.vo : p.ko) + (size_t)(row0 + sub) * (is_v ? p.v_stride : p.k_stride) + h * a.d + j * 8;
  const uint8_t* held = static_cast<const uint8_t*>(is_v ? a.v : a.k);
  const uint8_t* scales = is_v ? p.vs : p.ks;
  const int apart = is_v ? 4 * half : half;  // the two blocks' scales
#pragma unroll 1
  for (int first = sub; first < rows; first += kRows * x.side) {
    uint32_t w0[kRows], w1[kRows], s0[kRows], s1[kRows];
    bool here[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = i * x.side + first;
      const RowToken g = r < rows ? places[r] : RowToken{kNoRow, 0, 0};
      here[i] = g.token != kNoRow;
      if (!here[i]) continue;
      const uint32_t token = g.token + head;
      const uint8_t* row = held + (uint64_t)token * (a.d / 2);
      const int word = is_v ? four_v_word(b, t, g.slot, blocks) : four_k_word(b, t, blocks);
      const uint8_t* scale = scales + (is_v ? (uint64_t)(token - (g.slot & 15)) * blocks + four_v_scale(b, g.slot, blocks)
                                            : (uint64_t)token * blocks + b);
      w0[i] = __ldcs(reinterpret_cast<const uint32_t*>(row + word));
      w1[i] = __ldcs(reinterpret_cast<const uint32_t*>(row + (is_v ? word ^ half * 16 : word + half * 4)));
      s0[i] = scale[0];
      s1[i] = scale[apart];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (here[i]) {
        __stcs(reinterpret_cast<uint4*>(out), four_values(w0[i], s0[i], is_v));
        __stcs(reinterpret_cast<uint4*>(out + a.d / 2), four_values(w1[i], s1[i], is_v));
      }
      out += stride;
    }
  }
}

int row_units4(const PagedArgs& a, bool with_q) { return (2 * a.Hkv + (with_q ? a.H : 0)) * (a.d / 16); }

}  // namespace

// Rows of a thread: one where those blocks are on the SMs at once, else twice as many until they are, up to kMostRows (rows that few threads
// take one after the other wait for each other's angles: one token of each of 128 sequences, appended and read back, 16.3 us with one row,
// 20.9 with two and 26.8 with four).
int thread_rows4(const PagedArgs& a, int units) {
  int n = 1;
  while (n < kMostRows && append_blocks(a, units, n).copies > kResident * kSMs) n *= 2;
  return n;
}

bool append4_fits(const PagedArgs& a, bool with_q) {
  const int units = row_units4(a, with_q);
  return append_blocks(a, units, thread_rows4(a, units)).fit();
}

cudaError_t launch_cache_append4(const CacheAppendArgs& x, void* ks, void* vs, cudaStream_t s) {
  Append4Params p = {};
  static_cast<AppendParams&>(p) = append_params(x);
  p.ks = static_cast<uint8_t*>(ks);
  p.vs = static_cast<uint8_t*>(vs);
  const int units = row_units4(p.a, p.qn != nullptr);
  p.thread_rows = thread_rows4(p.a, units);
  return launch_append(p.rot == 0 ? cache_append4_kernel<kNone> : p.pairs ? cache_append4_kernel<kPairs> : cache_append4_kernel<kHalves>,
                       p, units, s, p.thread_rows);
}

cudaError_t launch_cache_read4(const CacheAppendArgs& x, void* ks, void* vs, cudaStream_t s) {
  Read4Params p = {};
  static_cast<AppendParams&>(p) = append_params(x);
  p.ks = static_cast<const uint8_t*>(ks);
  p.vs = static_cast<const uint8_t*>(vs);
  p.ko = static_cast<__nv_bfloat16*>(const_cast<void*>(x.k));
  p.vo = static_cast<__nv_bfloat16*>(const_cast<void*>(x.v));
  const int units = row_units4(p.a, false);
  p.thread_rows = thread_rows4(p.a, units);
  TraceScope trace("cache_read", s);
  const cudaError_t e = launch_dependent(cache_read4_kernel, dim3(static_cast<unsigned>(append_blocks(p.a, units, p.thread_rows).copies)),
                                         dim3(kThreads), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fox
