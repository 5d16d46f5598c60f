// What the decode kernels and their merge share: the parameter block, the work line and the layout
// of the partial results.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fox_internal.h"
#include "fox_paged.h"
#include "fox_ptx.cuh"

namespace fox {

// Work on the shared prefix (fox_prefix.cu).
struct PrefixPlan {
  int hp, head_chunks;  // query heads of a row tile; such chunks of a key head's group
  int tpt;              // tokens of a row tile: its row r is token r / hp, head r % hp
  int row_tiles;        // of one key head: token blocks x head chunks, the chunks of a block side by side
  int items;            // of one key head: pairs of row tiles, or the only row tile
  int kap_tiles;        // gate terms of a stage: one set, or one a row tile
  int key_tiles;        // 0: no shared prefix
  int workers;
  float2* ml;           // [(worker + item) * 2 + stream][128] maximum (against c_last) and sum
  float* po;            // [(worker + item) * 2 + stream][128][d]
};

struct DecodeParams {
  PagedArgs a;
  const void* q;
  long long q_stride;  // elements from one row to the next
  float scale2;        // scale * log2 e
  int bias_from_j;
  int walk_prefix;     // the items walk the prefix's keys themselves (nothing shares it out)
  void* o;
  float* lse;
  // Own items
  int Rt, Rs, RTmax;   // rows of a row tile; rows kept of a slot; most row tiles of a sequence
  int Gp;              // rows of a token (padded_group)
  int workers;
  long long* cum;      // [B + 1] units of one key head before each sequence
  float2* ml;          // [slots][Rs] row maximum (log2 units) and sum of a partial result
  float* po;           // [slots][Rs][d] its weighted sum of V
  PrefixPlan pre;
};

// Unit offsets of the sequences into cum[0 .. B] (shared memory), by the whole block.
// `scratch` holds one value a warp. Ends with a block barrier.
__device__ __forceinline__ void scan_units(const DecodeParams& p, long long* cum, long long* scratch) {
  const PagedArgs& a = p.a;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = ceil_div(a.B, nt), b0 = tid * each, b1 = min(a.B, b0 + each);
  long long mine = 0;
  bool any_bad = false;
  for (int b = b0; b < b1; ++b) {
    bool bad;
    const SeqInfo s = seq_info(a, b, &bad);
    any_bad |= bad;
    const long long u = seq_units(a, s, p.Rt, p.Gp, p.walk_prefix);
    cum[b] = u;
    mine += u;
  }
  if (any_bad && blockIdx.x == 0 && a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  long long before = x - mine;
  for (int w = 0; w < warp; ++w) before += scratch[w];
  for (int b = b0; b < b1; ++b) {
    const long long u = cum[b];
    cum[b] = before;
    before += u;
  }
  if (b0 < a.B && b1 == a.B) cum[a.B] = before;
  __syncthreads();
}

// The sequence whose units hold unit u of a key head (cum[b] <= u < cum[b + 1]).
__device__ __forceinline__ int find_seq(const long long* cum, int B, long long u) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Cumulative log gate of (page, slot), head h (natural log).
__device__ __forceinline__ double gate_sum(const PagedArgs& a, int page, int slot, int h) {
  const float2 base = *reinterpret_cast<const float2*>(a.gbase + gbase_offset(a, page, h));
  return static_cast<double>(base.x) + base.y + a.g[g_offset(a, page, h, slot)];
}

// Cumulative log gate of own token p of sequence b (natural log), 0 with a report where the table is bad.
__device__ __forceinline__ double gate_at(const PagedArgs& a, int b, int p, int h) {
  const int page = own_page(a, b, p);
  if (page < 0) {
    if (a.err) atomicOr(a.err, DEV_ERR_BOUNDS);
    return 0.0;
  }
  return gate_sum(a, page, p % a.page_size, h);
}

template <typename T>
__device__ __forceinline__ void put_out(T* dst, const float* f, int n);
template <>
__device__ __forceinline__ void put_out<float>(float* dst, const float* f, int n) {
  for (int i = 0; i < n; i += 2) *reinterpret_cast<float2*>(dst + i) = make_float2(f[i], f[i + 1]);
}
template <>
__device__ __forceinline__ void put_out<__nv_bfloat16>(__nv_bfloat16* dst, const float* f, int n) {
  for (int i = 0; i < n; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(f[i], f[i + 1]);
}

// The bf16 kernel on the tensor cores (fox_decode_mma.cu): its row tile for `rows` rows a sequence
// and key head, its workers, its launch.
int decode_mma_rows(int rows);
int decode_mma_workers(int d);
cudaError_t launch_decode_mma(const DecodeParams& p, cudaStream_t s);
PrefixPlan prefix_plan(const PagedArgs& a);
cudaError_t launch_prefix(const DecodeParams& p, cudaStream_t s);

}  // namespace fox
