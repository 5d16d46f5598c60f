// Pages of the pool: one step's bookkeeping, packing, and copies of pages. C ABI, validation and kernels; the contract is in
// include/fox.h.
//
// step and compact are integers all: what bounds them is latency, a dependent trip to memory or a barrier after the other, so that they take
// few of both. step: one CTA for what hangs together, behind a kernel that copies references and table rows where the new state is
// apart from the old, and one that counts references where there are many (512 sequences on 65536 pages 12 us, in one kernel 61; 8 of a
// search on 2048 pages 8.2). compact: a count of the
// pages in use by blocks of them, then every block knows its pages' ranks, then tables (262144 pages, 1024 sequences 13 us; by one CTA
// 407); a small pool by one CTA (6.4 us).
// copy is bound by memory: each page read once and written once, 16 KB a block (1.28 GB read and written 188 us, 6.8 TB/s; 26 MB 5.2 us),
// or of many small pages 1024 units of 16 bytes, whatever their array (40000 of 2.1 KB: 174 MB in 35 us, 5.0 TB/s).
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/fox.h"
#include "fox_cache.h"
#include "fox_ptx.cuh"

namespace fox {
namespace {

constexpr int kPageThreads = 1024, kCopyThreads = 256;

struct Pool {
  int num_pages, shift, B, stride, prefix_len;  // page_size = 1 << shift
  int32_t* refs;
  int32_t* lens;
  int32_t* table;
  int32_t* prefix;
};

// Tokens of a sequence behind the prefix; a length that its row cannot hold is reported and counts as none.
__device__ __forceinline__ int own_tokens(const Pool& x, int len, uint32_t* err) {
  if (len == 0) return 0;
  const long long cap = (long long)x.stride << x.shift, own = (long long)len - x.prefix_len;
  if (len > 0 && own >= 0 && own <= cap) return static_cast<int>(own);
  atomicOr(err, DEV_ERR_BOUNDS);
  return -1;
}
__device__ __forceinline__ int pages_of(const Pool& x, int own) { return own <= 0 ? 0 : (own - 1 >> x.shift) + 1; }

// Sum over the threads before this one of the block; `all` gets the total. Ends with a barrier.
__device__ __forceinline__ int block_before(int mine, int* scratch, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    scratch[lane] = y;
  }
  __syncthreads();
  *all = scratch[31];
  const int before = x - mine + (warp > 0 ? scratch[warp - 1] : 0);
  __syncthreads();
  return before;
}

struct StepParams {
  Pool in, out;
  const int32_t* parent;
  const int32_t* add;
  int32_t* copies;
  int32_t* list;  // [num_pages] of the workspace: of a shared last page the last sequence that goes on in it; then free pages, the lowest first
  bool begun;     // pages_begin_kernel was launched
  bool counted;   // and pages_refs_kernel
  uint32_t* err;
};

__device__ __forceinline__ int parent_of(const StepParams& p, int b) {
  const int src = p.parent ? p.parent[b] : b;
  if (src >= -1 && src < p.in.B) return src;
  atomicOr(p.err, DEV_ERR_BOUNDS);
  return -1;
}

// What of the old state the new one begins with: references, and a row of the table a block.
__global__ void __launch_bounds__(kCopyThreads) pages_begin_kernel(const StepParams p) {
  const Pool &in = p.in, &out = p.out;
  grid_dep_wait();
  grid_dep_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  if (out.refs != in.refs)
    for (int i = b * kCopyThreads + tid; i < in.num_pages; i += gridDim.x * kCopyThreads) out.refs[i] = in.refs[i];
  if (b >= out.B || out.table == in.table) return;
  const int src = parent_of(p, b);
  if (src < 0) return;
  const int n = pages_of(in, own_tokens(in, in.lens[src], p.err));
  for (int c = tid; c < n; c += kCopyThreads) {
    const int id = in.table[(size_t)src * in.stride + c];
    if (id < 0 || id >= in.num_pages) atomicOr(p.err, DEV_ERR_BOUNDS);
    out.table[(size_t)b * out.stride + c] = id;
  }
}

// References of an old sequence's pages, a block a sequence: by its children less one.
__global__ void __launch_bounds__(kCopyThreads) pages_refs_kernel(const StepParams p) {
  const Pool& in = p.in;
  grid_dep_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  int mine = 0;
  for (int i = tid; i < p.out.B; i += kCopyThreads) mine += p.parent[i] == b;
  const int kids = __syncthreads_count(mine & 1) + 2 * __syncthreads_count(mine >> 1 & 1) + 4 * __syncthreads_count(mine >> 2 & 1) +
                   8 * __syncthreads_count(mine >> 3);  // at most 8 of a thread
  static_assert(kMaxSeqs <= 8 * kCopyThreads, "");
  const int n = kids == 1 ? 0 : pages_of(in, own_tokens(in, in.lens[b], p.err));
  grid_dep_wait();
#pragma unroll 4
  for (int c = tid; c < n; c += kCopyThreads) {
    const int id = in.table[(size_t)b * in.stride + c];
    if (id >= 0 && id < in.num_pages)
      atomicAdd(p.out.refs + id, kids - 1);
    else
      atomicOr(p.err, DEV_ERR_BOUNDS);
  }
}

__global__ void __launch_bounds__(kPageThreads) pages_step_kernel(const StepParams p) {
  constexpr int kEach = kMaxSeqs / kPageThreads, kLoad = 16, kNoPages = 0x7FFFFFFF;
  __shared__ int kids[kMaxSeqs];       // children of the old sequences; then whether a new one's last page is copied
  __shared__ int upto[kMaxSeqs];       // pages wanted by the new sequences up to each; before, pages of the old ones
  __shared__ int first_new[kMaxSeqs];  // a new sequence's entry for its first wanted page; kNoPages: it gets none. Before, old
                                       // sequences whose references change
  __shared__ int scratch[32], changed;
  const Pool &in = p.in, &out = p.out;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = tid; b < in.B; b += kPageThreads) kids[b] = 0;
  if (tid == 0) changed = 0;
  // Behind pages_begin_kernel, which let this one start once all before it were through, what the call was given may be read at once.
  if (!p.begun) grid_dep_wait();
  grid_dep_trigger();
  __syncthreads();
  // Sequence b is thread b's, and b + 1024 too.
  int len[kEach], n0[kEach], n1[kEach], add[kEach], last[kEach], old_len[kEach];
  bool grows[kEach], part[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid + i * kPageThreads;
    old_len[i] = p.parent && !p.counted && b < in.B ? in.lens[b] : 0;
    last[i] = -1;
    len[i] = n0[i] = n1[i] = add[i] = 0;
    grows[i] = part[i] = false;
    if (b >= out.B) continue;
    const int src = parent_of(p, b);
    add[i] = p.add[b];
    len[i] = src >= 0 ? in.lens[src] : 0;
    if (src >= 0) atomicAdd(&kids[src], 1);
    int own = own_tokens(in, len[i], p.err);
    if (own < 0) len[i] = own = 0;
    if (add[i] < 0) {
      atomicOr(p.err, DEV_ERR_BOUNDS);
      add[i] = 0;
    }
    n0[i] = pages_of(in, own);
    const long long cap = (long long)in.stride << in.shift;
    grows[i] = add[i] > 0 && own + (long long)add[i] <= cap;
    if (add[i] > 0 && !grows[i]) atomicOr(p.err, DEV_ERR_BOUNDS);
    n1[i] = grows[i] ? pages_of(in, own + add[i]) : n0[i];
    if (grows[i] && (own & ((1 << in.shift) - 1)) != 0) {
      last[i] = in.table[(size_t)src * in.stride + n0[i] - 1];
      part[i] = last[i] >= 0 && last[i] < in.num_pages;
      if (part[i])
        p.list[last[i]] = -1;
      else
        atomicOr(p.err, DEV_ERR_BOUNDS);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid + i * kPageThreads;
    if (old_len[i] == 0 || kids[b] == 1) continue;
    upto[b] = pages_of(in, own_tokens(in, old_len[i], p.err));
    if (upto[b] > 0) first_new[atomicAdd(&changed, 1)] = b;
  }
  if (p.begun) grid_dep_wait();
  __threadfence();
  __syncthreads();
  // References: every entry of an old sequence by its children less one.
  for (int x = warp; x < changed; x += kPageThreads / 32) {
    const int b = first_new[x], d = kids[b] - 1, n = upto[b];
#pragma unroll 4
    for (int c = lane; c < n; c += 32) {
      const int id = in.table[(size_t)b * in.stride + c];
      if (id >= 0 && id < in.num_pages)
        atomicAdd(out.refs + id, d);
      else
        atomicOr(p.err, DEV_ERR_BOUNDS);
    }
  }
  // A partly filled last page is copied by all that go on in it, unless they are all that hold it: the last of them then keeps it.
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (part[i]) {
      atomicSub(out.refs + last[i], 1);
      atomicMax(p.list + last[i], tid + i * kPageThreads);
    }
  __threadfence();
  __syncthreads();
  bool copied[kEach];
  int need[kEach], start[kEach], total = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    copied[i] = part[i] && (__ldcg(out.refs + last[i]) > 0 || __ldcg(p.list + last[i]) != tid + i * kPageThreads);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (part[i] && !copied[i]) atomicAdd(out.refs + last[i], 1);
    need[i] = grows[i] ? n1[i] - n0[i] + copied[i] : 0;
    int all;
    start[i] = total + block_before(need[i], scratch, &all);
    total += all;
    upto[tid + i * kPageThreads] = start[i] + need[i];
  }
  if (total > 0) {
    __threadfence();
    __syncthreads();
  }
  // Free pages, as many as are wanted, into the list.
  int found = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < in.num_pages && found < total; i0 += kPageThreads * kLoad) {
    const int i = i0 + tid * kLoad;
    uint32_t mask = 0;
    if (i + kLoad <= in.num_pages && (reinterpret_cast<uintptr_t>(out.refs) & 15) == 0) {
#pragma unroll
      for (int k = 0; k < kLoad; k += 4) {
        const int4 r = __ldcg(reinterpret_cast<const int4*>(out.refs + i + k));
        mask |= (uint32_t(r.x <= 0) | uint32_t(r.y <= 0) << 1 | uint32_t(r.z <= 0) << 2 | uint32_t(r.w <= 0) << 3) << k;
      }
    } else {
      for (int k = 0; k < kLoad; ++k)
        if (i + k < in.num_pages) mask |= uint32_t(__ldcg(out.refs + i + k) <= 0) << k;
    }
    int all, at = found + block_before(__popc(mask), scratch, &all);
    for (; mask && at < total; mask &= mask - 1) p.list[at++] = i + __ffs(mask) - 1;
    found += all;
  }
  // Lengths, and who gets what.
  bool short_of = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid + i * kPageThreads;
    if (b >= out.B) continue;
    const bool served = grows[i] && (need[i] == 0 || start[i] + need[i] <= found), copies = served && copied[i];
    short_of |= grows[i] && !served;
    out.lens[b] = served ? (len[i] > 0 ? len[i] : in.prefix_len) + add[i] : len[i];
    p.copies[2 * b] = copies ? last[i] : -1;
    if (!copies) p.copies[2 * b + 1] = -1;
    if (copied[i] && !served) atomicAdd(out.refs + last[i], 1);  // it still holds it
    kids[b] = copies;
    first_new[b] = served ? n0[i] - copies : kNoPages;
  }
  if (short_of) atomicOr(p.err, DEV_ERR_BOUNDS);
  __syncthreads();
  for (int rank = tid; rank < min(found, total); rank += kPageThreads) {
    int lo = -1, hi = out.B - 1;  // upto[lo] <= rank < upto[hi]
    while (hi - lo > 1) {
      const int mid = lo + hi >> 1;
      if (upto[mid] <= rank)
        lo = mid;
      else
        hi = mid;
    }
    const int k = rank - (hi > 0 ? upto[hi - 1] : 0), to = first_new[hi];
    if (to == kNoPages) continue;
    const int page = p.list[rank];
    out.refs[page] = 1;
    out.table[(size_t)hi * out.stride + to + k] = page;
    if (k == 0 && kids[hi]) p.copies[2 * hi + 1] = page;
  }
}

struct CompactParams {
  Pool in, out;
  int32_t* map;
  int2* moves;
  int max_moves;
  int32_t* used;
  int32_t* counts;  // of the workspace: pages in use of each block of kCountPages
  uint32_t* err;
};

// Renames a table's entries; a page's place in map may stand there as -1 - its move.
__device__ __forceinline__ int renamed(const CompactParams& p, int id) {
  if (id < 0 || id >= p.in.num_pages) {
    atomicOr(p.err, DEV_ERR_BOUNDS);
    return id;
  }
  const int to = __ldcg(p.map + id);
  return to >= 0 ? to : __ldcg(&p.moves[-1 - to].y);
}
__device__ __forceinline__ void rename_row(const CompactParams& p, int b, int first, int step) {
  const Pool& in = p.in;
  const int n = pages_of(in, own_tokens(in, in.lens[b], p.err));
  for (int c = first; c < n; c += step) p.out.table[(size_t)b * in.stride + c] = renamed(p, in.table[(size_t)b * in.stride + c]);
}
__device__ __forceinline__ void move_refs(const CompactParams& p, int r) {
  const int2 x = p.moves[r];
  p.map[x.x] = x.y;
  p.out.refs[x.y] = p.in.refs[x.x];  // in place: nobody else has either
  p.out.refs[x.x] = 0;
}

constexpr int kCountPages = 4096, kCountEach = kCountPages / kPageThreads;

// Pages in use among four of a thread's, as bits.
__device__ __forceinline__ uint32_t in_use(const Pool& x, int i) {
  uint32_t mask = 0;
#pragma unroll
  for (int k = 0; k < kCountEach; ++k)
    if (i + k < x.num_pages) mask |= uint32_t(x.refs[i + k] > 0) << k;
  return mask;
}

// The moves of a thread's pages i .. i + 3, `mask` of them in use, `rank` pages in use before them: of U in all, n that stand behind U,
// m of which move. map gets a moving page's move as -1 - r where the moves are another block's too (`later`).
__device__ __forceinline__ void place_pages(const CompactParams& p, int i, uint32_t mask, int rank, int U, int m, bool later) {
#pragma unroll
  for (int k = 0; k < kCountEach; ++k) {
    const int page = i + k;
    if (page >= p.in.num_pages) break;
    const bool used = mask >> k & 1;
    int to = page;
    if (used && page >= U) {
      const int r = U - 1 - rank;  // pages in use behind this one
      if (r < m) {
        p.moves[r].x = page;
        if (later) to = -1 - r;
      }
      if (r == m) p.used[1] = page + 1;
    } else if (!used && page < U && page - rank < m) {
      p.moves[page - rank].y = page;
    }
    p.map[page] = to;
    if (p.out.refs != p.in.refs) p.out.refs[page] = p.in.refs[page];
    rank += used;
  }
}

__global__ void __launch_bounds__(kPageThreads) pages_count_kernel(const CompactParams p) {
  __shared__ int scratch[32];
  grid_dep_wait();
  grid_dep_trigger();
  int all;
  block_before(__popc(in_use(p.in, (blockIdx.x * kPageThreads + threadIdx.x) * kCountEach)), scratch, &all);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = all;
}

// Each block finds the moves of its pages: U and the counts before it from all counts, and how many pages move from those before U.
__global__ void __launch_bounds__(kPageThreads) pages_place_kernel(const CompactParams p) {
  __shared__ int scratch[32];
  const Pool& in = p.in;
  const int tid = threadIdx.x, blocks = gridDim.x, mine = blockIdx.x;
  const int i = (mine * kPageThreads + tid) * kCountEach;
  grid_dep_wait();
  grid_dep_trigger();
  const uint32_t mask = in_use(in, i);
  int sum = 0, before = 0;
  for (int b = tid; b < blocks; b += kPageThreads) {
    const int n = __ldcg(p.counts + b);
    sum += n;
    before += b < mine ? n : 0;
  }
  int U, here, all;
  block_before(sum, scratch, &U);
  block_before(before, scratch, &before);
  const int rank = before + block_before(__popc(mask), scratch, &here);  // pages in use before this thread's
  const int edge = U / kCountPages;                                      // the block that page U is in
  int front = 0;
  for (int b = tid; b < min(edge, blocks); b += kPageThreads) front += __ldcg(p.counts + b);
  const int at = edge * kCountPages + tid * kCountEach;
  const uint32_t those = in_use(in, at);
#pragma unroll
  for (int k = 0; k < kCountEach; ++k) front += at + k < U && (those >> k & 1);
  block_before(front, scratch, &all);
  const int n = U - all, m = min(n, p.max_moves);  // free places in front, and pages behind that move there
  place_pages(p, i, mask, rank, U, m, true);
  for (int r = m + mine * kPageThreads + tid; r < p.max_moves; r += blocks * kPageThreads) p.moves[r] = make_int2(-1, -1);
  if (mine == 0 && tid == 0) {
    p.used[0] = U;
    if (m == n) p.used[1] = U;
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_rename_kernel(const CompactParams p) {
  const Pool& in = p.in;
  grid_dep_wait();
  grid_dep_trigger();
  const int tid = threadIdx.x, b = blockIdx.x;
  if (b < in.B) {
    rename_row(p, b, tid, kCopyThreads);
  } else {
    const int first = (b - in.B) * kCopyThreads + tid, step = (gridDim.x - in.B) * kCopyThreads;
    for (int c = first; c < pages_of(in, in.prefix_len); c += step) p.out.prefix[c] = renamed(p, in.prefix[c]);
    for (int r = first; r < p.max_moves; r += step)
      if (p.moves[r].x >= 0) move_refs(p, r);
  }
}

// A small pool by one CTA: the same in one launch.
__global__ void __launch_bounds__(kPageThreads) pages_compact_kernel(const CompactParams p) {
  __shared__ int scratch[32];
  grid_dep_wait();
  grid_dep_trigger();
  const Pool& in = p.in;
  const int tid = threadIdx.x, i = tid * kCountEach;
  const uint32_t mask = in_use(in, i);
  int U, all, front = 0;
  const int rank = block_before(__popc(mask), scratch, &U);
#pragma unroll
  for (int k = 0; k < kCountEach; ++k) front += i + k < U && (mask >> k & 1);
  block_before(front, scratch, &all);
  const int n = U - all, m = min(n, p.max_moves);
  place_pages(p, i, mask, rank, U, m, false);
  for (int r = m + tid; r < p.max_moves; r += kPageThreads) p.moves[r] = make_int2(-1, -1);
  if (tid == 0) {
    p.used[0] = U;
    if (m == n) p.used[1] = U;
  }
  __syncthreads();
  for (int r = tid; r < m; r += kPageThreads) move_refs(p, r);
  __syncthreads();
  for (int b = tid >> 5; b < in.B; b += kPageThreads / 32) rename_row(p, b, tid & 31, 32);
  for (int c = tid; c < pages_of(in, in.prefix_len); c += kPageThreads) p.out.prefix[c] = renamed(p, in.prefix[c]);
}

// ---- copies ----
constexpr int kCopyLoads = 4, kArrays = PageArrays::kMost;
constexpr int kCopyBytes = kCopyThreads * kCopyLoads * 16;  // of a block

struct CopyParams {
  char* at[kArrays];
  long long bytes[kArrays];  // of a page: a multiple of 16, of gbase of 8
  int chunks[kArrays + 1];   // blocks of a page before the array
  int arrays, num_pages;
  const int2* pairs;
  uint32_t* err;
};

template <typename T>
__device__ __forceinline__ void copy_chunk(char* to, const char* from, long long left) {
  T x[kCopyLoads];
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    const long long at = (long long)(i * kCopyThreads + threadIdx.x) * sizeof(T);
    if (at < left) x[i] = __ldcs(reinterpret_cast<const T*>(from + at));
  }
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    const long long at = (long long)(i * kCopyThreads + threadIdx.x) * sizeof(T);
    if (at < left) __stcs(reinterpret_cast<T*>(to + at), x[i]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyParams p) {
  grid_dep_wait();
  grid_dep_trigger();
  const int per = p.chunks[p.arrays], pair = blockIdx.x / per, chunk = blockIdx.x - pair * per;
  const int2 x = p.pairs[pair];
  if (x.x < 0 || x.x >= p.num_pages || x.y < 0 || x.y >= p.num_pages) {
    if ((x.x != -1 || x.y != -1) && threadIdx.x == 0) atomicOr(p.err, DEV_ERR_BOUNDS);
    return;
  }
  int k = 0;
  while (chunk >= p.chunks[k + 1]) ++k;
  const long long bytes = p.bytes[k];
  if (bytes % 16 == 0) {
    const long long at = (long long)(chunk - p.chunks[k]) * kCopyBytes;
    copy_chunk<uint4>(p.at[k] + x.y * bytes + at, p.at[k] + x.x * bytes + at, bytes - at);
  } else {
    const long long at = (long long)(chunk - p.chunks[k]) * (kCopyBytes / 2);
    copy_chunk<uint2>(p.at[k] + x.y * bytes + at, p.at[k] + x.x * bytes + at, bytes - at);
  }
}

// Small pages: the pairs' units of 8 or 16 bytes of all arrays in one row, 1024 a block, so that no block has a few of one array alone.
struct UnitParams {
  char* at[kArrays];
  uint32_t bytes[kArrays];      // of a page
  uint32_t first[kArrays + 1];  // units of a page before the array
  uint32_t wide;                // bit k: array k in units of 16 bytes, else 8
  int arrays, num_pages, n;
  const int2* pairs;
  uint32_t* err;
};
__global__ void __launch_bounds__(kCopyThreads) pages_copy_units_kernel(const UnitParams p) {
  grid_dep_wait();
  grid_dep_trigger();
  const uint32_t per = p.first[p.arrays];
  const uint64_t begin = static_cast<uint64_t>(blockIdx.x) * (kCopyThreads * kCopyLoads);
  const int pair0 = static_cast<int>(begin / per);
  const uint32_t rest = static_cast<uint32_t>(begin - static_cast<uint64_t>(pair0) * per);
  uint4 x[kCopyLoads];
  char* to[kCopyLoads];
  bool wide[kCopyLoads];
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    const uint32_t at = rest + i * kCopyThreads + threadIdx.x;
    const int pair = pair0 + static_cast<int>(at / per);
    const uint32_t unit = at % per;
    to[i] = nullptr;
    if (pair >= p.n) continue;
    const int2 y = p.pairs[pair];
    if (y.x < 0 || y.x >= p.num_pages || y.y < 0 || y.y >= p.num_pages) {
      if ((y.x != -1 || y.y != -1) && unit == 0) atomicOr(p.err, DEV_ERR_BOUNDS);
      continue;
    }
    char* base = p.at[0];
    uint32_t bytes = p.bytes[0], first = 0;
    int k = 0;
#pragma unroll
    for (int j = 1; j < kArrays; ++j)
      if (j < p.arrays && unit >= p.first[j]) {
        base = p.at[j];
        bytes = p.bytes[j];
        first = p.first[j];
        k = j;
      }
    wide[i] = p.wide >> k & 1;
    const uint32_t offset = (unit - first) * (wide[i] ? 16 : 8);
    const char* from = base + static_cast<uint64_t>(y.x) * bytes + offset;
    to[i] = base + static_cast<uint64_t>(y.y) * bytes + offset;
    if (wide[i]) {
      x[i] = __ldcs(reinterpret_cast<const uint4*>(from));
    } else {
      const uint2 z = __ldcs(reinterpret_cast<const uint2*>(from));
      x[i] = make_uint4(z.x, z.y, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    if (!to[i]) continue;
    if (wide[i])
      __stcs(reinterpret_cast<uint4*>(to[i]), x[i]);
    else
      __stcs(reinterpret_cast<uint2*>(to[i]), make_uint2(x[i].x, x[i].y));
  }
}

// ---- host ----
bool ints(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
  uintptr_t at;
  size_t bytes;
  bool over(const Range& o) const { return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes; }
};
Range range(const void* p, size_t n, size_t element = 4) { return {reinterpret_cast<uintptr_t>(p), p ? n * element : 0}; }

fox_status check_pool(const fox_pages* x) {
  if (!x || x->num_pages < 1 || x->B < 0 || x->table_stride < 1 || x->prefix_len < 0) return FOX_ERR_INVALID_ARG;
  if (x->page_size != 16 && x->page_size != 32 && x->page_size != 64 && x->page_size != 128) return FOX_ERR_UNSUPPORTED;
  if (x->num_pages > 1 << 24 || x->B > kMaxSeqs) return FOX_ERR_UNSUPPORTED;
  if ((long long)x->prefix_len + (long long)x->table_stride * x->page_size > 0x7fffffffLL) return FOX_ERR_UNSUPPORTED;
  // what all sequences together may want is an int
  if ((long long)x->B * (x->table_stride + 1LL) > 1LL << 30) return FOX_ERR_UNSUPPORTED;
  return FOX_OK;
}
fox_status check_two(const fox_pages* in, const fox_pages* out) {
  fox_status st = check_pool(in);
  if (st == FOX_OK) st = check_pool(out);
  if (st != FOX_OK) return st;
  return in->num_pages == out->num_pages && in->page_size == out->page_size && in->table_stride == out->table_stride &&
                 in->prefix_len == out->prefix_len
             ? FOX_OK
             : FOX_ERR_INVALID_ARG;
}
Pool pool_of(const fox_pages* x) {
  const int shift = x->page_size == 16 ? 4 : x->page_size == 32 ? 5 : x->page_size == 64 ? 6 : 7;
  return {x->num_pages, shift, x->B, x->table_stride, x->prefix_len, x->refs, x->lens, x->table, x->prefix_table};
}
size_t prefix_pages(const fox_pages* x) { return ((size_t)x->prefix_len + x->page_size - 1) / x->page_size; }

// Whether outputs lie apart from each other and from what is read; an output may be the input of the same number.
template <int kOut, int kIn>
bool apart(const Range (&out)[kOut], const Range (&in)[kIn]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < kIn; ++j)
      if (out[i].over(in[j]) && !(i == j && out[i].at == in[j].at)) return false;
    for (int j = 0; j < i; ++j)
      if (out[i].over(out[j])) return false;
  }
  return true;
}
fox_status check_header(void* ws, size_t bytes, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && bytes >= need ? FOX_OK : FOX_ERR_WORKSPACE;
}
// The header, and an int a page (step's list; compact's counts are fewer).
size_t pages_workspace(const fox_pages* x) { return kCacheHeaderBytes + align_up(sizeof(int32_t) * (size_t)x->num_pages, 256); }
int32_t* behind_header(void* ws) { return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kCacheHeaderBytes); }
// References of large tables by a kernel of their own: one SM's atomics take a nanosecond each. By it and by the step's CTA: 8 sequences of 64
// entries 9.9 and 8.2 us, 64 of a search of 64 10.5 and 10.8, 256 10.7 and 15.7, 1024 of 94 14.8 and 46; 512 of 129, most of which go on,
// 12.0 and 15.8.
bool counts_apart(const fox_pages* in, const int32_t* parent) { return parent && (long long)in->B * in->table_stride > 2048; }
// One CTA has a pool of 4096 pages in its registers, and renames 32 pieces of 32 entries at a time, half a microsecond or more each. By one
// CTA and by three kernels: 16 sequences of 32 entries (512 pages) 3.9 and 6.4 us, 64 of 64 (4096 pages: 4 rounds) 9.4 and 10.5, 128 of 512
// (64 rounds) 42 and 11, 2048 of 32 63 and 12.
bool compacts_alone(const fox_pages* x) {
  return x->num_pages <= kCountPages && x->B * (long long)ceil_div(x->table_stride, 32) <= 4 * kPageThreads / 32;
}

CopyParams copy_params(const PageArrays& x) {
  CopyParams p = {};
  p.arrays = x.n;
  for (int k = 0; k < x.n; ++k) {
    const long long piece = x.bytes[k] % 16 == 0 ? kCopyBytes : kCopyBytes / 2;
    p.at[k] = x.at[k];
    p.bytes[k] = x.bytes[k];
    p.chunks[k + 1] = p.chunks[k] + static_cast<int>((x.bytes[k] + piece - 1) / piece);
  }
  return p;
}

// Pages below 24 KB by units, where there are more blocks of chunks than the SMs hold at once. By units and by chunks: 40000 pages of 2.1 KB
// 35 and 283 us, 30000 of 5.1 KB 58 and 153, 20000 of 12.6 KB 92 and 143, 10000 of 21 KB 78.1 and 79.4, 6000 of 42 KB 93 and 78,
// 8000 of 84 KB 240 and 202; 48 of 2.1 KB 3.3 and 2.2.
bool copies_units(const PageArrays& x, int n) {
  long long bytes = 0;
  for (int k = 0; k < x.n; ++k) bytes += x.bytes[k];
  return bytes < 24576 && (long long)n * copy_params(x).chunks[x.n] > 2048 / kCopyThreads * kSMs;
}
UnitParams unit_params(const PageArrays& x) {
  UnitParams p = {};
  p.arrays = x.n;
  for (int k = 0; k < x.n; ++k) {
    const bool wide = x.bytes[k] % 16 == 0;
    p.at[k] = x.at[k];
    p.bytes[k] = static_cast<uint32_t>(x.bytes[k]);
    p.wide |= static_cast<uint32_t>(wide) << k;
    p.first[k + 1] = p.first[k] + p.bytes[k] / (wide ? 16 : 8);
  }
  return p;
}
long long copy_blocks(const PageArrays& x, int n) {
  constexpr int kUnits = kCopyThreads * kCopyLoads;
  if (copies_units(x, n)) return ((long long)n * unit_params(x).first[x.n] + kUnits - 1) / kUnits;
  return (long long)n * copy_params(x).chunks[x.n];
}

}  // namespace

bool pages_copy_fits(const PageArrays& x, int n) { return copy_blocks(x, n) <= 0x7fffffffLL; }

cudaError_t launch_pages_copy(const PageArrays& x, int num_pages, const int32_t* pairs, int n, uint32_t* err, cudaStream_t s) {
  const dim3 blocks(static_cast<unsigned>(copy_blocks(x, n)));
  TraceScope trace("pages_copy", s);
  cudaError_t e;
  if (copies_units(x, n)) {
    UnitParams p = unit_params(x);
    p.num_pages = num_pages;
    p.n = n;
    p.pairs = reinterpret_cast<const int2*>(pairs);
    p.err = err;
    e = launch_dependent(pages_copy_units_kernel, blocks, dim3(kCopyThreads), 0, s, p);
  } else {
    CopyParams p = copy_params(x);
    p.num_pages = num_pages;
    p.pairs = reinterpret_cast<const int2*>(pairs);
    p.err = err;
    e = launch_dependent(pages_copy_kernel, blocks, dim3(kCopyThreads), 0, s, p);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fox

using namespace fox;

extern "C" {

size_t fox_pages_workspace_bytes(const fox_pages* in, const fox_pages* out) {
  return check_two(in, out) == FOX_OK ? pages_workspace(in) : 0;
}

fox_status fox_pages_step(const fox_pages* in, const fox_pages* out, const int32_t* parent, const int32_t* add,
                          int32_t* copies, void* workspace, size_t workspace_bytes, void* stream) {
  fox_status st = check_two(in, out);
  if (st != FOX_OK) return st;
  if (!parent && in->B != out->B) return FOX_ERR_INVALID_ARG;
  if (!ints(in->refs) || !ints(out->refs)) return FOX_ERR_INVALID_ARG;
  if (in->B > 0 && (!ints(in->lens) || !ints(in->table))) return FOX_ERR_INVALID_ARG;
  if (out->B > 0 && (!ints(out->lens) || !ints(out->table) || !ints(add) || !ints(copies))) return FOX_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(parent) & 3u) return FOX_ERR_INVALID_ARG;
  const size_t Bi = in->B, Bo = out->B, E = in->table_stride, N = in->num_pages;
  const Range outs[] = {range(out->refs, N), range(out->lens, Bo), range(out->table, Bo * E), range(copies, 2 * Bo)};
  const Range ins[] = {range(in->refs, N), range(in->lens, Bi),  range(in->table, Bi * E), range(nullptr, 0),
                       range(add, Bo),     range(parent, Bo)};
  if (!apart(outs, ins)) return FOX_ERR_INVALID_ARG;
  if (parent && (out->refs == in->refs || (Bi && Bo && (out->lens == in->lens || out->table == in->table))))
    return FOX_ERR_INVALID_ARG;
  st = check_header(workspace, workspace_bytes, pages_workspace(in));
  if (st != FOX_OK) return st;
  const StepParams p = {pool_of(in), pool_of(out), parent, add, copies, behind_header(workspace),
                        in->refs != out->refs || in->table != out->table, counts_apart(in, parent), static_cast<uint32_t*>(workspace)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (p.begun) {
    TraceScope trace("pages_begin", s);
    const int blocks = ceil_div(in->num_pages, kCopyThreads), wide = blocks < kSMs ? blocks : kSMs;
    e = launch_dependent(pages_begin_kernel, dim3(out->B > wide ? out->B : wide), dim3(kCopyThreads), 0, s, p);
  }
  if (e == cudaSuccess && p.counted) {
    TraceScope trace("pages_refs", s);
    e = launch_dependent(pages_refs_kernel, dim3(in->B), dim3(kCopyThreads), 0, s, p);
  }
  if (e == cudaSuccess) {
    TraceScope trace("pages_step", s);
    e = launch_dependent(pages_step_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FOX_OK : FOX_ERR_CUDA;
}

fox_status fox_pages_compact(const fox_pages* in, const fox_pages* out, int32_t* map, int32_t* moves, int max_moves,
                             int32_t* used, void* workspace, size_t workspace_bytes, void* stream) {
  fox_status st = check_two(in, out);
  if (st != FOX_OK) return st;
  if (in->B != out->B || max_moves < 0) return FOX_ERR_INVALID_ARG;
  if (!ints(in->refs) || !ints(out->refs) || !ints(map) || !ints(used)) return FOX_ERR_INVALID_ARG;
  if (max_moves > 0 && (!moves || (reinterpret_cast<uintptr_t>(moves) & 7u))) return FOX_ERR_INVALID_ARG;
  if (in->B > 0 && (!ints(in->lens) || !ints(in->table) || !ints(out->table))) return FOX_ERR_INVALID_ARG;
  if (in->prefix_len > 0 && (!ints(in->prefix_table) || !ints(out->prefix_table))) return FOX_ERR_INVALID_ARG;
  const size_t B = in->B, E = in->table_stride, N = in->num_pages, P = prefix_pages(in);
  const Range outs[] = {range(out->refs, N), range(out->table, B * E), range(out->prefix_table, P),
                        range(map, N),       range(moves, 2 * (size_t)max_moves), range(used, 2)};
  const Range ins[] = {range(in->refs, N), range(in->table, B * E), range(in->prefix_table, P),
                       range(nullptr, 0),  range(nullptr, 0),       range(nullptr, 0), range(in->lens, B)};
  if (!apart(outs, ins)) return FOX_ERR_INVALID_ARG;
  st = check_header(workspace, workspace_bytes, pages_workspace(in));
  if (st != FOX_OK) return st;
  const CompactParams p = {pool_of(in), pool_of(out), map, reinterpret_cast<int2*>(moves), max_moves, used, behind_header(workspace),
                           static_cast<uint32_t*>(workspace)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (compacts_alone(in)) {
    TraceScope trace("pages_compact", s);
    e = launch_dependent(pages_compact_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  } else {
    const int blocks = ceil_div(in->num_pages, kCountPages);
    {
      TraceScope trace("pages_count", s);
      e = launch_dependent(pages_count_kernel, dim3(blocks), dim3(kPageThreads), 0, s, p);
    }
    if (e == cudaSuccess) {
      TraceScope trace("pages_place", s);
      e = launch_dependent(pages_place_kernel, dim3(blocks), dim3(kPageThreads), 0, s, p);
    }
    if (e == cudaSuccess) {
      TraceScope trace("pages_rename", s);
      const int work = max_moves > 0 ? ceil_div(max_moves, 4 * kCopyThreads) : 1;
      e = launch_dependent(pages_rename_kernel, dim3(in->B + (work < kSMs ? work : kSMs)), dim3(kCopyThreads), 0, s, p);
    }
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FOX_OK : FOX_ERR_CUDA;
}

}  // extern "C"
