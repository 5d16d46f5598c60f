// Pages of the pool: one step's bookkeeping, packing, and copies of pages. C ABI, validation and kernels; the contract is in
// include/fox.h.
//
// step and compact are integers all: what bounds them is latency. One CTA does each: references, places by prefix sums over the sequences
// and over the pages, table entries.
// copy is bound by memory: each page read once and written once, 16 KB a block.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/fox.h"
#include "fox_cache.h"
#include "fox_ptx.cuh"

namespace fox {
namespace {

constexpr int kPageThreads = 1024;

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
  uint32_t* err;
};

// What a new sequence begins with and asks for.
struct Want {
  int src, len, n0, n1, last;  // parent (-1: none), its tokens, pages held and needed; page of its last token
};

__global__ void __launch_bounds__(kPageThreads) pages_step_kernel(const StepParams p) {
  constexpr int kEach = kMaxSeqs / kPageThreads;
  __shared__ int kids[kMaxSeqs];   // children of the old sequences; then the pages that stand to be copied
  __shared__ int upto[kMaxSeqs];   // pages wanted by the new sequences up to each
  __shared__ int scratch[32];
  grid_dep_wait();
  grid_dep_trigger();
  const Pool &in = p.in, &out = p.out;
  const int tid = threadIdx.x;
  for (int b = tid; b < in.B; b += kPageThreads) kids[b] = 0;
  if (out.refs != in.refs)
    for (int i = tid; i < in.num_pages; i += kPageThreads) out.refs[i] = in.refs[i];
  __syncthreads();
  Want w[kEach];
  bool grows[kEach], part[kEach];
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    w[i] = {-1, 0, 0, 0, -1};
    grows[i] = part[i] = false;
    if (b >= out.B) continue;
    int src = p.parent ? p.parent[b] : b;
    if (src < -1 || src >= in.B) {
      atomicOr(p.err, DEV_ERR_BOUNDS);
      src = -1;
    }
    int len = src >= 0 ? in.lens[src] : 0, own = own_tokens(in, len, p.err);
    if (src >= 0) atomicAdd(&kids[src], 1);
    if (own < 0) len = own = 0;
    int add = p.add[b];
    if (add < 0) {
      atomicOr(p.err, DEV_ERR_BOUNDS);
      add = 0;
    }
    const int n0 = pages_of(in, own);
    const long long cap = (long long)in.stride << in.shift;
    grows[i] = add > 0 && own + (long long)add <= cap;
    if (add > 0 && !grows[i]) atomicOr(p.err, DEV_ERR_BOUNDS);
    w[i] = {src, len, n0, grows[i] ? pages_of(in, own + add) : n0, n0 > 0 ? in.table[(size_t)src * in.stride + n0 - 1] : -1};
    part[i] = grows[i] && (own & ((1 << in.shift) - 1)) != 0 && w[i].last >= 0 && w[i].last < in.num_pages;
    upto[b] = add;  // for now
  }
  __syncthreads();
  // References: every entry of an old sequence by its children less one.
  for (int b = tid >> 5; b < in.B; b += kPageThreads / 32) {
    const int d = kids[b] - 1, own = d ? own_tokens(in, in.lens[b], p.err) : 0, n = own > 0 ? pages_of(in, own) : 0;
    for (int c = tid & 31; c < n; c += 32) {
      const int id = in.table[(size_t)b * in.stride + c];
      if (id >= 0 && id < in.num_pages)
        atomicAdd(out.refs + id, d);
      else
        atomicOr(p.err, DEV_ERR_BOUNDS);
    }
  }
  __threadfence();
  __syncthreads();
  for (int i = 0; i < kEach; ++i)
    if (tid * kEach + i < out.B) kids[tid * kEach + i] = part[i] ? w[i].last : -1;
  __syncthreads();
  // A partly filled last page is copied unless its other holders were copied before.
  int need[kEach], add[kEach], mine = 0;
  bool copied[kEach];
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    need[i] = 0;
    copied[i] = false;
    if (b >= out.B) continue;
    add[i] = upto[b];
    if (part[i]) {
      int left = __ldcg(out.refs + w[i].last);
      for (int o = 0; o < b; ++o) left -= kids[o] == w[i].last;
      copied[i] = left > 1;
    }
    need[i] = grows[i] ? w[i].n1 - w[i].n0 + copied[i] : 0;
    mine += need[i];
  }
  __syncthreads();
  int total, at = block_before(mine, scratch, &total);
  int first[kEach];
  for (int i = 0; i < kEach; ++i) {
    first[i] = at;
    at += need[i];
    if (tid * kEach + i < out.B) upto[tid * kEach + i] = at;
  }
  __syncthreads();
  // Free pages, up to as many as are wanted.
  int found = 0;
  for (int i0 = 0; i0 < in.num_pages && found < total; i0 += kPageThreads) {
    const int i = i0 + tid;
    found += __syncthreads_count(i < in.num_pages && __ldcg(out.refs + i) <= 0);
  }
  // Lengths, copies, and the entries that the sequences begin with.
  bool short_of = false;
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    if (b >= out.B) continue;
    const bool served = grows[i] && (need[i] == 0 || first[i] + need[i] <= found);
    short_of |= grows[i] && !served;
    out.lens[b] = served ? (w[i].len > 0 ? w[i].len : in.prefix_len) + add[i] : w[i].len;
    if (!(served && copied[i])) {
      p.copies[2 * b] = p.copies[2 * b + 1] = -1;
    } else {
      p.copies[2 * b] = w[i].last;
      atomicSub(out.refs + w[i].last, 1);
    }
    for (int c = 0; c < w[i].n0; ++c)
      if (out.table != in.table) out.table[(size_t)b * out.stride + c] = in.table[(size_t)w[i].src * in.stride + c];
    kids[b] = served ? (copied[i] ? -w[i].n0 - 1 : w[i].n0) : 0x7fffffff;  // where the new pages go
  }
  if (short_of) atomicOr(p.err, DEV_ERR_BOUNDS);
  __threadfence();
  __syncthreads();
  int rank0 = 0;
  for (int i0 = 0; i0 < in.num_pages && rank0 < min(found, total); i0 += kPageThreads) {
    const int i = i0 + tid;
    const bool free = i < in.num_pages && __ldcg(out.refs + i) <= 0;
    int all;
    const int rank = rank0 + block_before(free, scratch, &all);
    rank0 += all;
    if (!free || rank >= total) continue;
    int lo = -1, hi = out.B - 1;  // upto[lo] <= rank < upto[hi]
    while (hi - lo > 1) {
      const int mid = lo + hi >> 1;
      if (upto[mid] <= rank)
        lo = mid;
      else
        hi = mid;
    }
    const int k = rank - (hi > 0 ? upto[hi - 1] : 0), to = kids[hi];
    if (to == 0x7fffffff) continue;
    out.refs[i] = 1;
    const int n0 = to < 0 ? -to - 1 : to, c = to < 0 ? n0 + k - 1 : n0 + k;
    out.table[(size_t)hi * out.stride + c] = i;
    if (to < 0 && k == 0) p.copies[2 * hi + 1] = i;
  }
}

struct CompactParams {
  Pool in, out;
  int32_t* map;
  int2* moves;
  int max_moves;
  int32_t* used;
  uint32_t* err;
};

__global__ void __launch_bounds__(kPageThreads) pages_compact_kernel(const CompactParams p) {
  __shared__ int scratch[32];
  grid_dep_wait();
  grid_dep_trigger();
  const Pool &in = p.in, &out = p.out;
  const int tid = threadIdx.x, N = in.num_pages;
  int U = 0, front = 0;
  for (int i0 = 0; i0 < N; i0 += kPageThreads) U += __syncthreads_count(i0 + tid < N && in.refs[i0 + tid] > 0);
  for (int i0 = 0; i0 < U; i0 += kPageThreads) front += __syncthreads_count(i0 + tid < U && in.refs[i0 + tid] > 0);
  const int n = U - front, m = min(n, p.max_moves);
  for (int i = tid; i < p.max_moves; i += kPageThreads) p.moves[i] = make_int2(-1, -1);
  for (int i = tid; i < N; i += kPageThreads) p.map[i] = i;
  if (tid == 0) {
    p.used[0] = U;
    p.used[1] = U;
  }
  __syncthreads();
  int done = 0;
  for (int i0 = 0; i0 < U; i0 += kPageThreads) {  // free places in front, the lowest first
    const bool free = i0 + tid < U && in.refs[i0 + tid] <= 0;
    int all;
    const int r = done + block_before(free, scratch, &all);
    done += all;
    if (free && r < m) p.moves[r].y = i0 + tid;
  }
  done = 0;
  for (int i0 = U; i0 < N; i0 += kPageThreads) {  // pages in use behind, the highest first
    const bool used = i0 + tid < N && in.refs[i0 + tid] > 0;
    int all;
    const int r = n - 1 - done - block_before(used, scratch, &all);
    done += all;
    if (used && r < m) p.moves[r].x = i0 + tid;
    if (used && r == m) p.used[1] = i0 + tid + 1;
  }
  if (out.refs != in.refs)
    for (int i = tid; i < N; i += kPageThreads) out.refs[i] = in.refs[i];
  __syncthreads();
  for (int r = tid; r < m; r += kPageThreads) {
    const int2 x = p.moves[r];
    p.map[x.x] = x.y;
    const int refs = in.refs[x.x];
    out.refs[x.y] = refs;
    out.refs[x.x] = 0;
  }
  __syncthreads();
  auto renamed = [&](int id) {
    if (id >= 0 && id < N) return p.map[id];
    atomicOr(p.err, DEV_ERR_BOUNDS);
    return id;
  };
  for (int b = tid >> 5; b < in.B; b += kPageThreads / 32) {
    const int own = own_tokens(in, in.lens[b], p.err), n_pages = own > 0 ? pages_of(in, own) : 0;
    for (int c = tid & 31; c < n_pages; c += 32)
      out.table[(size_t)b * in.stride + c] = renamed(in.table[(size_t)b * in.stride + c]);
  }
  for (int c = tid; c < pages_of(in, in.prefix_len); c += kPageThreads) out.prefix[c] = renamed(in.prefix[c]);
}

// ---- copies ----
constexpr int kCopyThreads = 256, kCopyLoads = 4, kArrays = PageArrays::kMost;
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
size_t pages_workspace(const fox_pages*) { return kCacheHeaderBytes; }

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

}  // namespace

bool pages_copy_fits(const PageArrays& x, int n) { return (long long)n * copy_params(x).chunks[x.n] <= 0x7fffffffLL; }

cudaError_t launch_pages_copy(const PageArrays& x, int num_pages, const int32_t* pairs, int n, uint32_t* err, cudaStream_t s) {
  CopyParams p = copy_params(x);
  p.num_pages = num_pages;
  p.pairs = reinterpret_cast<const int2*>(pairs);
  p.err = err;
  TraceScope trace("pages_copy", s);
  const cudaError_t e = launch_dependent(pages_copy_kernel, dim3(static_cast<unsigned>(n) * p.chunks[p.arrays]),
                                         dim3(kCopyThreads), 0, s, p);
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
  const StepParams p = {pool_of(in), pool_of(out), parent, add, copies, static_cast<uint32_t*>(workspace)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("pages_step", s);
  const cudaError_t e = launch_dependent(pages_step_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
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
  const CompactParams p = {pool_of(in), pool_of(out), map,  reinterpret_cast<int2*>(moves),
                           max_moves,   used,         static_cast<uint32_t*>(workspace)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace("pages_compact", s);
  const cudaError_t e = launch_dependent(pages_compact_kernel, dim3(1), dim3(kPageThreads), 0, s, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FOX_OK : FOX_ERR_CUDA;
}

}  // extern "C"
