// Internal declarations of the paged cache: launches, workspace and tensor maps.
#pragma once

#include "fox_internal.h"
#include "fox_paged.h"

namespace fox {

constexpr int kSMs = 152;  // of one GB300: grids of resident workers are sized for it, any count works

// New tokens into the cache (k, v rotated and gates), and attention over it. Every kernel is launched as a
// programmatic dependent of what is ahead of it on the stream; the first of a call waits for that before it
// reads or writes anything in memory (and only then lets the next start), so that its launch and set-up
// overlap the end of the call before (step after step: one token appended 16.0 -> 14.3 us, a decode of 65536 keys
// 59.0 -> 57.5, one behind a prefix of 16384 tokens 55.8 -> 53.5).
// Strides are elements from one token's row to the next.
constexpr size_t kCacheHeaderBytes = 16384;  // error word, then a counter a decode worker: all zero between calls
struct CacheAppendArgs {
  PagedArgs a;
  const void* k;
  const void* v;
  const float* z;
  const void* q;  // rotated into q_out, or null
  void* q_out;
  long long k_stride, v_stride, z_stride, q_stride;
  const float* cos;
  const float* sin;
  int max_pos, rot, pairs;
  float* g_low;  // what the rounding of g leaves of the sums, laid out like g, or null
};
bool append_fits(const PagedArgs& a, bool with_q, bool f32);  // its blocks are one grid's
cudaError_t launch_cache_append(const CacheAppendArgs& x, bool f32, cudaStream_t s);
struct DecodeArgs {
  PagedArgs a;
  const void* q;
  long long q_stride;
  float scale;
  int bias_from_j;
  void* o;
  float* lse;
};
bool decode_fits(const PagedArgs& a, bool f32);  // its work is counted in ints
size_t decode_workspace_bytes(const PagedArgs& a, bool f32);
cudaError_t launch_decode(const DecodeArgs& x, bool f32, char* ws, cudaStream_t s);

// 4-D bf16 tensor map over a paged pool [pages, Hkv, page_size, d], box 64 channels x box_rows tokens, 128-byte swizzle.
bool make_page_map(CUtensorMap* map, const void* base, int d, int page_size, int Hkv, int pages, int box_rows);
// 3-D bf16 tensor map over query rows [rows, H, d], `stride` elements a row, box 64 channels x box_heads x box_rows.
bool make_q_rows_map(CUtensorMap* map, const void* base, int d, int H, int rows, long long stride, int box_heads,
                     int box_rows);

}  // namespace fox
