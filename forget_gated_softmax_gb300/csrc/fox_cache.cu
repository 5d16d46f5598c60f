// C ABI of the paged cache: argument validation, tensor maps and launches. See include/fox.h for the contract.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fox.h"
#include "fox_cache.h"

namespace fox {

bool make_page_map(CUtensorMap* map, const void* base, int d, int page_size, int Hkv, int pages, int box_rows) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)Hkv, (cuuint64_t)pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)page_size * d * 2, (cuuint64_t)Hkv * page_size * d * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_q_rows_map(CUtensorMap* map, const void* base, int d, int H, int rows, long long stride, int box_heads,
                     int box_rows) {
  if (rows == 1) stride = (long long)H * d;  // one row has no next
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace fox

using namespace fox;

static_assert(FOX_CACHE_ZERO_BYTES == kCacheHeaderBytes, "the header that include/fox.h documents");

namespace {

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fox_status check_cache(const fox_cache* c) {
  if (!c) return FOX_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->H < 1 || c->Hkv < 1 || c->H % c->Hkv != 0 || c->d <= 0) return FOX_ERR_INVALID_ARG;
  if (c->dtype != FOX_DTYPE_BF16 && c->dtype != FOX_DTYPE_F32) return FOX_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FOX_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FOX_ERR_UNSUPPORTED;
  if (c->H > 65536 || (long long)c->num_pages * c->page_size > (1LL << 40)) return FOX_ERR_UNSUPPORTED;
  return FOX_OK;
}

// Sizes of the batch; `max_new` becomes the exact count where every sequence has the same.
fox_status check_batch(const fox_cache* c, const fox_batch* s, int rows, PagedArgs* a) {
  if (!s || s->B < 0 || rows < 0 || s->prefix_len < 0 || s->table_stride < 1) return FOX_ERR_INVALID_ARG;
  if (s->B > kMaxSeqs) return FOX_ERR_UNSUPPORTED;
  int max_new = s->max_new;
  if (s->cu_new) {
    if (max_new < 1) return FOX_ERR_INVALID_ARG;
    if (max_new > rows) max_new = rows > 0 ? rows : 1;
  } else {
    if (s->B > 0 && rows % s->B != 0) return FOX_ERR_INVALID_ARG;
    max_new = s->B > 0 && rows > 0 ? rows / s->B : 1;
  }
  // positions, row counts of a key head and work units stay inside 32 and 64 bits
  if ((long long)s->prefix_len + (long long)s->table_stride * c->page_size > 0x7fffffffLL) return FOX_ERR_UNSUPPORTED;
  if ((long long)rows * c->H > 0x3fffffffLL) return FOX_ERR_UNSUPPORTED;
  if (a) {
    *a = PagedArgs{};
    a->num_pages = c->num_pages;
    a->page_size = c->page_size;
    a->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    a->H = c->H;
    a->Hkv = c->Hkv;
    a->d = c->d;
    a->B = s->B;
    a->rows = rows;
    a->max_new = max_new;
    a->table_stride = s->table_stride;
    a->prefix_len = s->prefix_len;
    a->cu = s->cu_new;
    a->lens = s->lens;
    a->table = s->table;
    a->prefix = s->prefix_table;
    a->k = c->k;
    a->v = c->v;
    a->g = c->g;
    a->gbase = c->gbase;
  }
  return FOX_OK;
}

fox_status check_pointers(const fox_cache* c, const fox_batch* s) {
  if (!c->k || !c->v || !c->g || !c->gbase || !s->lens || !s->table) return FOX_ERR_INVALID_ARG;
  if (s->prefix_len > 0 && !s->prefix_table) return FOX_ERR_INVALID_ARG;
  if (!at16(c->k) || !at16(c->v) || !at16(c->g) || !at16(c->gbase)) return FOX_ERR_INVALID_ARG;
  const uintptr_t ints = reinterpret_cast<uintptr_t>(s->lens) | reinterpret_cast<uintptr_t>(s->table) |
                         reinterpret_cast<uintptr_t>(s->cu_new) | reinterpret_cast<uintptr_t>(s->prefix_table);
  return (ints & 3u) ? FOX_ERR_INVALID_ARG : FOX_OK;
}

// A row of `heads` heads of d elements, `stride` elements from the next (one row has no next).
bool row_ok(const void* p, int64_t stride, int heads, const fox_cache* c, int rows) {
  const int es = c->dtype == FOX_DTYPE_BF16 ? 2 : 4;
  if (!p || !at16(p)) return false;
  return rows <= 1 || (stride >= (int64_t)heads * c->d && stride < (1LL << 40) && stride * es % 16 == 0);
}

// The bytes from the first to the last of `rows` rows, `stride` elements apart (one row has no next).
struct Span {
  uintptr_t at;
  __int128 bytes;
};
Span span(const void* p, int rows, int64_t stride, int64_t elements, int element) {
  return {reinterpret_cast<uintptr_t>(p), ((__int128)(rows - 1) * (rows > 1 ? stride : 0) + elements) * element};
}
// Whether a call's output lies over something else that the call reads or writes.
bool overlap(const Span& a, const Span& b) { return a.at < b.at + b.bytes && b.at < a.at + a.bytes; }
// The same for rows of `row` bytes, `stride` from one to the next in both: they may lie between each other's.
bool rows_overlap(const Span& a, const Span& b, int64_t stride, int64_t row) {
  if (!overlap(a, b)) return false;
  const int64_t r = static_cast<int64_t>((a.at > b.at ? a.at - b.at : b.at - a.at) % static_cast<uint64_t>(stride));
  return r < row || stride - r < row;
}
int element(const fox_cache* c) { return c->dtype == FOX_DTYPE_BF16 ? 2 : 4; }

fox_status check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || bytes < need) return FOX_ERR_WORKSPACE;
  return FOX_OK;
}

Held held_by(const fox_cache* c) { return c->dtype == FOX_DTYPE_F32 ? Held::kF32 : Held::kBf16; }

// A 4-bit cache as the bf16 one of its shape, whose rows k, v, q and o have, and its scales.
fox_cache as_bf16(const fox_cache4* c) {
  if (!c) return fox_cache{};  // refused, with no pages
  return {c->num_pages, c->page_size, c->H, c->Hkv, c->d, FOX_DTYPE_BF16, c->k, c->v, c->g, c->gbase};
}
struct Four {
  void* ks;
  void* vs;
  bool counted;  // the kernels count a head's tokens through the pool in 32 bits
};
Four four_of(const fox_cache4* c) {
  return c ? Four{c->ks, c->vs, (long long)c->num_pages * c->page_size * c->Hkv < (1LL << 32)} : Four{};
}
fox_status check_four(const Four* f) {
  if (!f->counted) return FOX_ERR_UNSUPPORTED;
  return f->ks && f->vs && at16(f->ks) && at16(f->vs) ? FOX_OK : FOX_ERR_INVALID_ARG;
}

fox_status append_to(const fox_cache* c, const Four* four, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                     const void* v, int64_t v_stride, const float* z, int64_t z_stride, const fox_rotary* rot, float* g_low,
                     void* workspace, size_t workspace_bytes, void* stream) {
  fox_status st = check_cache(c);
  if (st != FOX_OK) return st;
  CacheAppendArgs x = {};
  st = check_batch(c, s, rows, &x.a);
  if (st != FOX_OK) return st;
  if (rot) {
    if (rot->dim < 0 || rot->max_pos < 0 || (rot->pairs != 0 && rot->pairs != 1)) return FOX_ERR_INVALID_ARG;
    if (rot->dim > c->d || rot->dim % 16 != 0) return FOX_ERR_UNSUPPORTED;
  }
  if (s->B == 0 || rows == 0) return FOX_OK;
  st = check_pointers(c, s);
  if (st == FOX_OK && four) st = check_four(four);
  if (st != FOX_OK) return st;
  if (!row_ok(k, k_stride, c->Hkv, c, rows) || !row_ok(v, v_stride, c->Hkv, c, rows)) return FOX_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(g_low) & 3u) return FOX_ERR_INVALID_ARG;
  if (four ? !append4_fits(x.a, rot && rot->q) : !append_fits(x.a, rot && rot->q, c->dtype == FOX_DTYPE_F32)) return FOX_ERR_UNSUPPORTED;
  if (!z || (reinterpret_cast<uintptr_t>(z) & 3u) || (rows > 1 && (z_stride < c->H || z_stride >= (1LL << 40))))
    return FOX_ERR_INVALID_ARG;
  if (rot) {
    if (rot->dim > 0 && (!rot->cos || !rot->sin || !at16(rot->cos) || !at16(rot->sin))) return FOX_ERR_INVALID_ARG;
    if (rot->q && (!row_ok(rot->q, rot->q_stride, c->H, c, rows) || !rot->q_out || !at16(rot->q_out)))
      return FOX_ERR_INVALID_ARG;
    x.cos = rot->cos;
    x.sin = rot->sin;
    x.max_pos = rot->max_pos;
    x.rot = rot->dim;
    x.pairs = rot->pairs;
    x.q = rot->q;
    x.q_out = rot->q_out;
    x.q_stride = rot->q_stride;
  }
  st = check_ws(workspace, workspace_bytes, kErrWordBytes);
  if (st != FOX_OK) return st;
  if (rot && rot->q) {
    const int es = element(c);
    const int64_t row = (int64_t)c->H * c->d, kv = (int64_t)c->Hkv * c->d;
    const Span out = span(rot->q_out, rows, row, row, es);
    const int64_t angles = (int64_t)rot->max_pos * (rot->dim / 2);
    if (overlap(out, span(rot->q, rows, rot->q_stride, row, es)) || overlap(out, span(k, rows, k_stride, kv, es)) ||
        overlap(out, span(v, rows, v_stride, kv, es)) || overlap(out, span(z, rows, z_stride, c->H, 4)) ||
        overlap(out, span(rot->cos, 1, 0, angles, 4)) || overlap(out, span(rot->sin, 1, 0, angles, 4)))
      return FOX_ERR_INVALID_ARG;
  }
  x.a.err = static_cast<uint32_t*>(workspace);
  x.k = k;
  x.v = v;
  x.z = z;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  x.z_stride = z_stride;
  x.g_low = g_low;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const cudaError_t e = four ? launch_cache_append4(x, four->ks, four->vs, on) : launch_cache_append(x, c->dtype == FOX_DTYPE_F32, on);
  return e == cudaSuccess ? FOX_OK : FOX_ERR_CUDA;
}

fox_status decode_over(const fox_cache* c, const Four* four, const fox_batch* s, int rows, const void* q, int64_t q_stride,
                       float scale, int bias_from_j, void* o, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream) {
  fox_status st = check_cache(c);
  if (st != FOX_OK) return st;
  DecodeArgs x = {};
  st = check_batch(c, s, rows, &x.a);
  if (st != FOX_OK) return st;
  if (!(scale >= 0.f) || std::isinf(scale)) return FOX_ERR_INVALID_ARG;
  if (bias_from_j != 0 && bias_from_j != 1) return FOX_ERR_INVALID_ARG;
  if (s->B == 0 || rows == 0) return FOX_OK;
  st = check_pointers(c, s);
  if (st == FOX_OK && four) st = check_four(four);
  if (st != FOX_OK) return st;
  if (!row_ok(q, q_stride, c->H, c, rows) || !o || !at16(o) || !lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FOX_ERR_INVALID_ARG;
  const Held held = four ? Held::kFour : held_by(c);
  if (!decode_fits(x.a, held)) return FOX_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, decode_workspace_bytes(x.a, held));
  if (st != FOX_OK) return st;
  const int64_t row = (int64_t)c->H * c->d;
  const Span so = span(o, rows, row, row, element(c)), sl = span(lse, rows, c->H, c->H, 4);
  const Span sq = span(q, rows, q_stride, row, element(c));  // a row of which several workers read
  if (overlap(so, sq) || overlap(sl, sq) || overlap(so, sl)) return FOX_ERR_INVALID_ARG;
  x.a.err = static_cast<uint32_t*>(workspace);
  x.q = q;
  x.q_stride = q_stride;
  x.scale = scale == 0.f ? 1.f / std::sqrt((float)c->d) : scale;
  x.bias_from_j = bias_from_j;
  x.o = o;
  x.lse = lse;
  x.ks = four ? four->ks : nullptr;
  x.vs = four ? four->vs : nullptr;
  return launch_decode(x, held, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FOX_OK
             : FOX_ERR_CUDA;
}

fox_status copy_in(const fox_cache* c, const Four* four, float* g_low, const int32_t* pairs, int n, void* workspace,
                   size_t workspace_bytes, void* stream) {
  fox_status st = check_cache(c);
  if (st != FOX_OK) return st;
  if (n < 0) return FOX_ERR_INVALID_ARG;
  if (n == 0) return FOX_OK;
  if (!c->k || !c->v || !c->g || !c->gbase || !at16(c->k) || !at16(c->v) || !at16(c->g) || !at16(c->gbase) || !at16(g_low))
    return FOX_ERR_INVALID_ARG;
  if (four && (st = check_four(four)) != FOX_OK) return st;
  if (!pairs || (reinterpret_cast<uintptr_t>(pairs) & 7u)) return FOX_ERR_INVALID_ARG;
  const long long tokens = (long long)c->Hkv * c->page_size, row = four ? c->d / 2 : (long long)c->d * element(c);
  PageArrays x = {};
  x.add(c->k, tokens * row);
  x.add(c->v, tokens * row);
  if (four) {
    x.add(four->ks, tokens * (c->d / 32));
    x.add(four->vs, tokens * (c->d / 32));
  }
  x.add(c->g, (long long)c->H * c->page_size * 4);
  x.add(g_low, (long long)c->H * c->page_size * 4);
  x.add(c->gbase, (long long)c->H * 8);
  if (!pages_copy_fits(x, n)) return FOX_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, kErrWordBytes);
  if (st != FOX_OK) return st;
  return launch_pages_copy(x, c->num_pages, pairs, n, static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FOX_OK
             : FOX_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t fox_cache_workspace_bytes(const fox_cache* c, const fox_batch* s, int rows) {
  PagedArgs a;
  if (check_cache(c) != FOX_OK || check_batch(c, s, rows, &a) != FOX_OK) return 0;
  if (a.B == 0 || rows == 0) return kCacheHeaderBytes;
  if (!decode_fits(a, held_by(c))) return 0;
  return decode_workspace_bytes(a, held_by(c));
}

fox_status fox_cache_append(const fox_cache* c, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* z, int64_t z_stride, const fox_rotary* rot,
                            void* workspace, size_t workspace_bytes, void* stream) {
  return fox_cache_append_low(c, s, rows, k, k_stride, v, v_stride, z, z_stride, rot, nullptr, workspace, workspace_bytes,
                              stream);
}

fox_status fox_cache_append_low(const fox_cache* c, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, const float* z, int64_t z_stride,
                                const fox_rotary* rot, float* g_low, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return append_to(c, nullptr, s, rows, k, k_stride, v, v_stride, z, z_stride, rot, g_low, workspace, workspace_bytes, stream);
}

fox_status fox_decode(const fox_cache* c, const fox_batch* s, int rows, const void* q, int64_t q_stride, float scale,
                      int bias_from_j, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_over(c, nullptr, s, rows, q, q_stride, scale, bias_from_j, o, lse, workspace, workspace_bytes, stream);
}

size_t fox_cache4_workspace_bytes(const fox_cache4* c, const fox_batch* s, int rows) {
  PagedArgs a;
  const fox_cache as = as_bf16(c);
  if (check_cache(&as) != FOX_OK || check_batch(&as, s, rows, &a) != FOX_OK) return 0;
  if (a.B == 0 || rows == 0) return kCacheHeaderBytes;
  return decode_fits(a, Held::kFour) ? decode_workspace_bytes(a, Held::kFour) : 0;
}

fox_status fox_cache4_append(const fox_cache4* c, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const float* z, int64_t z_stride, const fox_rotary* rot,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const fox_cache as = as_bf16(c);
  const Four four = four_of(c);
  return append_to(&as, &four, s, rows, k, k_stride, v, v_stride, z, z_stride, rot, c ? c->g_low : nullptr, workspace,
                   workspace_bytes, stream);
}

fox_status fox_cache4_decode(const fox_cache4* c, const fox_batch* s, int rows, const void* q, int64_t q_stride, float scale,
                             int bias_from_j, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const fox_cache as = as_bf16(c);
  const Four four = four_of(c);
  return decode_over(&as, &four, s, rows, q, q_stride, scale, bias_from_j, o, lse, workspace, workspace_bytes, stream);
}

fox_status fox_cache4_read(const fox_cache4* c, const fox_batch* s, int rows, void* k, int64_t k_stride, void* v,
                           int64_t v_stride, void* workspace, size_t workspace_bytes, void* stream) {
  const fox_cache as = as_bf16(c);
  const Four four = four_of(c);
  fox_status st = check_cache(&as);
  if (st != FOX_OK) return st;
  CacheAppendArgs x = {};
  st = check_batch(&as, s, rows, &x.a);
  if (st != FOX_OK) return st;
  if (s->B == 0 || rows == 0) return FOX_OK;
  st = check_pointers(&as, s);
  if (st == FOX_OK) st = check_four(&four);
  if (st != FOX_OK) return st;
  if (!row_ok(k, k_stride, c->Hkv, &as, rows) || !row_ok(v, v_stride, c->Hkv, &as, rows)) return FOX_ERR_INVALID_ARG;
  const int64_t row = (int64_t)c->Hkv * c->d;
  const Span sk = span(k, rows, k_stride, row, 2), sv = span(v, rows, v_stride, row, 2);
  if (rows > 1 && k_stride == v_stride ? rows_overlap(sk, sv, 2 * k_stride, 2 * row) : overlap(sk, sv)) return FOX_ERR_INVALID_ARG;
  if (!append4_fits(x.a, false)) return FOX_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, kErrWordBytes);
  if (st != FOX_OK) return st;
  x.a.err = static_cast<uint32_t*>(workspace);
  x.k = k;
  x.v = v;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  return launch_cache_read4(x, four.ks, four.vs, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FOX_OK : FOX_ERR_CUDA;
}

fox_status fox_cache_copy(const fox_cache* c, float* g_low, const int32_t* pairs, int n, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return copy_in(c, nullptr, g_low, pairs, n, workspace, workspace_bytes, stream);
}

fox_status fox_cache4_copy(const fox_cache4* c, const int32_t* pairs, int n, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const fox_cache as = as_bf16(c);
  const Four four = four_of(c);
  return copy_in(&as, &four, c ? c->g_low : nullptr, pairs, n, workspace, workspace_bytes, stream);
}

}  // extern "C"
