// Paged cache: argument block and index arithmetic shared by the append and decode kernels
// and by the host. Plain C++ apart from the qualifiers, so that the arithmetic that decides
// every read and write of the cache can be checked without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define FOX_HD __host__ __device__ __forceinline__
#else
#define FOX_HD inline
#endif

namespace fox {

constexpr int kMaxSeqs = 2048;  // sequences of one call: every CTA holds their work offsets in shared memory

struct PagedArgs {
  int num_pages, page_size, page_shift, H, Hkv, d;  // page_size = 1 << page_shift
  int B, rows, max_new;  // max_new: at least every sequence's count of new tokens
  int table_stride, prefix_len;
  const int32_t* cu;      // [B + 1] first row of each sequence, or null: rows / B rows each
  const int32_t* lens;    // [B] tokens of each sequence, prefix and new ones included; 0: an idle sequence
  const int32_t* table;   // [B][table_stride] pages of the tokens after the prefix
  const int32_t* prefix;  // [ceil(prefix_len / page_size)] pages of the shared prefix
  void* k;
  void* v;
  float* g;
  float* gbase;
  uint32_t* err;
};

// One sequence of the batch: its rows [row0, row0 + n) and its tokens after the prefix (the new
// ones among them). An idle sequence (lens 0) keeps its rows and has own = -1: nothing is appended
// for it and its rows attend to nothing. `bad` reports lengths that the batch cannot hold; the
// sequence then has no rows.
struct SeqInfo {
  int row0, n, own;
};

FOX_HD int first_row(const PagedArgs& a, int b) { return a.cu ? a.cu[b] : a.rows / a.B * b; }

FOX_HD SeqInfo seq_info(const PagedArgs& a, int b, bool* bad) {
  SeqInfo s;
  s.row0 = first_row(a, b);
  const int r1 = first_row(a, b + 1);
  const int len = a.lens[b];
  const long long cap = (long long)a.prefix_len + (long long)a.table_stride * a.page_size;
  const bool rows_ok = s.row0 >= 0 && r1 >= s.row0 && r1 <= a.rows && r1 - s.row0 <= a.max_new;
  s.n = r1 - s.row0;
  const bool ok = rows_ok && (len == 0 || (len > 0 && (long long)len >= (long long)a.prefix_len + s.n && len <= cap));
  *bad = !ok;
  if (!ok) {
    s.row0 = 0;
    s.n = 0;
    s.own = -1;
    return s;
  }
  s.own = len == 0 ? -1 : len - a.prefix_len;
  return s;
}

// The sequence that row i belongs to, or -1: behind the last sequence. With cu not rising the
// answer is some sequence in [0, B), whose seq_info then has to hold the row.
FOX_HD int seq_of_row(const PagedArgs& a, int i) {
  if (!a.cu) return i / (a.rows / a.B);
  if (i >= a.cu[a.B] || i < a.cu[0]) return -1;
  int lo = 0, hi = a.B;  // cu[lo] <= i < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The page of own token p of sequence b (0 <= p < table_stride * page_size), or -1 where the
// table's entry is no page of the pool.
FOX_HD int own_page(const PagedArgs& a, int b, int p) {
  const int id = a.table[(size_t)b * a.table_stride + (p >> a.page_shift)];
  return id >= 0 && id < a.num_pages ? id : -1;
}
FOX_HD int prefix_page(const PagedArgs& a, int p) {
  const int id = a.prefix[p >> a.page_shift];
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Elements from the pool's start to (page, head, slot).
FOX_HD size_t kv_offset(const PagedArgs& a, int page, int hkv, int slot) {
  return (((size_t)page * a.Hkv + hkv) * a.page_size + slot) * a.d;
}
FOX_HD size_t g_offset(const PagedArgs& a, int page, int h, int slot) {
  return ((size_t)page * a.H + h) * a.page_size + slot;
}
FOX_HD size_t gbase_offset(const PagedArgs& a, int page, int h) { return ((size_t)page * a.H + h) * 2; }

// ---- work of the decode kernels ----
// An item is (key head, sequence, row tile): `Rt` of the sequence's n * Gp query rows of that key
// head against its keys. Row r is token r / Gp and query head hkv * G + r % Gp of the group's G = H / Hkv;
// Gp is G, or its next multiple of Rt where G is larger than a row tile, so that a tile never holds the
// end of one token's group and the start of the next's (rows with r % Gp >= G are empty). An item's
// units are the key tiles of kKeyTile tokens. The units of all items lie on one line, items in the order (key head, sequence,
// row tile), and worker w takes units [w q, (w + 1) q): equal work whatever the lengths are.
// An item that lies in one worker's range is finished there; of the others a worker can leave a partial
// result, in slot worker + item: along the line each new (worker, item) pair raises one of the
// two, so no two pairs meet, and there are fewer than workers + items slots.
// Items of a key head are numbered so that the number follows from the sequence alone: by the most row tiles of any
// sequence, or, where sequences bring very different counts, by the rows before it: with x = Gp / Rt
// row tiles a row, sequence b has the numbers from floor(row0 x) + b on, ceil(n x) of them, which the next one's
// floor((row0 + n) x) + b + 1 is not below. (64 sequences on 32 / 8 heads of 128 channels, one of them with 16384 new
// tokens: 0.28 GB of partial results; by sequence 17.4 GB.) That takes row ranges that rise from sequence to sequence.
constexpr int kKeyTile = 32;

FOX_HD int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Key tiles that a sequence's items walk: with `walk_prefix` (nothing shares the prefix out) the prefix's
// first, then its own, each from a tile's start.
FOX_HD int walk_tiles(const PagedArgs& a, int own, bool walk_prefix) {
  return own < 0 ? 0 : (walk_prefix ? ceil_div(a.prefix_len, kKeyTile) : 0) + ceil_div(own, kKeyTile);
}
FOX_HD int padded_group(int G, int Rt) { return G <= Rt ? G : ceil_div(G, Rt) * Rt; }
struct Numbering {
  int items;                   // numbers of a key head
  int per_seq, per_row, shift; // of a sequence's first item: b per_seq + (row0 per_row >> shift)
  FOX_HD bool by_rows() const { return per_row > 0; }
};
FOX_HD int first_item(const Numbering& x, int b, int row0) { return b * x.per_seq + (row0 * x.per_row >> x.shift); }
// The one of the two that takes fewer numbers; `rt_shift`: Rt = 1 << rt_shift, `row_tiles`: the most of a sequence.
// `items` gets the count also where it is no int.
inline Numbering numbering(const PagedArgs& a, int Gp, int rt_shift, int row_tiles, long long* items) {
  const long long by_rows = ((long long)a.rows * Gp >> rt_shift) + a.B, by_seq = (long long)a.B * row_tiles;
  *items = by_rows < by_seq ? by_rows : by_seq;
  if (by_rows < by_seq) return {static_cast<int>(by_rows), 1, Gp, rt_shift};
  return {static_cast<int>(by_seq), row_tiles, 0, 0};
}
FOX_HD int seq_units(const PagedArgs& a, const SeqInfo& s, int Rt, int Gp, bool walk_prefix) {
  return walk_tiles(a, s.own, walk_prefix) * ceil_div(s.n * Gp, Rt);
}
// The most units that the batch's tables allow for so many items a key head.
FOX_HD long long most_units(const PagedArgs& a, long long items) {
  const long long cap = (long long)a.prefix_len + (long long)a.table_stride * a.page_size;
  return (cap / kKeyTile + 2) * items * a.Hkv;
}
// Whether every place on a line of at most `most` units that the kernels form is an int: the ends of ranges before they
// are cut off at the line's end, which lie up to a CTA's units (`warps` workers), or a worker's more, behind it.
FOX_HD bool line_fits(long long most, int workers, int warps) {
  const long long each = (most + workers - 1) / workers;
  return most <= 0x7fffffffLL && most + workers + (warps + 1) * each <= 0x7fffffffLL;
}
FOX_HD int units_per_worker(int total, int workers) {
  const int q = (total + workers - 1) / workers;
  return q > 0 ? q : 1;
}

}  // namespace fox
