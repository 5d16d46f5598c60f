// What the tensor-core decode kernels of the bf16 and the 4-bit cache share: a warp's ring of key tiles, its windows of pages, the rows of
// its items, and the register MMAs' operands.
#pragma once
#include "fox_decode.h"

namespace fox {
namespace {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
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

// Up to 32 successive key tiles of one item. The table's entries for them (with pages of 16 tokens two a
// tile) come to shared memory by asynchronous copies, so that no instruction waits for them before their use.
struct Window {
  int hkv, rt, tile, n, own;
};

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

}  // namespace
}  // namespace fox
