// What the tensor-core decode kernels of the bf16 and the 4-bit cache share: a warp's windows of key tiles, and the register MMAs' operands.
#pragma once
#include "fox_decode.h"

namespace fox {
namespace {

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
// Up to 32 successive key tiles of one item, whose table entries (with pages of 16 tokens two a tile) are asked for together, a window ahead.
struct Window {
  int hkv, rt, tile, n, own;
};

}  // namespace
}  // namespace fox
