// The 4-bit form of the paged cache: blocks of 32 channels of one token and key head, value = s u. Where its bytes lie,
// its scales, and how a block is made. Plain C++ apart from the qualifiers, as fox_paged.h.
#pragma once
#include <cmath>
#include <cstring>

#include "fox_paged.h"

namespace fox {

constexpr int kFourBlock = 32;        // channels that share a scale
constexpr int kFourMaxScale = 0xF7;   // 61440; larger bytes are no scales (in fp16 an infinity and NaNs)

// ---- layout, in bytes from the pool's start ----
FOX_HD size_t four_row(const PagedArgs& a, int page, int hkv, int slot) {
  return (((size_t)page * a.Hkv + hkv) * a.page_size + slot) * (a.d / 2);
}
FOX_HD size_t four_scale_row(const PagedArgs& a, int page, int hkv, int slot) {  // of K; of V the 16 tokens of the slot
  return (((size_t)page * a.Hkv + hkv) * a.page_size + slot) * (a.d / kFourBlock);
}
// Of a token's row: the word that holds channels 32 b + 8 t .. + 7. V's blocks are turned by the slot, so that eight tokens'
// 16 bytes of one block, which an ldmatrix reads at once, lie in different banks of shared memory.
FOX_HD int four_k_word(int b, int t, int blocks) { return (t * blocks + b) * 4; }
FOX_HD int four_v_place(int b, int slot, int blocks) { return b ^ (blocks == 4 ? (slot >> 1) & 3 : (slot >> 2) & 1); }
FOX_HD int four_v_word(int b, int t, int slot, int blocks) { return four_v_place(b, slot, blocks) * 16 + t * 4; }
// V's scales of 16 tokens: the four that a lane's part of an MMA operand needs side by side, 2 t and 2 t + 1 (bytes 0 and 2) and
// 2 t + 8 and 2 t + 9 (bytes 1 and 3).
FOX_HD int four_v_scale(int b, int slot, int blocks) {
  const int j = slot & 15;
  return ((j & 7) >> 1) * 4 * blocks + b * 4 + 2 * (j & 1) + (j >> 3);
}
// ---- codes of eight channels to a word, nibble c of `code` channel c's (u + 8) ----
// V: as they are. K: in the order 7 2 0 4 6 3 1 5, rotated right by 2, so that channels 2 i and 2 i + 1 lie 16 bits apart, those of
// i = 0 at bits 9 .. 6 of each half and of i = 1 at bits 5 .. 2, and those of i = 3 and 2 after a rotation by 8.
FOX_HD uint32_t four_k_order(uint32_t code) {
  const uint32_t w = (code >> 28 & 15u) | (code >> 8 & 15u) << 4 | (code & 15u) << 8 | (code >> 16 & 15u) << 12 |
                     (code >> 24 & 15u) << 16 | (code >> 12 & 15u) << 20 | (code >> 4 & 15u) << 24 | (code >> 20 & 15u) << 28;
  return w >> 2 | w << 30;
}

// ---- scales: 5 exponent bits (bias 15), 3 mantissa bits ----
FOX_HD float bits_float(uint32_t x) {
#ifdef __CUDA_ARCH__
  return __uint_as_float(x);
#else
  float f;
  std::memcpy(&f, &x, 4);
  return f;
#endif
}
FOX_HD uint32_t float_bits(float f) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(f);
#else
  uint32_t x;
  std::memcpy(&x, &f, 4);
  return x;
#endif
}
FOX_HD float four_scale(uint32_t byte) {
  return byte >= 8 ? bits_float((byte + (112u << 3)) << 20) : static_cast<float>(byte) * 0x1p-17f;
}
// The smallest scale with 7 s >= amax (a bf16 magnitude, not NaN). amax has 8 significant bits and 7 s has 7: where they
// differ they do by 2^-9 at least, so amax / 7 is formed by a product, 2^-12 below it, and no rounding of that matters.
FOX_HD uint32_t four_scale_byte(float amax) {
  const float t = amax * (0.14285714285714285f * (1.f - 0x1p-12f));
  if (!(t < 61440.f)) return kFourMaxScale;
  if (t < 0x1p-14f) return static_cast<uint32_t>(ceilf(t * 0x1p17f));
  return (float_bits(t) + 0xFFFFFu >> 20) - (112u << 3);
}
// u + 8 of a finite x of at most 7 s, in bits above kFourNone's; inv = 1 / s within 2^-22 of it (0 where s is): x / s is a half or 2^-11
// away from one, so a factor of 1 + 2^-15 brings halves (0.5 at least) 2^-16 away from zero, and nothing else over a half. The nearest
// integer is then what an fma with 1.5 * 2^23 leaves in the low bits.
constexpr uint32_t kFourNone = 0x4B400000u;
FOX_HD uint32_t four_code_bits(float x, float inv) { return float_bits(fmaf(x, inv * (1.f + 0x1p-15f), 12582912.f + 8.f)); }

#ifdef __CUDACC__
// ---- eight channels at once, on the device ----
__device__ __forceinline__ uint32_t four_bf16(uint32_t n, uint32_t s2) {  // nibbles at bits 3..0 of both halves: s u, exactly
  uint32_t x, y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(n), "r"(0x000F000Fu), "r"(0x43004300u));  // 128 + n
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xC308C308u));                          // - 136
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(y), "r"(s2));
  return x;
}
// The fp16 values of a word of V, an infinity for 65536 and above. Pairs of 1024 + n, less 1032, times s: exact.
__device__ __forceinline__ uint32_t four_f16(uint32_t n, uint32_t s2) {  // nibbles at bits 3..0 of both halves
  uint32_t x, y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(n), "r"(0x000F000Fu), "r"(0x64006400u));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xE408E408u));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(y), "r"(s2));
  return x;
}
__device__ __forceinline__ uint4 four_v16(uint32_t w, uint32_t byte) {
  const uint32_t s2 = byte * 0x00800080u;  // a byte's nibbles 16 bits apart: times 0x1001
  return make_uint4(four_f16((w & 255u) * 0x1001u, s2), four_f16((w >> 8 & 255u) * 0x1001u, s2), four_f16((w >> 16 & 255u) * 0x1001u, s2),
                    four_f16((w >> 24) * 0x1001u, s2));
}
// The bf16 values of a word of K or of V.
__device__ __forceinline__ uint4 four_values(uint32_t w, uint32_t byte, bool is_v) {
  const uint32_t s = float_bits(four_scale(byte)) >> 16, s2 = s << 16 | s;
  if (is_v) {  // a byte's nibbles 16 bits apart: times 0x1001
    const uint32_t b[4] = {(w & 255u) * 0x1001u, (w >> 8 & 255u) * 0x1001u, (w >> 16 & 255u) * 0x1001u, (w >> 24) * 0x1001u};
    return make_uint4(four_bf16(b[0], s2), four_bf16(b[1], s2), four_bf16(b[2], s2), four_bf16(b[3], s2));
  }
  return make_uint4(four_bf16(w >> 6, s2), four_bf16(w >> 2, s2), four_bf16(w >> 10, s2), four_bf16(w >> 14 | w << 18, s2));
}
// The larger magnitude in both halves of two bf16 pairs, a NaN where there is one; the signs are no numbers'.
__device__ __forceinline__ uint32_t four_larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t four_larger(const uint4& w) { return four_larger(four_larger(w.x, w.y), four_larger(w.z, w.w)); }
// Codes of eight values: nibble c is channel c's.
__device__ __forceinline__ uint32_t four_codes(const float* f, float inv) {
  uint32_t code = four_code_bits(f[7], inv), none = kFourNone;
#pragma unroll
  for (int e = 6; e >= 0; --e) {
    code = code * 16 + four_code_bits(f[e], inv);
    none = none * 16 + kFourNone;
  }
  return code - none;
}
#endif

}  // namespace fox
