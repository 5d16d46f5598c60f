// The 4-bit form of the paged cache: blocks of 32 channels of one token and key head, value = s u. Where its bytes lie,
// its scales, and how a block is made. Plain C++ apart from the qualifiers, as fox_paged.h.
#pragma once
#include <cmath>
#include <cstring>

#include "fox_paged.h"

namespace fox {

constexpr int kFourBlock = 32;        // channels that share a scale
constexpr int kFourTop = 7;           // codes are u + 8, u = -7 .. 7
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
FOX_HD uint32_t four_k_code(uint32_t w) {
  w = w << 2 | w >> 30;
  return (w >> 8 & 15u) | (w >> 24 & 15u) << 4 | (w >> 4 & 15u) << 8 | (w >> 20 & 15u) << 12 | (w >> 12 & 15u) << 16 |
         (w >> 28 & 15u) << 20 | (w >> 16 & 15u) << 24 | (w & 15u) << 28;
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
// u + 8 of x, inv = 1 / s (0 where s is): |x| / s rounded, halves up. A bf16 value over s is a half or 2^-11 away from it,
// which the 2^-12 makes up for the rounding of inv and of the product.
FOX_HD uint32_t four_code(float x, float inv) {
  const float y = fabsf(x) * inv + (0.5f + 0x1p-12f);
  const int u = y >= kFourTop ? kFourTop : y >= 1.f ? static_cast<int>(y) : 0;  // NaN: 0
  return static_cast<uint32_t>(8 + (x < 0.f ? -u : u));
}

}  // namespace fox
