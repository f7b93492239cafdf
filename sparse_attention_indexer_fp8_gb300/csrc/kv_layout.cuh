// The attention cache's record and its dequantisation, shared by the writer, the
// read-back and the attention kernels.
//
// Block of bs tokens: the e4m3 latent of token i at 512 i, its rotated bf16
// position dims at 512 bs + 128 i, its four E8M0 codes (one per 128 dims) at
// 640 bs + 4 i.
#pragma once

#include "common.cuh"

namespace idx {

constexpr int kKvLatent = IDX_KV_LATENT;           // 512 e4m3 dims: keys and values
constexpr int kKvRope = IDX_KV_ROPE;               // 64 bf16 dims: keys only
constexpr int kKvDim = kKvLatent + kKvRope;
constexpr int kKvRopeAt = kKvLatent;               // x block_size: where the position dims start
constexpr int kKvScaleAt = kKvLatent + 2 * kKvRope;  // x block_size: where the scale codes start
constexpr int kKvMaxScaleCode = 134;               // 2^7
constexpr int kKvNanScaleCode = 255;               // 128 dims one of which was not finite: all read as NaN
constexpr int kKvCodeLimit = kKvMaxScaleCode + 1;  // readers hold codes to it: its multiplier is infinity

idx_status_t check_kv_cache(const char* fn, const void* cache, int32_t num_blocks, int32_t block_size,
                            int64_t block_stride);  // kv_cache.cu

// bf16x2 multiplier that turns an e4m3 byte spread into a bf16 (below) into its value times
// 2^(code - 127). Above kKvMaxScaleCode only kKvNanScaleCode is written, with 128 zero bytes: held to
// kKvCodeLimit it makes the multiplier infinity, and zero times infinity the NaN that they stand for.
__device__ __forceinline__ uint32_t kv_dequant_multiplier(uint32_t code) {
  // 2^(120 + code - 127) has exponent field code + 120
  return (min(code, static_cast<uint32_t>(kKvCodeLimit)) + 120u) * 0x00800080u;
}

// The same of a code that is known to be at most kKvCodeLimit.
__device__ __forceinline__ uint32_t kv_multiplier_of(uint32_t code) { return code * 0x00800080u + 120u * 0x00800080u; }

// Four e4m3 bytes to four bf16 (lo: bytes 0, 1; hi: bytes 2, 3), times the multiplier.
// A byte s eeee mmm placed as the bf16 s 0000eeee mmm0000 has the e4m3 value times
// 2^-120, subnormals included (both formats extend their lowest exponent linearly),
// so one bf16 multiplication by 2^(120 + scale exponent) gives the scaled value. It
// is exact: four significant bits, a power of two. Bytes 0x7F and 0xFF (e4m3's NaN), which
// are never written, read as +-480 times the scale.
__device__ __forceinline__ void kv_dequant4(uint32_t w, uint32_t mul, uint32_t& lo, uint32_t& hi) {
  const uint32_t p = __byte_perm(w, 0u, 0x1404);  // byte 1 -> bits 24-31, byte 0 -> bits 8-15
  const uint32_t q = __byte_perm(w, 0u, 0x3424);
  const uint32_t a = ((p >> 4) & 0x07F007F0u) | (p & 0x80008000u);
  const uint32_t b = ((q >> 4) & 0x07F007F0u) | (q & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(mul));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(mul));
}

// The same with bytes 0, 2 in `even` and 1, 3 in `odd`: no byte shuffles, so five
// operations of the half-rate integer pipe for four values instead of eight.
__device__ __forceinline__ void kv_dequant4_even_odd(uint32_t w, uint32_t mul, uint32_t& even, uint32_t& odd) {
  const uint32_t a = ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u);
  const uint32_t b = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(a), "r"(mul));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(b), "r"(mul));
}

// The same as kv_dequant4 in eight operations instead of nine to ten: each byte beside eight copies of its sign, both
// shifted at once, and one mask for what belongs to neither the sign nor the seven bits.
__device__ __forceinline__ void kv_dequant4_signs(uint32_t w, uint32_t mul, uint32_t& lo, uint32_t& hi) {
  uint32_t p, q;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(p) : "r"(w));  // bytes 0, sign of 0, 1, sign of 1
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(q) : "r"(w));
  const uint32_t a = (p << 4) & 0x87F087F0u;
  const uint32_t b = (q << 4) & 0x87F087F0u;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(mul));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(mul));
}

}  // namespace idx
