// mxs_cache.cuh -- the K/V cache pool as the serving kernels see it.
#pragma once

#include "mxs_internal.cuh"

namespace mxs {

struct CacheView {
  uint8_t *codes[2], *scales[2];          // K, V
  int64_t code_pitch[2], scale_pitch[2];
  uint32_t code_slot[2], scale_slot[2];   // bytes from a slot to the next
  int64_t n_slots;                        // < 2^31
  int32_t n_kvh, d, bits;
};

// Host: checks the cache (one width, identity layout, matching rows) and
// fills *v.
mxs_status cache_view(const mxs_kv_cache *c, CacheView *v);

// Records an index out of range in the device status word (a timeout that
// is already there stays).
__device__ __forceinline__ void record_bad_index(int *status) { atomicCAS(status, 0, static_cast<int>(MXS_ERR_SHAPE)); }

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// bf16 bits of 2^(b - 129), the step of a 4-bit block with scale byte b.
__device__ __forceinline__ uint32_t step4(uint32_t b) { return b >= 3u ? (b - 2u) << 7 : 1u << (b + 4u); }
// ... and 2^(b - 133), that of an 8-bit block.
__device__ __forceinline__ uint32_t step8(uint32_t b) { return b >= 7u ? (b - 6u) << 7 : 1u << b; }

// 8 codes -> 8 exact bf16 values.  4 bits (one word): the nibble with its
// sign bit flipped in the mantissa of 128.0 is 136 + q, and
// fma(136 + q, s, -136 s) = q s.  8 bits (two words), q = 16 h + l:
// fma(136 + h, 16 s, -2304 s) = (16 h - 128) s, then fma(128 + l, s, .) = q s;
// every intermediate is exact in bf16.  Two codes per instruction come from
// the two halves of a word, so the values leave in the order 0 4 1 5 2 6 3 7
// (4 bits) or 0 2 1 3 of each word (8 bits).
template <int M>
struct BlockScale {
  uint32_t s, c, s16;
};
template <>
struct BlockScale<4> {
  uint32_t s, c;
};
constexpr uint32_t kTopScale = 249;              // above, -136 s leaves bf16's range
template <int M>
__device__ __forceinline__ BlockScale<M> scale_factors(uint32_t b) {
  const uint32_t c = (0x8000u | ((b + 5u) << 7) | (M == 4 ? 8u : 16u)) * 0x10001u;
  if constexpr (M == 4) return {step4(b) * 0x10001u, c};
  else return {step8(b) * 0x10001u, c, step4(b) * 0x10001u};
}
// The same where both factors are normal bf16 values, linear in b: all
// scale bytes but a few at either end.
template <int M>
__device__ __forceinline__ bool mid_scale(uint32_t b) {
  constexpr uint32_t lo = M == 4 ? 3 : 7;
  return b - lo <= kTopScale - lo;
}
template <int M>
__device__ __forceinline__ BlockScale<M> mid_factors(uint32_t b) {
  const uint32_t x = b * 0x00800080u;
  constexpr uint32_t c = ((0x8000u | (M == 4 ? 8u : 16u)) + (5u << 7)) * 0x10001u;
  if constexpr (M == 4) return {x - 0x01000100u, x + c};
  else return {x - 0x03000300u, x + c, x - 0x01000100u};
}
template <int M>
__device__ __forceinline__ uint4 decode8(uint32_t w0, uint32_t w1, const BlockScale<M> &k) {
  uint32_t o[4];
  if constexpr (M == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fma2(((w0 >> (4 * i)) & 0x000F000Fu) ^ 0x43084308u, k.s, k.c);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i < 2 ? w0 : w1) >> (8 * (i & 1));
      o[i] = fma2((w & 0x000F000Fu) | 0x43004300u, k.s, fma2(((w >> 4) & 0x000F000Fu) ^ 0x43084308u, k.s16, k.c));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace mxs
