// mxs_rope.cuh -- the rotation shared by mxs_rope and mxs_kv_write: phases,
// cos and sin, and vector loads of 8 values.
#pragma once

#include "mxs_internal.cuh"

namespace mxs {

// cos and sin (times the plan's gain) of pair i at position pos.  The phase
// is the 64-bit product pos * step modulo one turn, taken as a signed
// fraction of half a turn: no range reduction, and the rounding to a double
// is off by at most 2^-55 turns at any position.
__device__ __forceinline__ double2 rope_turn(uint64_t step, double gain, int64_t pos, bool inverse) {
  const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(pos) * step);
  double s, c;
  sincospi(static_cast<double>(phase) * 0x1p-63, &s, &c);
  return make_double2(c * gain, inverse ? -s * gain : s * gain);
}

// One turned pair.  Both kernels must give the same bits: the products and
// the sum are spelled out, so that no other contraction is possible.
__device__ __forceinline__ void rope_pair(float &u, float &v, double2 cs) {
  const double a = u, b = v;
  u = __double2float_rn(__fma_rn(a, cs.x, -__dmul_rn(b, cs.y)));
  v = __double2float_rn(__fma_rn(b, cs.x, __dmul_rn(a, cs.y)));
}

template <bool F32>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if constexpr (F32) return static_cast<const float *>(p)[i];
  else return bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]);
}
// 8 consecutive values from a 16-byte aligned place, as they are in memory
// (fetched early, widened late: half the registers for bf16).
template <bool F32>
struct Raw8 {
  uint4 q[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> fetch8(const void *p, int64_t i) {
  Raw8<F32> r;
  if constexpr (F32) {
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
    r.q[0] = s[0];
    r.q[1] = s[1];
  } else {
    r.q[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void widen8(const Raw8<F32> &r, float (&v)[8]) {
  if constexpr (F32) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool F32>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
  if constexpr (F32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(bf16_pair(v, 0.f));
}
template <bool F32>
__device__ __forceinline__ void store8(void *p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
}

// Host: a plan as mxs_rope_plan_make leaves it, with rot <= d.
mxs_status check_rope_plan(const mxs_rope_plan *plan, int64_t d);
// Host: the pointer and strides (elements of `size` bytes) allow 16-byte
// accesses at every multiple of 8 values.
inline bool vec8_ok(const void *p, int64_t ldt, int64_t ldh, size_t size) {
  return aligned16(p) && (ldt * static_cast<int64_t>(size)) % 16 == 0 && (ldh * static_cast<int64_t>(size)) % 16 == 0;
}
// Number of SMs of the current device.
int device_sms();

}  // namespace mxs
