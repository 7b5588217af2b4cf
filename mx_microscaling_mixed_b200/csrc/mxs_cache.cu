// mxs_cache.cu -- new tokens into the MXINT K/V cache, and back.
//
// Coding as the quantisers do: a block of 32 positions has e = floor(log2
// max|x|) (E8M0 byte e + 127) and codes clamp(rint(x 2^(m-2-e))).  The keys
// are first turned to their positions, x_u cos a - x_v sin a, rounded once
// to fp32.
#include <algorithm>

#include "mxs_cache.cuh"
#include "mxs_ptx.cuh"
#include "mxs_rope.cuh"

namespace mxs {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kReadThreads = 256;
constexpr float kRoundMagic = 12582912.0f;       // 1.5 * 2^23: adding it rounds to an integer, ties to even
constexpr uint32_t kRoundBits = 0x4B400000u;

struct WriteArgs {
  CacheView c;
  const void *src[2];
  int64_t ldt[2], ldh[2];
  const int64_t *slot, *pos;
  int64_t T;
  int32_t rope, tokens;
  int *status;
};

// The block's scale factor 2^(m-2-e) from the magnitude bits of its maximum,
// as two factors: tiny blocks (below 2^-121) need more than one.
struct CodeScale {
  float pre, sc;
  uint32_t byte;
};
template <int M>
__device__ __forceinline__ CodeScale code_scale(uint32_t amax_bits) {
  CodeScale r;
  r.byte = amax_bits >> 23;
  int k = M - 2 - (r.byte == 0 ? -127 : static_cast<int>(r.byte) - 127);
  r.pre = 1.f;
  if (k > 127) {
    r.pre = 18446744073709551616.0f;             // 2^64, exact
    k -= 64;
  }
  r.sc = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
  return r;
}
template <int M>
__device__ __forceinline__ uint32_t code_of(float x, CodeScale s) {
  constexpr uint32_t L = (1u << (M - 1)) - 1u;
  const uint32_t b = __float_as_uint(fmaf(x * s.pre, s.sc, kRoundMagic));
  return min(max(b, kRoundBits - L), kRoundBits + L) & ((1u << M) - 1u);
}
// Both halves to lo..hi.  As fp16 values these small integers are subnormal
// and in the same order, and fp16 pairs have instructions for it.
__device__ __forceinline__ uint32_t clamp2(uint32_t x, uint32_t lo, uint32_t hi) {
  asm("max.f16x2 %0, %0, %1;\n\tmin.f16x2 %0, %0, %2;" : "+r"(x) : "r"(lo), "r"(hi));
  return x;
}
// A word of codes from 32 / M values.  With 2^(M-1) more in the constant (an
// even number: ties go the same way) the sums' low halves are code +
// 2^(M-1), from 0 to 2^M; two of them are clamped at once, the fields added
// up, and flipping their top bits makes two's complement of them.
template <int M>
__device__ __forceinline__ uint32_t code_word(const float *x, float sc) {
  constexpr uint32_t kHalf = 1u << (M - 1), kTop = 2 * kHalf - 1;
  constexpr float kMagic = kRoundMagic + kHalf;
  constexpr int N = 16 / M;                      // pairs k, k + N
  uint32_t sum = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t lo = __float_as_uint(fmaf(x[k], sc, kMagic)), hi = __float_as_uint(fmaf(x[k + N], sc, kMagic));
    sum += clamp2(prmt(lo, hi, 0x5410), 0x00010001u, kTop * 0x10001u) << (M * k);
  }
  return sum ^ (M == 4 ? 0x88888888u : 0x80808080u);
}
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

}  // namespace

// A CTA takes `tokens` tokens at a time; cos and sin of their positions are
// evaluated once into shared memory and used by all heads.
// 8192 tokens of 8 heads of 128, bf16 to 4 bits: 24 us (17 without rope),
// issue slots 0.58 busy; the 43 MB read and written need 6.5.
//   VEC: a unit is two vectors of 8 values that are n/2 apart in a run of n
//   positions (n a multiple of 64): both sides of the pairs in the half
//   layout.  Four neighbouring lanes hold a block of 32 in each vector, so
//   the block maximum is two shuffles and the codes go out as words.  A
//   thread keeps one unit of a token and goes through the tokens; the table
//   holds the k-th pairs of neighbouring units side by side, which leaves no
//   bank conflict.  Otherwise one warp per block, one lane per position.
template <bool F32, int M, bool VEC>
__global__ void __launch_bounds__(kWriteThreads, 4) kv_write_kernel(WriteArgs a, const __grid_constant__ mxs_rope_plan plan) {
  extern __shared__ double2 turn[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int half = a.rope ? plan.rot >> 1 : 0;
  const bool inter = plan.layout == MXS_ROPE_INTERLEAVED;
  const int d = a.c.d, nh = a.c.n_kvh;
  const int shift = !VEC ? 0 : inter ? 2 : 3, group = 1 << shift, groups = (half + group - 1) >> shift;
  const int t_first = half ? threadIdx.x / half : 0, p_first = threadIdx.x - t_first * half;
  const int t_by = half ? kWriteThreads / half : 0, p_by = kWriteThreads - t_by * half;
  // the first unit's values of B tokens are on their way while cos and sin
  // are evaluated (two tokens', at three CTAs per SM, took the same for bf16 and 11.0 against 9.1 us for fp32)
  constexpr int B = 1, kSize = F32 ? 4 : 2;
  const int per_head = d / 16, per_token = 2 * nh * per_head;      // K units, then V units; a multiple of 8
  const int wide = min(per_token, kWriteThreads), abreast = kWriteThreads / wide;
  const int sub = threadIdx.x / wide;
  int r0 = threadIdx.x - sub * wide;
  // (each scheduler of an SM takes every fourth warp: with K first everywhere two of them would have all the turning)
  if (wide <= kWriteThreads / 2 && sub * wide >= kWriteThreads / 2) r0 = r0 < wide / 2 ? r0 + wide / 2 : r0 - wide / 2;
  Raw8<F32> fv[B], fw[B];
  int64_t fs[B];
  struct Unit {
    int isv, turned, e0, e1;                         // (turned: of K, to be turned)
    uint32_t code_at, scale_at;                      // from a slot's first byte to the head's
    const uint8_t *src;                              // of token 0
  };
  auto unit = [&](int r) {
    Unit k;
    k.isv = r >= nh * per_head;
    const int rr = r - k.isv * nh * per_head;
    const int h = rr / per_head, u = rr - h * per_head;
    // K in the half layout: the turned run, then the rest; else one run
    const int split = !k.isv && a.rope && !inter ? plan.rot : 0;
    const int run0 = u < split / 16 ? 0 : split;
    k.turned = !k.isv && a.rope && (inter || run0 == 0);
    k.e0 = run0 + 8 * (u - run0 / 16);
    k.e1 = k.e0 + (u < split / 16 ? split : d - split) / 2;
    k.code_at = h * static_cast<uint32_t>(a.c.code_pitch[k.isv]);
    k.scale_at = h * static_cast<uint32_t>(a.c.scale_pitch[k.isv]);
    k.src = static_cast<const uint8_t *>(a.src[k.isv]) + h * a.ldh[k.isv] * kSize;
    return k;
  };
  Unit un = unit(r0);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * a.tokens) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.T - t0));
    auto fetch = [&](int t) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int tb = t + b * abreast;
        fs[b] = tb < nt ? a.slot[t0 + tb] : -1;
        if (tb < nt) {                               // (also of a token without a slot: it is there)
          const uint8_t *p = un.src + (t0 + tb) * a.ldt[un.isv] * kSize;
          fv[b] = fetch8<F32>(p, un.e0);
          fw[b] = fetch8<F32>(p, un.e1);
        }
      }
    };
    if (VEC && sub < abreast) fetch(sub);
    __syncthreads();
    if (half) {
      for (int t = t_first, p = p_first; t < nt;) {
        turn[(t * group + (p & (group - 1))) * groups + (p >> shift)] =
            rope_turn(plan.step[p], plan.gain, a.pos[t0 + t], false);
        t += t_by;
        p += p_by;
        if (p >= half) {
          p -= half;
          ++t;
        }
      }
    }
    if (threadIdx.x < nt && a.slot[t0 + threadIdx.x] >= a.c.n_slots) record_bad_index(a.status);
    __syncthreads();
    if constexpr (VEC) {
      if (sub >= abreast) continue;
      const uint32_t four = 0xFu << (lane & ~3);         // the lanes of a block of 32 values
      for (int r = r0; r < per_token; r += wide) {
        if (r > r0) un = unit(r);
        for (int tt = sub; tt < nt; tt += B * abreast) {
          if (r > r0 || tt > sub) fetch(tt);
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const int t = tt + b * abreast;
            if (static_cast<uint64_t>(fs[b]) >= static_cast<uint64_t>(a.c.n_slots)) continue;   // all lanes of the block
            const uint32_t slot = static_cast<uint32_t>(fs[b]);
            float x[2][8];
            widen8<F32>(fv[b], x[0]);
            widen8<F32>(fw[b], x[1]);
            if (un.turned) {
              const double2 *cs = turn + t * group * groups;
              if (!inter) {
                cs += un.e0 / 8;
#pragma unroll
                for (int k = 0; k < 8; ++k) rope_pair(x[0][k], x[1][k], cs[k * groups]);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (un.e0 / 2 + k < half) rope_pair(x[0][2 * k], x[0][2 * k + 1], cs[k * groups + un.e0 / 8]);
                  if (un.e1 / 2 + k < half) rope_pair(x[1][2 * k], x[1][2 * k + 1], cs[k * groups + un.e1 / 8]);
                }
              }
            }
            uint32_t m[2];
#pragma unroll
            for (int side = 0; side < 2; ++side) {
              float top = 0.f;
#pragma unroll
              for (int k = 0; k < 8; k += 2) top = max3_abs(top, x[side][k], x[side][k + 1]);
              m[side] = __float_as_uint(top);
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
              m[0] = max(m[0], __shfl_xor_sync(four, m[0], o));
              m[1] = max(m[1], __shfl_xor_sync(four, m[1], o));
            }
            uint8_t *cd = a.c.codes[un.isv] + (static_cast<uint64_t>(slot) * a.c.code_slot[un.isv] + un.code_at);
            uint8_t *sd = a.c.scales[un.isv] + (static_cast<uint64_t>(slot) * a.c.scale_slot[un.isv] + un.scale_at);
            // the factors 2^(M-2-e), below 2^128 where the scale byte is M - 2 or more
            float sc[2];
#pragma unroll
            for (int side = 0; side < 2; ++side)
              sc[side] = __uint_as_float(((M - 2u + 254u) << 23) - (m[side] & 0x7F800000u));
            if (__builtin_expect(min(m[0], m[1]) < ((M - 2u) << 23), 0)) {
#pragma unroll
              for (int side = 0; side < 2; ++side) {
                const CodeScale s = code_scale<M>(m[side]);
                sc[side] = s.sc;
#pragma unroll
                for (int k = 0; k < 8; ++k) x[side][k] *= s.pre;
              }
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
              const int e = side ? un.e1 : un.e0;
              if constexpr (M == 4) {
                *reinterpret_cast<uint32_t *>(cd + e / 2) = code_word<4>(x[side], sc[side]);
              } else {
                *reinterpret_cast<uint2 *>(cd + e) =
                    make_uint2(code_word<8>(x[side], sc[side]), code_word<8>(x[side] + 4, sc[side]));
              }
              if ((lane & 3) == 0) sd[e / kBlock] = static_cast<uint8_t>(m[side] >> 23);
            }
          }
        }
        if (r + wide >= per_token && r > r0) un = unit(r0);
      }
    } else {
      const int nb = d / kBlock, per_token = 2 * nh * nb;
      for (int i = threadIdx.x >> 5; i < nt * per_token; i += kWriteThreads / 32) {
        const int t = i / per_token, r = i - t * per_token;
        const int isv = r >= nh * nb, rr = r - isv * nh * nb;
        const int h = rr / nb, b = rr - h * nb, e = b * kBlock + lane;
        const int64_t slot = a.slot[t0 + t];
        if (slot < 0 || slot >= a.c.n_slots) continue;              // the whole warp
        const int64_t si = (t0 + t) * a.ldt[isv] + h * a.ldh[isv];
        float x = load1<F32>(a.src[isv], si + e);
        if (!isv && a.rope && e < plan.rot) {
          const bool second = inter ? e & 1 : e >= half;
          const int p = inter ? e >> 1 : (second ? e - half : e);
          const int f = inter ? e ^ 1 : (second ? e - half : e + half);
          float y = load1<F32>(a.src[isv], si + f);
          if (second) {
            rope_pair(y, x, turn[t * half + p]);
          } else {
            rope_pair(x, y, turn[t * half + p]);
          }
        }
        const CodeScale s = code_scale<M>(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu));
        const uint32_t q = code_of<M>(x, s);
        const uint32_t q1 = __shfl_down_sync(0xffffffffu, q, 1);
        const int64_t row = slot * nh + h;
        uint8_t *cd = a.c.codes[isv] + row * a.c.code_pitch[isv];
        if (M == 8) cd[e] = static_cast<uint8_t>(q);
        else if ((lane & 1) == 0) cd[e / 2] = static_cast<uint8_t>(q | (q1 << 4));
        if (lane == 0) a.c.scales[isv][row * a.c.scale_pitch[isv] + b] = static_cast<uint8_t>(s.byte);
      }
    }
  }
}

namespace {

struct ReadArgs {
  CacheView c;
  void *dst[2];
  int64_t ldt[2], ldh[2];
  const int64_t *slot;
  int64_t T;
  int32_t first, count;      // which of K (0) and V (1)
  int32_t tokens;            // tokens of a CTA step
  int *status;
};

}  // namespace

// A thread keeps one place of 8 values of a token (side, head, offset) and
// goes through tokens, four at a time, so that four loads are in flight and
// the next tokens' slots are on their way; no index is divided in the loop and no
// address takes a 64-bit product.  131072 tokens of 8 heads of 128, 4 bits to
// bf16: 123 us, 0.85 of the copy rate; 150 with 64-bit products, 266 with one
// value group per grid-stride step and its division.
template <bool FOUT, int M, bool VEC>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int per_head = a.c.d / 8, per_side = per_head * a.c.n_kvh, per_token = per_side * a.count;
  const int wide = min(per_token, kReadThreads), abreast = kReadThreads / wide;
  const int sub = threadIdx.x / wide;
  if (sub >= abreast) return;
  const int64_t t_first = static_cast<int64_t>(blockIdx.x) * a.tokens, t_step = static_cast<int64_t>(gridDim.x) * a.tokens;
  constexpr int B = 4;
  for (int r = threadIdx.x - sub * wide; r < per_token; r += wide) {
    const int side = r / per_side, rr = r - side * per_side, sv = a.first + side;
    const int h = rr / per_head, e = 8 * (rr - h * per_head);
    const uint8_t *cd = a.c.codes[sv] + h * a.c.code_pitch[sv] + e * M / 8;
    const uint8_t *sd = a.c.scales[sv] + h * a.c.scale_pitch[sv] + e / kBlock;
    const uint32_t code_slot = a.c.code_slot[sv], scale_slot = a.c.scale_slot[sv];
    constexpr int kSize = FOUT ? 4 : 2;
    uint8_t *dst = static_cast<uint8_t *>(a.dst[sv]) + ((t_first + sub) * a.ldt[sv] + h * a.ldh[sv] + e) * kSize;
    const int64_t dst_next = abreast * a.ldt[sv] * kSize, dst_step = t_step * a.ldt[sv] * kSize;
    int64_t next[B];
    auto slots = [&](int64_t t0) {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t t = t0 + sub + k * abreast;
        next[k] = sub + k * abreast < a.tokens && t < a.T ? __ldg(a.slot + t) : -1;
      }
    };
    slots(t_first);
    for (int64_t t0 = t_first; t0 < a.T; t0 += t_step, dst += dst_step) {
      bool real[B];
      uint2 c[B];
      uint32_t b[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        real[k] = static_cast<uint64_t>(next[k]) < static_cast<uint64_t>(a.c.n_slots);
        if (!real[k] && next[k] >= 0) record_bad_index(a.status);
        const uint32_t slot = static_cast<uint32_t>(next[k]);
        c[k] = make_uint2(0, 0);
        b[k] = 0;
        if (!real[k]) continue;
        const uint8_t *cp = cd + static_cast<uint64_t>(slot) * code_slot;
        if constexpr (M == 4) c[k].x = *reinterpret_cast<const uint32_t *>(cp);
        else c[k] = *reinterpret_cast<const uint2 *>(cp);
        b[k] = sd[static_cast<uint64_t>(slot) * scale_slot];
      }
      if (t0 + t_step < a.T) slots(t0 + t_step);
      uint8_t *o = dst;
#pragma unroll
      for (int k = 0; k < B; ++k, o += dst_next) {
        if (!real[k]) continue;
        // 8 exact bf16 values (a fifth of the instructions of widening them one by one), put in order
        const bool mid = mid_scale<M>(b[k]);
        BlockScale<M> factors = mid_factors<M>(b[k]);
        if (!mid) factors = scale_factors<M>(min(b[k], kTopScale));
        uint4 w = decode8<M>(c[k].x, c[k].y, factors);
        if constexpr (M == 4)
          w = make_uint4(prmt(w.x, w.y, 0x5410), prmt(w.z, w.w, 0x5410), prmt(w.x, w.y, 0x7632), prmt(w.z, w.w, 0x7632));
        else
          w = make_uint4(prmt(w.x, w.y, 0x5410), prmt(w.x, w.y, 0x7632), prmt(w.z, w.w, 0x5410), prmt(w.z, w.w, 0x7632));
        float v[8];
        widen8<false>(Raw8<false>{w}, v);
        if (!mid && b[k] > kTopScale) {
          const float step = pow2f(static_cast<int>(b[k]) - 127 - M + 2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = M == 4 ? static_cast<int>(c[k].x << (28 - 4 * i)) >> 28
                                 : static_cast<int>((i < 4 ? c[k].x : c[k].y) << (24 - 8 * (i & 3))) >> 24;
            v[i] = code_to_float(q) * step;
          }
          w = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
        }
        if constexpr (VEC) {
          if constexpr (FOUT) store8<true>(o, 0, v);
          else *reinterpret_cast<uint4 *>(o) = w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) store1<FOUT>(o, i, v[i]);
        }
      }
    }
  }
}

mxs_status cache_view(const mxs_kv_cache *c, CacheView *v) {
  if (!c || c->n_kvh < 1) return MXS_ERR_ARG;
  mxs_status st;
  if ((st = check_mxtensor(&c->K)) != MXS_OK || (st = check_mxtensor(&c->V)) != MXS_OK) return st;
  const mxs_mxtensor *t[2] = {&c->K, &c->V};
  const int64_t d = c->K.lay.K;
  const int seg = c->K.lay.seg[2].k_real == d ? 2 : 0;
  if (d < kBlock || d > 256 || d % kBlock || c->n_kvh > 65535) return MXS_ERR_SHAPE;
  if (c->K.rows != c->V.rows || c->K.rows % c->n_kvh || c->K.rows > (int64_t{1} << 40)) return MXS_ERR_SHAPE;
  for (int i = 0; i < 2; ++i) {
    if (t[i]->lay.perm || t[i]->lay.K != d || t[i]->lay.seg[seg].k_real != d) return MXS_ERR_SHAPE;
    v->codes[i] = t[i]->codes[seg];
    v->scales[i] = t[i]->scales[seg];
    v->code_pitch[i] = t[i]->code_pitch[seg];
    v->scale_pitch[i] = t[i]->scale_pitch[seg];
    const __int128 cs = static_cast<__int128>(c->n_kvh) * t[i]->code_pitch[seg];
    const __int128 ss = static_cast<__int128>(c->n_kvh) * t[i]->scale_pitch[seg];
    if (cs > UINT32_MAX || ss > UINT32_MAX) return MXS_ERR_SHAPE;
    v->code_slot[i] = static_cast<uint32_t>(cs);
    v->scale_slot[i] = static_cast<uint32_t>(ss);
  }
  if (c->K.rows / c->n_kvh > INT32_MAX) return MXS_ERR_SHAPE;
  v->n_slots = c->K.rows / c->n_kvh;
  v->n_kvh = static_cast<int32_t>(c->n_kvh);
  v->d = static_cast<int32_t>(d);
  v->bits = kSegBits[seg];
  return MXS_OK;
}

namespace {

template <bool F32, int M>
void launch_write(const WriteArgs &a, const mxs_rope_plan &plan, bool vec, int grid, size_t smem, cudaStream_t s) {
  if (vec) launch_pdl(kv_write_kernel<F32, M, true>, dim3(grid), dim3(kWriteThreads), smem, s, a, plan);
  else launch_pdl(kv_write_kernel<F32, M, false>, dim3(grid), dim3(kWriteThreads), smem, s, a, plan);
}
template <bool FOUT, int M>
void launch_read(const ReadArgs &a, bool vec, int grid, cudaStream_t s) {
  if (vec) launch_pdl(kv_read_kernel<FOUT, M, true>, dim3(grid), dim3(kReadThreads), 0, s, a);
  else launch_pdl(kv_read_kernel<FOUT, M, false>, dim3(grid), dim3(kReadThreads), 0, s, a);
}

}  // namespace
}  // namespace mxs

using namespace mxs;

extern "C" mxs_status mxs_kv_write(const void *k, int64_t ldkt, int64_t ldkh, const void *v, int64_t ldvt,
                                   int64_t ldvh, mxs_dtype dt, int64_t T, const int64_t *slot, const int64_t *pos,
                                   const mxs_rope_plan *plan, const mxs_kv_cache *cache, void *stream) {
  if (T < 0) return MXS_ERR_ARG;
  if (!dtype_ok(dt)) return MXS_ERR_DTYPE;
  WriteArgs a{};
  mxs_status st = cache_view(cache, &a.c);
  if (st != MXS_OK) return st;
  if (plan && (st = check_rope_plan(plan, a.c.d)) != MXS_OK) return st;
  if (T == 0) return MXS_OK;
  if (!k || !v || !slot || (plan && !pos)) return MXS_ERR_ARG;
  if (ldkt < 0 || ldkh < 0 || ldvt < 0 || ldvh < 0) return MXS_ERR_SHAPE;
  if ((st = check_device()) != MXS_OK) return st;
  a.src[0] = k;
  a.src[1] = v;
  a.ldt[0] = ldkt;
  a.ldh[0] = ldkh;
  a.ldt[1] = ldvt;
  a.ldh[1] = ldvh;
  a.slot = slot;
  a.pos = pos;
  a.T = T;
  a.rope = plan != nullptr;
  if (!(a.status = device_status_word())) return MXS_ERR_CUDA;
  const size_t es = dtype_size(dt);
  const bool half_pairs = plan && plan->layout == MXS_ROPE_HALF;
  const bool vec = a.c.d % 64 == 0 && (!half_pairs || plan->rot % 64 == 0) && vec8_ok(k, ldkt, ldkh, es) &&
                   vec8_ok(v, ldvt, ldvh, es);
  const mxs_rope_plan none{};
  const int half = plan ? plan->rot / 2 : 0, sms = device_sms();
  // as many tokens as the threads take at once, twice where that leaves every SM several CTAs
  const int64_t per_token = 2 * static_cast<int64_t>(a.c.n_kvh) * (a.c.d / 16);
  const int64_t abreast = std::max<int64_t>(1, std::min<int64_t>(16, kWriteThreads / per_token));
  a.tokens = static_cast<int32_t>(T >= 8 * abreast * sms ? 2 * abreast : T >= abreast * sms ? abreast : 1);
  const int64_t steps = (T + a.tokens - 1) / a.tokens;
  // no more CTAs than run at once: a thread's place costs as much as coding 16 values
  const int grid = static_cast<int>(std::min<int64_t>(steps, static_cast<int64_t>(sms) * 4));
  const size_t smem = sizeof(double2) * a.tokens * ((half + 3) / 4 * 4);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const mxs_rope_plan &p = plan ? *plan : none;
  if (a.c.bits == 4) {
    if (dt == MXS_F32) launch_write<true, 4>(a, p, vec, grid, smem, s);
    else launch_write<false, 4>(a, p, vec, grid, smem, s);
  } else {
    if (dt == MXS_F32) launch_write<true, 8>(a, p, vec, grid, smem, s);
    else launch_write<false, 8>(a, p, vec, grid, smem, s);
  }
  count_launch();
  return cuda_status(cudaGetLastError());
}

extern "C" mxs_status mxs_kv_read(const mxs_kv_cache *cache, int64_t T, const int64_t *slot, void *k, int64_t ldkt,
                                  int64_t ldkh, void *v, int64_t ldvt, int64_t ldvh, mxs_dtype ot, void *stream) {
  if (T < 0) return MXS_ERR_ARG;
  if (!dtype_ok(ot)) return MXS_ERR_DTYPE;
  ReadArgs a{};
  mxs_status st = cache_view(cache, &a.c);
  if (st != MXS_OK) return st;
  if (T == 0) return MXS_OK;
  if (!slot || (!k && !v)) return MXS_ERR_ARG;
  a.dst[0] = k;
  a.dst[1] = v;
  a.ldt[0] = ldkt;
  a.ldh[0] = ldkh;
  a.ldt[1] = ldvt;
  a.ldh[1] = ldvh;
  a.slot = slot;
  a.T = T;
  a.first = k ? 0 : 1;
  a.count = (k != nullptr) + (v != nullptr);
  bool vec = true;
  for (int i = 0; i < 2; ++i) {
    if (!a.dst[i]) continue;
    // the rows of the output must not overlap
    if (a.ldh[i] < a.c.d || a.ldt[i] < a.c.d ||
        (a.ldt[i] < static_cast<__int128>(a.ldh[i]) * (a.c.n_kvh - 1) + a.c.d &&
         a.ldh[i] < static_cast<__int128>(a.ldt[i]) * (T - 1) + a.c.d))
      return MXS_ERR_SHAPE;
    vec = vec && vec8_ok(a.dst[i], a.ldt[i], a.ldh[i], dtype_size(ot));
  }
  if ((st = check_device()) != MXS_OK) return st;
  if (!(a.status = device_status_word())) return MXS_ERR_CUDA;
  // four tokens for every thread, fewer while that leaves SMs without work
  const int sms = device_sms();
  const int64_t per_token = static_cast<int64_t>(a.count) * a.c.n_kvh * (a.c.d / 8);
  const int64_t abreast = std::max<int64_t>(1, kReadThreads / per_token);
  a.tokens = static_cast<int32_t>(abreast * std::max<int64_t>(1, std::min<int64_t>(4, T / (abreast * 2 * sms))));
  const int grid = static_cast<int>(std::min<int64_t>((T + a.tokens - 1) / a.tokens, static_cast<int64_t>(sms) * 8));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.c.bits == 4) {
    if (ot == MXS_F32) launch_read<true, 4>(a, vec, grid, s);
    else launch_read<false, 4>(a, vec, grid, s);
  } else {
    if (ot == MXS_F32) launch_read<true, 8>(a, vec, grid, s);
    else launch_read<false, 8>(a, vec, grid, s);
  }
  count_launch();
  return cuda_status(cudaGetLastError());
}
