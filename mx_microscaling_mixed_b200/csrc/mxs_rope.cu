// mxs_rope.cu -- rotary positions: the plan (host) and the kernel.
//
// y_u = x_u cos a - x_v sin a, y_v = x_v cos a + x_u sin a for the pairs
// (u, v) of a head's first `rot` positions, a = pos * f.
#include <algorithm>
#include <cmath>

#include "mxs_rope.cuh"

namespace mxs {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const void *x;
  void *out;
  const int64_t *pos;
  int64_t T, ldxt, ldxh, ldot, ldoh;
  int32_t heads, d, inverse, tokens;     // tokens per CTA step
};

}  // namespace

// A CTA takes `tokens` tokens at a time: it evaluates their cos and sin once
// into shared memory, where all heads find them.  A thread keeps one work
// unit of a token (head and place in it) and goes through the tokens, so the
// unit's place is worked out once.  VEC: a unit is 8 values of a head (in the
// half layout, 8 values of each side of the pairs), and the table holds the
// k-th pairs of neighbouring units side by side: a unit's reads of it meet no
// bank conflict (stored pair by pair they took 72 us for 8192 tokens of 32
// heads of 128, bf16, where the 134 MB of x and y need 20).  Otherwise a unit
// is one pair or one copied value.
template <bool FIN, bool FOUT, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(RopeArgs a, const __grid_constant__ mxs_rope_plan plan) {
  extern __shared__ double2 turn[];
  pdl_wait();
  pdl_trigger();
  const int half = plan.rot >> 1;
  const bool inter = plan.layout == MXS_ROPE_INTERLEAVED;
  const int step = VEC ? 8 : 1;
  const int shift = !VEC ? 0 : inter ? 2 : 3, group = 1 << shift;    // pairs of a unit
  // units of a head: turned ones first, then copied ones
  const int turned = (half + group - 1) >> shift;
  const int first_copied = VEC && inter ? turned * 8 : plan.rot;
  const int per_head = turned + (a.d - first_copied) / step;
  const int per_token = per_head * a.heads;
  const int wide = min(per_token, kRopeThreads);
  const int abreast = kRopeThreads / wide;               // tokens that the CTA's threads take at once
  const int sub = threadIdx.x / wide, r0 = threadIdx.x - sub * wide;
  const int t_first = threadIdx.x / half, p_first = threadIdx.x - t_first * half;
  const int t_by = kRopeThreads / half, p_by = kRopeThreads - t_by * half;
  const int h0 = r0 / per_head;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * a.tokens) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.T - t0));
    // a unit's values of B tokens are on their way while cos and sin are
    // evaluated, turned and copied units alike (twice as many, at three CTAs
    // per SM, took 30.3 us where these take 29.3)
    constexpr int B = FIN ? 1 : 2;
    Raw8<FIN> v[B], w[B];
    auto fetch = [&](int h, int u, int t) {
      const int e = u < turned ? u * 8 : first_copied + (u - turned) * 8;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int tb = t + b * abreast;
        const int64_t xi = (t0 + tb) * a.ldxt + h * a.ldxh + e;
        if (tb < nt) v[b] = fetch8<FIN>(a.x, xi);
        if (tb < nt && u < turned && !inter) w[b] = fetch8<FIN>(a.x, xi + half);
      }
    };
    if (VEC && sub < abreast) fetch(h0, r0 - h0 * per_head, sub);
    __syncthreads();
    for (int t = t_first, p = p_first; t < nt;) {
      turn[(t * group + (p & (group - 1))) * turned + (p >> shift)] =
          rope_turn(plan.step[p], plan.gain, a.pos[t0 + t], a.inverse);
      t += t_by;
      p += p_by;
      if (p >= half) {
        p -= half;
        ++t;
      }
    }
    __syncthreads();
    if (sub >= abreast) continue;
    for (int r = r0; r < per_token; r += wide) {
      const int h = r == r0 ? h0 : r / per_head, u = r - h * per_head;
      const bool turns = u < turned;
      if constexpr (VEC) {
        const int e = turns ? u * 8 : first_copied + (u - turned) * 8;
        const bool two = turns && !inter;
        for (int t = sub; t < nt; t += B * abreast) {
          if (r > r0 || t > sub) fetch(h, u, t);
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const int tb = t + b * abreast;
            if (tb >= nt) break;
            const double2 *cs = turn + tb * group * turned + u;
            const int64_t oi = (t0 + tb) * a.ldot + h * a.ldoh + e;
            float x[8], y[8];
            widen8<FIN>(v[b], x);
            if (two) {
              widen8<FIN>(w[b], y);
#pragma unroll
              for (int k = 0; k < 8; ++k) rope_pair(x[k], y[k], cs[k * turned]);
              store8<FOUT>(a.out, oi + half, y);
            } else if (turns) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (e / 2 + k < half) rope_pair(x[2 * k], x[2 * k + 1], cs[k * turned]);
            }
            store8<FOUT>(a.out, oi, x);
          }
        }
      } else {
        for (int t = sub; t < nt; t += abreast) {
          const int64_t xi = (t0 + t) * a.ldxt + h * a.ldxh, oi = (t0 + t) * a.ldot + h * a.ldoh;
          if (!turns) {
            const int e = plan.rot + u - turned;
            store1<FOUT>(a.out, oi + e, load1<FIN>(a.x, xi + e));
          } else {
            const int e = inter ? 2 * u : u, f = inter ? e + 1 : e + half;
            float v = load1<FIN>(a.x, xi + e), w = load1<FIN>(a.x, xi + f);
            rope_pair(v, w, turn[t * turned + u]);
            store1<FOUT>(a.out, oi + e, v);
            store1<FOUT>(a.out, oi + f, w);
          }
        }
      }
    }
  }
}

namespace {

template <bool FIN, bool FOUT>
void launch_rope(const RopeArgs &a, const mxs_rope_plan &plan, bool vec, int grid, size_t smem, cudaStream_t s) {
  if (vec) launch_pdl(rope_kernel<FIN, FOUT, true>, dim3(grid), dim3(kRopeThreads), smem, s, a, plan);
  else launch_pdl(rope_kernel<FIN, FOUT, false>, dim3(grid), dim3(kRopeThreads), smem, s, a, plan);
}

}  // namespace

int device_sms() {
  int dev = 0, n = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

mxs_status check_rope_plan(const mxs_rope_plan *plan, int64_t d) {
  if (!plan || plan->rot < 2 || plan->rot > 2 * MXS_ROPE_MAX_PAIRS || plan->rot % 2 ||
      (plan->layout != MXS_ROPE_HALF && plan->layout != MXS_ROPE_INTERLEAVED) || !std::isfinite(plan->gain))
    return MXS_ERR_ARG;
  return plan->rot <= d ? MXS_OK : MXS_ERR_SHAPE;
}

}  // namespace mxs

using namespace mxs;

extern "C" mxs_status mxs_rope_plan_make(int32_t rot, int32_t layout, double theta, const mxs_rope_scaling *scaling,
                                         mxs_rope_plan *out) {
  if (!out || rot < 2 || rot > 2 * MXS_ROPE_MAX_PAIRS || rot % 2) return MXS_ERR_ARG;
  if (layout != MXS_ROPE_HALF && layout != MXS_ROPE_INTERLEAVED) return MXS_ERR_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta)) return MXS_ERR_ARG;
  const int kind = scaling ? scaling->kind : MXS_ROPE_PLAIN;
  if (kind < MXS_ROPE_PLAIN || kind > MXS_ROPE_YARN) return MXS_ERR_ARG;
  if (kind != MXS_ROPE_PLAIN && (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor))) return MXS_ERR_ARG;
  const bool blend = kind == MXS_ROPE_PARTS || kind == MXS_ROPE_YARN;
  if (blend && (!(scaling->low > 0.0) || !(scaling->high > scaling->low) || !std::isfinite(scaling->high) ||
                scaling->orig_len < 1))
    return MXS_ERR_ARG;
  // long double throughout (a relative error of a few 2^-64), then one rounding to 2^-64 turns
  const long double two_pi = 6.283185307179586476925286766559005768L;
  const long double th = theta, factor = blend || kind == MXS_ROPE_LINEAR ? scaling->factor : 1.0;
  long double a = 0, b = 0;
  if (kind == MXS_ROPE_YARN) {
    const long double per = rot / (2.0L * logl(th)), len = static_cast<long double>(scaling->orig_len);
    a = std::max(0.0L, floorl(per * logl(len / (two_pi * scaling->high))));
    b = std::min<long double>(rot - 1, ceill(per * logl(len / (two_pi * scaling->low))));
  }
  out->rot = rot;
  out->layout = layout;
  out->gain = kind == MXS_ROPE_YARN ? 0.1 * std::log(scaling->factor) + 1.0 : 1.0;
  for (int i = 0; i < MXS_ROPE_MAX_PAIRS; ++i) {
    out->step[i] = 0;
    if (i >= rot / 2) continue;
    const long double w = powl(th, -2.0L * i / rot);
    long double keep = 1.0L;
    if (kind == MXS_ROPE_LINEAR) keep = 0.0L;
    if (kind == MXS_ROPE_PARTS)
      keep = (scaling->orig_len * w / two_pi - scaling->low) / (static_cast<long double>(scaling->high) - scaling->low);
    if (kind == MXS_ROPE_YARN) keep = 1.0L - std::min(1.0L, std::max(0.0L, (i - a) / std::max(0.001L, b - a)));
    keep = std::min(1.0L, std::max(0.0L, keep));
    const long double f = w * (keep + (1.0L - keep) / factor);
    out->step[i] = static_cast<uint64_t>(roundl(f / two_pi * 0x1p64L));
  }
  return MXS_OK;
}

extern "C" mxs_status mxs_rope(const void *x, mxs_dtype xt, int64_t T, int64_t heads, int64_t d, int64_t ldxt,
                               int64_t ldxh, const int64_t *pos, const mxs_rope_plan *plan, int32_t inverse, void *out,
                               mxs_dtype ot, int64_t ldot, int64_t ldoh, void *stream) {
  if (T < 0 || heads < 0 || d < 0 || !plan) return MXS_ERR_ARG;
  if (!dtype_ok(xt) || !dtype_ok(ot)) return MXS_ERR_DTYPE;
  if (d < 2 || d > 2 * MXS_ROPE_MAX_PAIRS || d % 2 || heads > 65536) return MXS_ERR_SHAPE;
  mxs_status st = check_rope_plan(plan, d);
  if (st != MXS_OK) return st;
  if (T == 0 || heads == 0) return MXS_OK;
  if (!x || !pos || !out) return MXS_ERR_ARG;
  // strides: any on the input; the output's rows must not overlap
  if (ldxt < 0 || ldxh < 0 || ldot < 0 || ldoh < 0) return MXS_ERR_SHAPE;
  const bool token_major = ldoh >= d && ldot >= static_cast<__int128>(ldoh) * (heads - 1) + d;
  const bool head_major = ldot >= d && ldoh >= static_cast<__int128>(ldot) * (T - 1) + d;
  if (!(token_major || head_major || (heads == 1 && ldot >= d) || (T == 1 && ldoh >= d) || (heads == 1 && T == 1)))
    return MXS_ERR_SHAPE;
  if (x == out && (xt != ot || ldxt != ldot || ldxh != ldoh)) return MXS_ERR_SHAPE;
  if ((st = check_device()) != MXS_OK) return st;

  const int half = plan->rot / 2;
  const bool vec = vec8_ok(x, ldxt, ldxh, dtype_size(xt)) && vec8_ok(out, ldot, ldoh, dtype_size(ot)) && d % 8 == 0 &&
                   (plan->layout == MXS_ROPE_INTERLEAVED || half % 8 == 0);
  RopeArgs a{};
  a.x = x;
  a.out = out;
  a.pos = pos;
  a.T = T;
  a.ldxt = ldxt;
  a.ldxh = ldxh;
  a.ldot = ldot;
  a.ldoh = ldoh;
  a.heads = static_cast<int32_t>(heads);
  a.d = static_cast<int32_t>(d);
  a.inverse = inverse != 0;
  const int sms = device_sms();
  // as many tokens a step as a thread has in flight, one where there are few
  const int64_t units = heads * (vec ? (plan->layout == MXS_ROPE_HALF ? (d - half) / 8 : d / 8) : d - half);
  const int64_t abreast = std::max<int64_t>(1, kRopeThreads / units);
  const int64_t most = std::min<int64_t>(abreast * (xt == MXS_F32 ? 2 : 4), 2048 / std::max(half, 8));
  a.tokens = static_cast<int32_t>(T >= 4 * sms * most ? most : std::max<int64_t>(1, std::min(most, T / (2 * sms))));
  const int64_t steps = (T + a.tokens - 1) / a.tokens;
  const int grid = static_cast<int>(std::min<int64_t>(steps, static_cast<int64_t>(sms) * 8));
  const size_t smem = sizeof(double2) * a.tokens * ((half + 3) / 4 * 4);    // (interleaved units: whole groups of 4 pairs)
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fi = xt == MXS_F32, fo = ot == MXS_F32;
  if (fi && fo) launch_rope<true, true>(a, *plan, vec, grid, smem, s);
  else if (fi) launch_rope<true, false>(a, *plan, vec, grid, smem, s);
  else if (fo) launch_rope<false, true>(a, *plan, vec, grid, smem, s);
  else launch_rope<false, false>(a, *plan, vec, grid, smem, s);
  count_launch();
  return cuda_status(cudaGetLastError());
}
