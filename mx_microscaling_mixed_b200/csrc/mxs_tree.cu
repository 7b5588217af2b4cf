// mxs_tree.cu -- attention of drafted tokens (trees or chains) over the paged
// MXINT K/V cache.
//
//   s_p = sm_scale q . K_p,   out = sum_p softmax(s)_p V_p,
//   lse = ln sum_p e^(s_p)
// over the tokens a row sees: the whole context and the drafted tokens that
// its mask names.
#include <algorithm>
#include <cmath>

#include "mxs_cache.cuh"
#include "mxs_ptx.cuh"

namespace mxs {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
  const uint16_t *q;
  int64_t ldqt, ldqh;
  CacheView c;
  const int32_t *q_start, *length, *pages;
  int64_t ldp, rows, ldm;
  const uint32_t *mask;
  uint32_t page_size, page_mul, page_shift;
  int32_t B, n_qh, rep, max_q, max_len;
  float scale_log2;
  void *out;
  int64_t ldot, ldoh;
  float *lse;
  int *status;
};

struct Sequence {
  int first, n, ctx;       // first row, drafted tokens, context tokens; n = 0 where the sequence is left out
};

__device__ __forceinline__ Sequence sequence_of(const TreeArgs &a, int b, bool report) {
  Sequence s;
  s.first = a.q_start[b];
  const int64_t n = static_cast<int64_t>(a.q_start[b + 1]) - s.first;
  s.ctx = a.length[b];
  const bool bad = n < 0 || n > a.max_q || s.ctx < 0 || s.ctx + n > a.max_len || s.first < 0 || s.first + n > a.rows;
  if (bad && report) record_bad_index(a.status);
  s.n = bad ? 0 : static_cast<int>(n);
  return s;
}

// p / page_size for 0 <= p < 2^31.
__device__ __forceinline__ uint32_t page_of(const TreeArgs &a, uint32_t p) {
  return a.page_mul ? __umulhi(p, a.page_mul) >> a.page_shift : p;
}
// Slot of token p of sequence b, or -1 where its page is outside the pool.
__device__ __forceinline__ int64_t slot_of(const TreeArgs &a, int b, int p) {
  const uint32_t pg = page_of(a, p);
  const int page = a.pages[b * a.ldp + pg];
  const int64_t s = static_cast<int64_t>(page) * a.page_size + (p - pg * a.page_size);
  const bool ok = page >= 0 && s < a.c.n_slots;
  if (!ok) record_bad_index(a.status);
  return ok ? s : -1;
}

}  // namespace

// One CTA per (drafted token, query head): four warps take the tokens in
// turn, each with its own running maximum, sum and output.
template <int D, int M, bool FOUT>
__global__ void __launch_bounds__(128) tree_simple_kernel(TreeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int b = blockIdx.y, i = blockIdx.x / a.n_qh, h = blockIdx.x - i * a.n_qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Sequence sq = sequence_of(a, b, blockIdx.x == 0 && threadIdx.x == 0);
  if (i >= sq.n) return;
  const int g = h / a.rep, r = sq.first + i;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_bits_to_float(a.q[r * a.ldqt + h * a.ldqh + lane * E + e]);
    o[e] = 0.f;
  }
  for (int p = warp; p < sq.ctx + sq.n; p += 4) {
    const int j = p - sq.ctx;
    if (j >= 0 && !(a.mask ? (a.mask[r * a.ldm + (j >> 5)] >> (j & 31)) & 1 : j <= i)) continue;
    const int64_t slot = slot_of(a, b, p);
    if (slot < 0) continue;
    const int64_t row = slot * a.c.n_kvh + g;
    float kv[2][E];
#pragma unroll
    for (int sv = 0; sv < 2; ++sv) {
      const uint32_t sb = a.c.scales[sv][row * a.c.scale_pitch[sv] + lane * E / kBlock];
      const float step = pow2f(static_cast<int>(min(sb, 249u)) - 127 - M + 2);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = lane * E + e;
        const uint8_t *c = a.c.codes[sv] + row * a.c.code_pitch[sv];
        const int code = M == 8 ? static_cast<int8_t>(c[at]) : (static_cast<int>(c[at >> 1]) << (28 - 4 * (at & 1))) >> 28;
        kv[sv][e] = code * step;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kv[0][e], s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, w * kv[1][e]);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  const float M4 = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float total = 0.f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M4);
    total += f[w] * sl[w];
  }
  for (int e = threadIdx.x; e < D; e += 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += f[w] * so[w][e];
    v = total > 0.f ? v / total : total == 0.f ? 0.f : total;
    const int64_t at = r * a.ldot + h * a.ldoh + e;
    if constexpr (FOUT) static_cast<float *>(a.out)[at] = v;
    else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16(v);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<int64_t>(r) * a.n_qh + h] = total == 0.f ? -INFINITY : (M4 + log2f(total)) * kLn2;
}

namespace {

// Host checks that need no device; fills the shape part of *a.
mxs_status tree_check(const mxs_kv_cache *cache, const mxs_tree_batch *t, int64_t n_qh, TreeArgs *a) {
  if (!cache || !t) return MXS_ERR_ARG;
  mxs_status st = cache_view(cache, &a->c);
  if (st != MXS_OK) return st;
  if (t->B < 0 || t->rows < 0 || t->max_q < 0 || t->max_len < 0 || n_qh < 1) return MXS_ERR_ARG;
  if ((a->c.d != 64 && a->c.d != 128) || n_qh % a->c.n_kvh || n_qh > 65535) return MXS_ERR_SHAPE;
  if (t->B > 65535 || t->rows > INT32_MAX || t->max_len > INT32_MAX - 1024 || t->max_q > t->max_len ||
      t->max_q > INT32_MAX / n_qh)
    return MXS_ERR_SHAPE;
  if (t->page_size < 1 || t->page_size > INT32_MAX || t->ldp < 0 || t->ldp > INT32_MAX ||
      t->ldp * t->page_size < t->max_len)
    return MXS_ERR_SHAPE;
  if (t->mask && (t->ldm < 0 || t->ldm > INT32_MAX || t->ldm * 32 < t->max_q)) return MXS_ERR_SHAPE;
  a->q_start = t->q_start;
  a->length = t->length;
  a->pages = t->pages;
  a->ldp = t->ldp;
  a->rows = t->rows;
  a->mask = t->mask;
  a->ldm = t->ldm;
  a->B = static_cast<int32_t>(t->B);
  a->max_q = static_cast<int32_t>(t->max_q);
  a->max_len = static_cast<int32_t>(t->max_len);
  a->n_qh = static_cast<int32_t>(n_qh);
  a->rep = static_cast<int32_t>(n_qh / a->c.n_kvh);
  // p / page_size = (p * ceil(2^(31+l) / page_size)) >> (31 + l) for p < 2^31, l = ceil(log2 page_size)
  a->page_size = static_cast<uint32_t>(t->page_size);
  a->page_mul = a->page_shift = 0;
  if (t->page_size > 1) {
    int l = 1;
    while ((int64_t{1} << l) < t->page_size) ++l;
    const uint64_t ps = static_cast<uint64_t>(t->page_size);
    a->page_mul = static_cast<uint32_t>(((uint64_t{1} << (31 + l)) + ps - 1) / ps);
    a->page_shift = static_cast<uint32_t>(l - 1);
  }
  return MXS_OK;
}

template <int D, int M>
void launch_simple(const TreeArgs &a, bool fout, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.max_q) * a.n_qh, static_cast<unsigned>(a.B));
  if (fout) launch_pdl(tree_simple_kernel<D, M, true>, grid, dim3(128), 0, s, a);
  else launch_pdl(tree_simple_kernel<D, M, false>, grid, dim3(128), 0, s, a);
}

}  // namespace
}  // namespace mxs

using namespace mxs;

extern "C" mxs_status mxs_attn_tree_workspace_bytes(const mxs_kv_cache *cache, const mxs_tree_batch *batch,
                                                    int64_t n_qh, size_t *bytes) {
  if (!bytes) return MXS_ERR_ARG;
  TreeArgs a{};
  const mxs_status st = tree_check(cache, batch, n_qh, &a);
  if (st != MXS_OK) return st;
  *bytes = 0;
  return MXS_OK;
}

extern "C" mxs_status mxs_attn_tree(const void *q, int64_t n_qh, int64_t ldqt, int64_t ldqh, const mxs_kv_cache *cache,
                                    const mxs_tree_batch *batch, float sm_scale, void *out, mxs_dtype ot,
                                    int64_t ldot, int64_t ldoh, float *lse, void *ws, size_t ws_bytes, void *stream) {
  TreeArgs a{};
  mxs_status st = tree_check(cache, batch, n_qh, &a);
  if (st != MXS_OK) return st;
  if (!dtype_ok(ot)) return MXS_ERR_DTYPE;
  if (!std::isfinite(sm_scale)) return MXS_ERR_ARG;
  if (batch->B == 0 || batch->max_q == 0 || batch->rows == 0) return MXS_OK;
  if (!q || !out || !a.q_start || !a.length || !a.pages) return MXS_ERR_ARG;
  const int64_t d = a.c.d;
  if (ldqt < 0 || ldqh < 0 || ldot < d || ldoh < d ||
      (ldot < static_cast<__int128>(ldoh) * (n_qh - 1) + d && ldoh < static_cast<__int128>(ldot) * (batch->rows - 1) + d))
    return MXS_ERR_SHAPE;
  if (!aligned16(q) || ldqt % 8 || ldqh % 8) return MXS_ERR_ALIGN;
  (void)ws;
  (void)ws_bytes;
  if ((st = check_device()) != MXS_OK) return st;
  if (!(a.status = device_status_word())) return MXS_ERR_CUDA;
  a.q = static_cast<const uint16_t *>(q);
  a.ldqt = ldqt;
  a.ldqh = ldqh;
  a.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  a.out = out;
  a.ldot = ldot;
  a.ldoh = ldoh;
  a.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f = ot == MXS_F32;
  if (d == 64 && a.c.bits == 4) launch_simple<64, 4>(a, f, s);
  else if (d == 64) launch_simple<64, 8>(a, f, s);
  else if (a.c.bits == 4) launch_simple<128, 4>(a, f, s);
  else launch_simple<128, 8>(a, f, s);
  count_launch();
  return cuda_status(cudaGetLastError());
}
