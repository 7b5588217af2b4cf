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
#include "mxs_rope.cuh"

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
  int32_t row_tiles, splits, tiles_per_split;
  float *part, *part_lse;  // the splits' normalised outputs and base-2 lse: [split][row][head]([D])
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

}  // namespace

// ---------------------------------------------------------------- kernel
namespace {

constexpr int kTile = 128;                       // tokens of a tile
constexpr int kPeriod = 8;                       // tiles
constexpr int kAtom = kTile * 128;               // 64 bf16 values of each token of a tile
constexpr float kSlack = 24.f;                   // weights are kept below 2^kSlack
constexpr long long kTreeWait = 2000000000LL;    // cycles (about 1 s)

// R columns (query rows) per CTA; P bf16 pieces of a weight.
template <int D, int M, int R, int P>
struct Shape {
  static constexpr int kCols = R < 32 ? R : 32;          // columns of a softmax warp
  static constexpr int kSoftWarps = R / kCols * 4;
  static constexpr int kResident = R > 32 || (R == 32 && P > 1 && D > 64) ? 1 : 2;
  static constexpr int kDecodeWarps = kResident == 1 ? 8 : 4;    // 8: four for K, four for V
  static constexpr int kThreads = (kSoftWarps + kDecodeWarps) * 32;
  static constexpr int kN = R * P;                       // columns of the output product
  static constexpr int kKV = kTile * D * 2;
  static constexpr int kStages = kResident == 1 && R * P < 192 ? 2 : 1;    // of K and of V
  static constexpr int kPWidth = R < 64 ? R : 64;        // columns in a row of a swizzle atom of the weights
  static constexpr int kPAtom = kTile * kPWidth * 2;
  static constexpr int kPBytes = kTile * kN * 2;
  static constexpr int kPBufs = 2;
  static constexpr int kK = 0, kV = kStages * kKV, kP = 2 * kStages * kKV, kQ = kP + kPBufs * kPBytes;
  static constexpr int kAcc = kQ + R * D * 2;            // fp32 sums of output periods, [column][place]
  static constexpr int kStat = kAcc + (P > 1 ? R * D * 4 : 0);   // per column: reference, factor, 4 maxima or sums
  static constexpr int kPlace = kStat + 6 * R * 4;       // per column: where its output goes (64 bits)
  static constexpr int kBar = kPlace + R * 8;
  static constexpr int kBars = kBar + (2 * kStages + 8) * 8 + 16;
  // (heads of 64: the output product reads 64 places that nobody uses behind V's, which have to exist)
  static constexpr int kEnd = kBars > kV + kStages * kKV + kAtom ? kBars : kV + kStages * kKV + kAtom;
  static constexpr int kBytes = kEnd + 1024;
  static constexpr int kTmem = 2 * R + kN <= 64 ? 64 : 2 * R + kN <= 128 ? 128 : 2 * R + kN <= 256 ? 256 : 512;
  static_assert(kResident * (kBytes + 1024) <= 228 * 1024 && kResident * kTmem <= 512, "the CTAs of an SM fit it");
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kTile >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | (static_cast<uint32_t>(R >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (3u << 15) | (static_cast<uint32_t>(kN >> 3) << 17);
};

// Waits for a barrier's phase; gives up when the limit ran out or another
// role has given up.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *given_up, int *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*given_up) return false;
    if (clock64() - t0 > kTreeWait) {
      *given_up = 1;
      atomicExch(status, static_cast<int>(MXS_ERR_TIMEOUT));
      return false;
    }
  }
  return true;
}
// Among the 128 threads of a softmax warpgroup: does any of them say so?
__device__ __forceinline__ bool any_of(int group, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(group + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}
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
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 load_stream(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
// (4 bits) or 0 2 1 3 of each word (8 bits); q and the output follow it.
template <int M>
struct BlockScale {
  uint32_t s, c, s16;
  __device__ __forceinline__ explicit BlockScale(uint32_t b) {
    b = min(b, 249u);                            // above, -136 s leaves bf16's range
    if constexpr (M == 4) {
      s = step4(b) * 0x10001u;
      c = (0x8000u | ((b + 5u) << 7) | 8u) * 0x10001u;
      s16 = 0;
    } else {
      s = step8(b) * 0x10001u;
      s16 = step4(b) * 0x10001u;
      c = (0x8000u | ((b + 5u) << 7) | 16u) * 0x10001u;
    }
  }
};
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
// The same order for 8 values of q.
template <int M>
__device__ __forceinline__ uint4 reorder8(uint4 w) {
  if constexpr (M == 4)
    return make_uint4(prmt(w.x, w.z, 0x5410), prmt(w.x, w.z, 0x7632), prmt(w.y, w.w, 0x5410), prmt(w.y, w.w, 0x7632));
  else
    return make_uint4(prmt(w.x, w.y, 0x5410), prmt(w.x, w.y, 0x7632), prmt(w.z, w.w, 0x5410), prmt(w.z, w.w, 0x7632));
}
template <int M>
__device__ __forceinline__ int true_position(int e) {
  if constexpr (M == 4) return (e & ~7) | ((e & 7) >> 1) | ((e & 1) << 2);
  else return (e & ~3) | ((e & 3) >> 1) | ((e & 1) << 1);
}

// What a row tile of a sequence covers: its rows are (drafted token i, head
// h of the group) = (row / rep, row % rep) for rows row0 .. row0 + R - 1.
struct TileRange {
  int total;      // tokens that any of its rows can see
  int open;       // tokens below this are seen by all of them
};
__device__ __forceinline__ TileRange tile_range(const TreeArgs &a, const Sequence &sq, int row0, int R) {
  TileRange r;
  if (a.mask) {
    r.total = sq.ctx + sq.n;
    r.open = sq.ctx;
  } else {
    r.total = sq.ctx + min(sq.n, (row0 + R - 1) / a.rep + 1);
    r.open = sq.ctx + min(sq.n, row0 / a.rep + 1);
  }
  return r;
}

// Sum or maximum of v[k] over the lanes, for each of the N columns k at once:
// every step halves the columns a lane holds.  Lane l is left with column
// l * N / 32, in v[0].
template <int N, typename Op>
__device__ __forceinline__ float over_lanes(float (&v)[N], int lane, Op op) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

// Which of 32 tokens, from drafted token j0 on (negative: the context), row i
// of a sequence sees, one bit each.
__device__ __forceinline__ uint32_t seen_tokens(const TreeArgs &a, const Sequence &sq, int i, int j0) {
  if (i >= sq.n) return 0;
  const int limit = a.mask ? sq.n - j0 : i + 1 - j0;     // tokens up to the last that can be seen
  uint32_t w = 0xFFFFFFFFu;
  if (a.mask && j0 > -32) {
    const uint32_t *m = a.mask + (sq.first + i) * a.ldm;
    if (j0 < 0) {
      w = (m[0] << -j0) | ((1u << -j0) - 1u);
    } else {
      const int k = j0 >> 5, words = (sq.n + 31) >> 5;
      w = __funnelshift_r(k < words ? m[k] : 0u, k + 1 < words ? m[k + 1] : 0u, j0 & 31);
    }
  }
  return limit >= 32 ? w : limit <= 0 ? 0u : w & ((1u << limit) - 1u);
}

}  // namespace

// CTA = (sequence, kv head, split of the tokens, row tile).  Tokens are the
// 128 rows of the matrix instruction, query rows its columns, so that the
// work follows the number of rows (16 to 64 of them) while a cache tile is
// decoded once for all of them:
//   S^T [token][row] = K Q^T     A = K  (token x d, K-major),  B = Q
//   O^T [d][row]    += V^T P^T   A = V  (token x d, stored along d), B = P
// Both accumulate in tensor memory.  Four or eight warps fetch and decode the
// cache into shared memory, the first of K's and of V's issues the products;
// four or eight turn scores into weights.  A softmax thread owns one token
// and sums its weights per row over all tiles; the sums meet at the end.
//   The running maximum of a row is a reference that weights are relative
// to, common to all tokens: it is set by the first tile and moved only when
// a score passes it by more than 24 (weights of 2^24), which fp32 and bf16 hold with no loss
// of precision; so a tile usually needs no maximum over its tokens, only one
// vote that none of its scores is above.
//   The tensor core's fp32 sums are rounded towards zero at every step: an
// fp32 output is taken out of tensor memory every kPeriod tiles and summed
// outside it.
template <int D, int M, int R, int P, bool FOUT>
__global__ void __launch_bounds__(Shape<D, M, R, P>::kThreads, Shape<D, M, R, P>::kResident) tree_kernel(TreeArgs a) {
  using S = Shape<D, M, R, P>;
  constexpr int NS = S::kStages, C = S::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *ref = reinterpret_cast<float *>(smem + S::kStat), *factor = ref + R, *wstat = factor + R;   // wstat[4][R]
  int64_t *place = reinterpret_cast<int64_t *>(smem + S::kPlace);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::kBar);
  uint64_t *s_done = bar, *p_full = bar + 2, *o_done = bar + 4, *drained = bar + 6, *k_full = bar + 8, *v_full = k_full + NS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(v_full + NS);
  volatile int *given_up = reinterpret_cast<int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  int x = blockIdx.x;
  const int rt = x % a.row_tiles;
  x /= a.row_tiles;
  const int sp = x % a.splits;
  x /= a.splits;
  const int g = x % a.c.n_kvh, b = x / a.c.n_kvh;
  const Sequence sq = sequence_of(a, b, rt == 0 && sp == 0 && g == 0 && threadIdx.x == 0);
  const int row0 = rt * R;
  const TileRange range = tile_range(a, sq, row0, R);
  const int tile0 = sp * a.tiles_per_split;
  const int nt = min(a.tiles_per_split, (range.total + kTile - 1) / kTile - tile0);
  if (row0 >= sq.n * a.rep || (nt <= 0 && sp > 0)) {       // (split 0 writes the rows of an empty range)
    pdl_trigger();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(k_full + i, 4 * 32);
      ptx::mbar_init(v_full + i, 4 * 32);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_done + i, 1);
      ptx::mbar_init(p_full + i, S::kSoftWarps * 32);
      ptx::mbar_init(o_done + i, 1);
      ptx::mbar_init(drained + i, 1);
    }
    ptx::fence_mbar_init();
    *given_up = 0;
  }
  for (int i = threadIdx.x; i < R; i += S::kThreads) ref[i] = -INFINITY;
  // tensor memory is taken after the wait for earlier kernels and before
  // later ones may start: a CTA that waits for another kernel holds none
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, S::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + 2 * R;
  const uint32_t sbase = ptx::smem_addr(smem);

  if (warp >= S::kSoftWarps) {
    // ------------------------------------ fetching, decoding, and the products
    // Jobs are (tile, K or V): with four warps alternately K and V, with
    // eight one of them per group.  Two jobs are on their way in registers.
    constexpr bool kBoth = S::kDecodeWarps == 4;
    constexpr int BL = D / kBlock;                   // blocks of a cache row
    constexpr int kRows = 32 / BL;                   // rows per iteration of a warp
    constexpr int kIt = 32 / kRows;
    const int dw = warp - S::kSoftWarps, w = dw & 3;
    const int own = dw >> 2;                         // (eight warps) 0: K, 1: V
    const int q4 = lane >> 3, blk = q4 % BL;
    const int row_in = w * 32 + (q4 / BL) * 8 + (lane & 7);
    const uint32_t base = (blk / 2) * kAtom, chunk0 = (blk & 1) * 4;
    const int jobs = nt <= 0 ? 0 : kBoth ? 2 * nt : nt;
    uint4 raw[2][kIt][M / 4];
    uint32_t sc[2][kIt];
    int64_t at[kIt];
    int page[kIt];
    auto look_up = [&](int t) {                      // the pages of a tile
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int p = (tile0 + t) * kTile + it * kRows + row_in;
        page[it] = t < nt && p < range.total ? a.pages[b * a.ldp + page_of(a, p)] : -1;
      }
    };
    auto locate = [&](int t) {                       // its rows in the pool
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const uint32_t p = (tile0 + t) * kTile + it * kRows + row_in;
        const int64_t slot = static_cast<int64_t>(page[it]) * a.page_size + (p - page_of(a, p) * a.page_size);
        const bool ok = page[it] >= 0 && slot < a.c.n_slots;
        if (!ok && t < nt && static_cast<int>(p) < range.total) record_bad_index(a.status);
        at[it] = ok ? slot * a.c.n_kvh + g : -1;
      }
    };
    auto fetch = [&](int sv, int s) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        if (at[it] >= 0) {
          const uint8_t *c = a.c.codes[sv] + at[it] * a.c.code_pitch[sv] + blk * (kBlock * M / 8);
#pragma unroll
          for (int i = 0; i < M / 4; ++i) raw[s][it][i] = load_stream(c + 16 * i);
          sc[s][it] = __ldg(a.c.scales[sv] + at[it] * a.c.scale_pitch[sv] + blk);
        } else {
#pragma unroll
          for (int i = 0; i < M / 4; ++i) raw[s][it][i] = make_uint4(0, 0, 0, 0);
          sc[s][it] = 0;
        }
      }
    };
    auto decode = [&](int s, uint32_t dst) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int r = it * kRows + row_in;
        uint8_t *rowp = smem + dst + base + r * 128;
        const BlockScale<M> bs(sc[s][it]);
        const uint32_t *wd = reinterpret_cast<const uint32_t *>(&raw[s][it][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(rowp + (((chunk0 + j) ^ (r & 7)) << 4)) =
              decode8<M>(wd[j * M / 4], M == 8 ? wd[j * M / 4 + 1] : 0, bs);
      }
      ptx::fence_async_shared();
    };
    auto scores = [&](int t) {                       // one lane: waits for K(t) and the place of its scores
      bool ok = wait_phase(k_full + t % NS, (t / NS) & 1, given_up, a.status);
      if (t >= 2) ok = ok && wait_phase(p_full + (t & 1), ((t - 2) >> 1) & 1, given_up, a.status);
      if (!ok) return false;
      ptx::tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ptx::mma_bf16(tmem + (t & 1) * R, ptx::desc_sw128(sbase + S::kK + (t % NS) * S::kKV + (k / 4) * kAtom + (k % 4) * 32),
                      ptx::desc_sw128(sbase + S::kQ + (k / 4) * (R * 128) + (k % 4) * 32), S::kIdescS, k > 0);
      ptx::mma_commit(s_done + (t & 1));
      return true;
    };
    auto output = [&](int t) {                       // one lane: waits for V(t) and its weights
      const bool ok = wait_phase(v_full + t % NS, (t / NS) & 1, given_up, a.status) &&
                      wait_phase(p_full + (t & 1), (t >> 1) & 1, given_up, a.status);
      if (!ok) return false;
      ptx::tc_fence_after();
      const bool fresh = P > 1 ? t % kPeriod == 0 : t == 0;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        ptx::mma_bf16(tmem_o, ptx::desc_mn<64>(sbase + S::kV + (t % NS) * S::kKV + k * 2048, kAtom),
                      ptx::desc_mn<S::kPWidth>(sbase + S::kP + t % S::kPBufs * S::kPBytes + k * 32 * S::kPWidth, S::kPAtom),
                      S::kIdescO, !fresh || k > 0);
      ptx::mma_commit(o_done + (t & 1));
      return true;
    };
    // what the fetch of job j + 2 needs
    auto advance = [&](int j) {
      if (kBoth && (j & 1)) return;                  // V of the same tile
      const int t = kBoth ? j >> 1 : j;
      locate(t);
      look_up(t + 1);
    };
    if (jobs > 0) {
      look_up(0);
      advance(0);
      fetch(kBoth ? 0 : own, 0);
      advance(1);
      fetch(kBoth ? 1 : own, 1);
      if (kBoth || own == 0) {
        // q: row c of the tile, 16-byte chunks, zero where there is no such row
        for (int i = (dw & 3) * 32 + lane; i < R * (D / 8); i += 128) {
          const int c = i / (D / 8), e = i - c * (D / 8);
          const int rr = row0 + c, di = rr / a.rep, h = rr - di * a.rep;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (di < sq.n)
            v = *reinterpret_cast<const uint4 *>(a.q + (sq.first + di) * a.ldqt + (g * a.rep + h) * a.ldqh + e * 8);
          *reinterpret_cast<uint4 *>(smem + S::kQ + (e / 8) * (R * 128) + c * 128 + (((e & 7) ^ (c & 7)) << 4)) = reorder8<M>(v);
        }
      }
    }
    bool ok = true;
    auto job = [&](int j, int s) {
      const int t = kBoth ? j >> 1 : j;
      const int isv = kBoth ? s : own;
      const int u = t - NS;                          // the tile whose place this one takes
      if (u >= 0) ok = wait_phase((isv ? o_done : s_done) + (u & 1), (u >> 1) & 1, given_up, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      decode(s, (isv ? S::kV : S::kK) + (t % NS) * S::kKV);
      ptx::mbar_arrive((isv ? v_full : k_full) + t % NS);
      if (j + 2 < jobs) {
        advance(j + 2);
        fetch(isv, s);
      }
      if (w == 0) {
        if (lane == 0) {
          if (!isv) {
            ok = scores(t);
            if (kBoth && t > 0) ok = ok && output(t - 1);
          } else if (!kBoth || t == nt - 1) {
            ok = output(t);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    };
    for (int j = 0; j < jobs && ok; j += 2) {
      job(j, 0);
      if (j + 1 < jobs && ok) job(j + 1, 1);
    }
    if (!ok && w == 0 && lane == 0) {
      // leave no product in flight: a last commit covers all that this thread issued
      ptx::mma_commit(drained + own);
      ptx::mbar_wait_cycles(drained + own, 0, kTreeWait);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2, w4 = warp & 3;
    const int tok = w4 * 32 + lane, col0 = grp * C;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    // the swizzle of a row of 128, 64 or 32 bytes
    const int pswz = S::kPWidth == 64 ? tok & 7 : S::kPWidth == 32 ? (tok >> 1) & 3 : (tok >> 2) & 1;
    float *acc = reinterpret_cast<float *>(smem + S::kAcc) + col0 * D + tok;
    float sum[C];
#pragma unroll
    for (int k = 0; k < C; ++k) sum[k] = 0.f;
    bool ok = true;
    auto load_scores = [&](int t, uint32_t (&s)[C]) {
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += 16)
        ptx::tmem_ld16(tmem + lanes + (t & 1) * R + col0 + c0, *reinterpret_cast<uint32_t(*)[16]>(&s[c0]));
      ptx::tmem_wait_ld();
    };
    for (int t = 0; t < nt; ++t) {
      ok = wait_phase(s_done + (t & 1), (t >> 1) & 1, given_up, a.status);
      ptx::tc_fence_after();
      uint32_t see = 0xFFFFFFFFu;
      if ((tile0 + t + 1) * kTile > range.open) {
        // lane k: column k's tokens of this warp, then exchanged
        const int j0 = (tile0 + t) * kTile + w4 * 32 - sq.ctx;
        const uint32_t mine = seen_tokens(a, sq, (row0 + col0 + lane % C) / a.rep, j0);
        see = 0;
#pragma unroll
        for (int k = 0; k < C; ++k) see |= (__shfl_sync(0xffffffffu, mine, k) >> lane & 1u) << k;
      }
      uint32_t s[C];
      load_scores(t, s);
      float v[C], top = -INFINITY;
#pragma unroll
      for (int k = 0; k < C; k += 4) {
        const float4 r = *reinterpret_cast<const float4 *>(ref + col0 + k);
        v[k] = fmaf(__uint_as_float(s[k]), a.scale_log2, -r.x);
        v[k + 1] = fmaf(__uint_as_float(s[k + 1]), a.scale_log2, -r.y);
        v[k + 2] = fmaf(__uint_as_float(s[k + 2]), a.scale_log2, -r.z);
        v[k + 3] = fmaf(__uint_as_float(s[k + 3]), a.scale_log2, -r.w);
      }
      if (see != 0xFFFFFFFFu) {
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = (see >> k) & 1u ? v[k] : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        top = fmaxf(top, v[k]);
        v[k] = exp2_fast(v[k]);
      }
      // (its vote below also carries a wait that ran out: all of the group leave together)
      if (t >= S::kPBufs) {
        const int u = t - S::kPBufs;
        ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status) && ok;
      }
      const bool flush = P > 1 && t > 0 && t % kPeriod == 0;
      if (any_of(grp, top > kSlack || !ok || flush)) {
        // rare: a reference is overtaken (or not set yet), or an output period ends
        if (t > 0 && ok) {
          const int u = t - 1;
          ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
          ptx::tc_fence_after();
        }
        if (any_of(grp, !ok)) {
          ok = false;
          break;
        }
        load_scores(t, s);
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = (see >> k) & 1u ? __uint_as_float(s[k]) * a.scale_log2 : -INFINITY;
        {
          float m[C];
#pragma unroll
          for (int k = 0; k < C; ++k) m[k] = v[k];
          const float mine = over_lanes(m, lane, [](float p, float q) { return fmaxf(p, q); });
          if (lane % (32 / C) == 0) wstat[w4 * R + col0 + lane / (32 / C)] = mine;
        }
        group_sync(grp);
        if (tok < C) {
          // references move only as far as they have to: by nothing, unless passed by 2^kSlack
          const int c = col0 + tok;
          const float old = ref[c];
          float m = fmaxf(fmaxf(wstat[c], wstat[R + c]), fmaxf(wstat[2 * R + c], wstat[3 * R + c]));
          m = m - old > kSlack || old == -INFINITY ? m : old;
          factor[c] = m == old ? 1.f : exp2f(old - m);
          ref[c] = m;
        }
        group_sync(grp);
#pragma unroll
        for (int k = 0; k < C; ++k) {
          sum[k] *= factor[col0 + k];
          v[k] = (see >> k) & 1u ? exp2_fast(v[k] - ref[col0 + k]) : 0.f;
        }
        if (t > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < C; c0 += 16) {
            float part[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) part[k] = 0.f;
#pragma unroll 1
            for (int q = P - 1; q >= 0; --q) {
              uint32_t o[16];
              ptx::tmem_ld16(tmem_o + lanes + q * R + col0 + c0, o);
              ptx::tmem_wait_ld();
              if (flush) {
#pragma unroll
                for (int k = 0; k < 16; ++k) part[k] += __uint_as_float(o[k]);
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[col0 + c0 + k]);
                ptx::tmem_st16(tmem_o + lanes + q * R + col0 + c0, o);
              }
            }
            if (P > 1 && tok < D && (flush || t > kPeriod)) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float *z = acc + (c0 + k) * D;
                *z = ((t > kPeriod ? *z : 0.f) + part[k]) * factor[col0 + c0 + k];
              }
            }
          }
          ptx::tmem_wait_st();
        }
        group_sync(grp);                             // (factor and wstat may be written again)
      }
      // the weights as P bf16 pieces, each the rounding of what the ones before left
      uint8_t *prow = smem + S::kP + t % S::kPBufs * S::kPBytes + tok * (2 * S::kPWidth);
#pragma unroll
      for (int k = 0; k < C; ++k) sum[k] += v[k];
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += 8) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[k] = pack2(v[c0 + 2 * k], v[c0 + 2 * k + 1]);
            if (q + 1 < P) {
              v[c0 + 2 * k] -= __uint_as_float(o[k] << 16);
              v[c0 + 2 * k + 1] -= __uint_as_float(o[k] & 0xFFFF0000u);
            }
          }
          const int cc = q * R + col0 + c0;
          *reinterpret_cast<uint4 *>(prow + (cc / S::kPWidth) * S::kPAtom + (((cc % S::kPWidth) / 8 ^ pswz) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      ptx::fence_async_shared();
      ptx::tc_fence_before();
      ptx::mbar_arrive(p_full + (t & 1));
    }
    // the sums over the tokens: lanes, then warps, in a fixed order
    const float mine = over_lanes(sum, lane, [](float p, float q) { return p + q; });
    if (lane % (32 / C) == 0) wstat[w4 * R + col0 + lane / (32 / C)] = mine;
    group_sync(grp);
    if (tok < C) {
      const int c = col0 + tok, i = (row0 + c) / a.rep, h = row0 + c - i * a.rep;
      const float l = (wstat[c] + wstat[R + c]) + (wstat[2 * R + c] + wstat[3 * R + c]);
      const float lse2 = l == 0.f ? -INFINITY : ref[c] + log2f(l);
      const int64_t row = sq.first + i, head = g * a.rep + h;
      factor[c] = l == 0.f ? 0.f : 1.f / l;
      int64_t z = -1;
      if (i < sq.n) {
        if (a.splits == 1) {
          z = row * a.ldot + head * a.ldoh;
          if (a.lse) a.lse[row * a.n_qh + head] = lse2 * kLn2;
        } else {
          z = (sp * a.rows + row) * a.n_qh + head;
          a.part_lse[z] = lse2;
          z *= D;
        }
      }
      place[c] = z;
    }
    group_sync(grp);
    if (nt > 0) {
      const int u = nt - 1;
      ok = ok && wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
      ptx::tc_fence_after();
    }
    // out: thread = position tok of the head, one column after the other
    const int e = true_position<M>(tok);
#pragma unroll 1
    for (int c0 = 0; c0 < C; c0 += 16) {
      float o[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = 0.f;
      if (nt > 0) {
#pragma unroll
        for (int q = P - 1; q >= 0; --q) {
          uint32_t r[16];
          ptx::tmem_ld16(tmem_o + lanes + q * R + col0 + c0, r);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] += __uint_as_float(r[k]);
        }
      }
      if (tok < D) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int c = col0 + c0 + k;
          if (place[c] < 0) continue;
          float y = o[k];
          if (P > 1 && nt > kPeriod) y += acc[(c0 + k) * D];
          y = factor[c] == 0.f ? 0.f : y * factor[c];
          const int64_t z = place[c] + e;
          if (a.splits > 1) a.part[z] = y;
          else if constexpr (FOUT) static_cast<float *>(a.out)[z] = y;
          else static_cast<__nv_bfloat16 *>(a.out)[z] = __float2bfloat16(y);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, S::kTmem);
}

// One warp per (drafted token, head): the splits' outputs, weighted by
// 2^(lse_j - lse), in split order.
template <int D, bool FOUT>
__global__ void __launch_bounds__(128) tree_combine_kernel(TreeArgs a, int R) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = D / 32;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int u = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = u / a.n_qh, head = u - i * a.n_qh;
  const Sequence sq = sequence_of(a, b, false);
  if (i >= sq.n) return;
  const int row0 = (i * a.rep + head % a.rep) / R * R;
  const int tiles = (tile_range(a, sq, row0, R).total + kTile - 1) / kTile;
  const int n = max(1, (tiles + a.tiles_per_split - 1) / a.tiles_per_split);
  const int64_t row = sq.first + i, z0 = row * a.n_qh + head, step = a.rows * static_cast<int64_t>(a.n_qh);
  float m = -INFINITY;
  for (int j = lane; j < n; j += 32) {
    const float l = a.part_lse[z0 + j * step];
    m = l == l ? fmaxf(m, l) : l;
    if (m != m) break;
  }
  bool nan = m != m;
  nan = __any_sync(0xffffffffu, nan);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float total = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (m != -INFINITY) {
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float w = exp2f(a.part_lse[z0 + j * step] - m);
      const float *p = a.part + (z0 + j * step) * D + lane * E;
      total += w;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
  }
  const float inv = nan ? NAN : total == 0.f ? 0.f : 1.f / total;
  const int64_t at = row * a.ldot + head * a.ldoh + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (FOUT) static_cast<float *>(a.out)[at + e] = acc[e] * inv;
    else static_cast<__nv_bfloat16 *>(a.out)[at + e] = __float2bfloat16(acc[e] * inv);
  }
  if (a.lse && lane == 0) a.lse[z0] = nan ? NAN : total == 0.f ? -INFINITY : (m + log2f(total)) * kLn2;
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

// How a call is cut: columns of a row tile, row tiles, splits.
struct Cut {
  int R, pieces;
  int64_t row_tiles, splits, tiles_per_split, part_bytes, lse_bytes;
};
Cut tree_cut(const TreeArgs &a, bool fout, int sms) {
  Cut c{};
  c.pieces = fout ? 3 : 1;
  const int64_t group_rows = static_cast<int64_t>(a.max_q) * a.rep;
  c.R = group_rows <= 16 ? 16 : group_rows <= 32 ? 32 : 64;
  c.row_tiles = (group_rows + c.R - 1) / c.R;
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(a.max_len) + kTile - 1) / kTile);
  const int64_t base = c.row_tiles * a.c.n_kvh * a.B, room = 2 * sms;
  const int64_t want = std::max<int64_t>(1, std::min(tiles, (room + base - 1) / base));
  c.tiles_per_split = (tiles + want - 1) / want;
  c.splits = (tiles + c.tiles_per_split - 1) / c.tiles_per_split;
  if (c.splits > 1) {
    const int64_t n = c.splits * a.rows * a.n_qh;
    c.part_bytes = round_up(n * a.c.d * 4, 256);
    c.lse_bytes = n * 4;
  }
  return c;
}

template <int D, int M, int R, int P, bool FOUT>
mxs_status launch_tree(const TreeArgs &a, cudaStream_t s) {
  using S = Shape<D, M, R, P>;
  if (!ensure_smem(tree_kernel<D, M, R, P, FOUT>, S::kBytes)) return MXS_ERR_CUDA;
  const int64_t grid = static_cast<int64_t>(a.B) * a.c.n_kvh * a.splits * a.row_tiles;
  launch_pdl(tree_kernel<D, M, R, P, FOUT>, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), S::kBytes, s, a);
  count_launch();
  if (a.splits > 1) {
    const int64_t warps = static_cast<int64_t>(a.max_q) * a.n_qh;
    launch_pdl(tree_combine_kernel<D, FOUT>, dim3(static_cast<unsigned>((warps + 3) / 4), static_cast<unsigned>(a.B)),
               dim3(128), 0, s, a, R);
    count_launch();
  }
  return cuda_status(cudaGetLastError());
}
template <int D, int M>
mxs_status launch_shape(const TreeArgs &a, const Cut &c, cudaStream_t s) {
  if (c.pieces == 1) {
    if (c.R == 16) return launch_tree<D, M, 16, 1, false>(a, s);
    if (c.R == 32) return launch_tree<D, M, 32, 1, false>(a, s);
    return launch_tree<D, M, 64, 1, false>(a, s);
  }
  if (c.R == 16) return launch_tree<D, M, 16, 3, true>(a, s);
  if (c.R == 32) return launch_tree<D, M, 32, 3, true>(a, s);
  return launch_tree<D, M, 64, 3, true>(a, s);
}

}  // namespace
}  // namespace mxs

using namespace mxs;

extern "C" mxs_status mxs_attn_tree_workspace_bytes(const mxs_kv_cache *cache, const mxs_tree_batch *batch,
                                                    int64_t n_qh, mxs_dtype ot, size_t *bytes) {
  if (!bytes) return MXS_ERR_ARG;
  if (!dtype_ok(ot)) return MXS_ERR_DTYPE;
  TreeArgs a{};
  const mxs_status st = tree_check(cache, batch, n_qh, &a);
  if (st != MXS_OK) return st;
  const Cut c = tree_cut(a, ot == MXS_F32, device_sms());
  *bytes = static_cast<size_t>(c.part_bytes + c.lse_bytes);
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
  const Cut c = tree_cut(a, ot == MXS_F32, device_sms());
  if (static_cast<__int128>(a.B) * a.c.n_kvh * c.splits * c.row_tiles > INT32_MAX) return MXS_ERR_SHAPE;
  if (c.splits > 1 && (!ws || ws_bytes < static_cast<size_t>(c.part_bytes + c.lse_bytes) ||
                       (reinterpret_cast<uintptr_t>(ws) & 255u)))
    return MXS_ERR_WORKSPACE;
  if ((st = check_device()) != MXS_OK) return st;
  if (!(a.status = device_status_word())) return MXS_ERR_CUDA;
  a.q = static_cast<const uint16_t *>(q);
  a.ldqt = ldqt;
  a.ldqh = ldqh;
  a.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);   // log2(e)
  a.out = out;
  a.ldot = ldot;
  a.ldoh = ldoh;
  a.lse = lse;
  a.row_tiles = static_cast<int32_t>(c.row_tiles);
  a.splits = static_cast<int32_t>(c.splits);
  a.tiles_per_split = static_cast<int32_t>(c.tiles_per_split);
  a.part = static_cast<float *>(ws);
  a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + c.part_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64) return a.c.bits == 4 ? launch_shape<64, 4>(a, c, s) : launch_shape<64, 8>(a, c, s);
  return a.c.bits == 4 ? launch_shape<128, 4>(a, c, s) : launch_shape<128, 8>(a, c, s);
}
