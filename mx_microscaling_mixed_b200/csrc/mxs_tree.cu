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

// ---------------------------------------------------------------- kernel
namespace {

constexpr int kTile = 128;                       // tokens of a tile
constexpr int kDecodeWarps = 4;
constexpr int kAtom = kTile * 128;               // 64 bf16 values of each token of a tile
constexpr float kSlack = 60.f;                   // weights are kept below 2^kSlack
constexpr long long kTreeWait = 2000000000LL;    // cycles (about 1 s)

// R columns (query rows) per CTA; P bf16 pieces of a weight.
template <int D, int M, int R, int P>
struct Shape {
  static constexpr int kSoftWarps = R > 64 ? 8 : 4;
  static constexpr int kCols = R > 64 ? 64 : R;          // columns of a softmax warp
  static constexpr int kThreads = (kSoftWarps + kDecodeWarps + 1) * 32;
  static constexpr int kN = R * P;                       // columns of the output product
  static constexpr int kKV = kTile * D * 2;
  static constexpr int kPWidth = R < 64 ? R : 64;        // columns in a row of a swizzle atom of the weights
  static constexpr int kPAtom = kTile * kPWidth * 2;
  static constexpr int kPBytes = kTile * kN * 2;
  static constexpr int kPBufs = 2 * kPBytes + 2 * kKV + R * D * 2 <= 112 * 1024 || R > 64 ? 2 : 1;
  static constexpr int kK = 0, kV = kKV, kP = 2 * kKV, kQ = kP + kPBufs * kPBytes;
  static constexpr int kStat = kQ + R * D * 2;           // floats: reference, factor, 4 x maximum or sum per column
  static constexpr int kBar = kStat + 6 * R * 4;
  // (heads of 64: the output product reads 64 places that nobody uses behind V's, which have to exist)
  static constexpr int kEnd = kBar + 9 * 8 + 16 > kV + 2 * kAtom ? kBar + 9 * 8 + 16 : kV + 2 * kAtom;
  static constexpr int kBytes = kEnd + 1024;
  static constexpr int kTmem = 2 * R + kN <= 64 ? 64 : 2 * R + kN <= 128 ? 128 : 2 * R + kN <= 256 ? 256 : 512;
  static constexpr int kResident = 2 * (kBytes + 1024) <= 228 * 1024 && kTmem <= 256 && kThreads <= 288 ? 2 : 1;
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

}  // namespace

// CTA = (sequence, kv head, split of the tokens, row tile).  Tokens are the
// 128 rows of the matrix instruction, query rows its columns, so that the
// work follows the number of rows (16 to 128 of them) while a cache tile is
// decoded once for all of them:
//   S^T [token][row] = K Q^T     A = K  (token x d, K-major),  B = Q
//   O^T [d][row]    += V^T P^T   A = V  (token x d, stored along d), B = P
// Both accumulate in tensor memory.  Roles: four warps fetch and decode the
// cache into shared memory, one thread issues the products, four or eight
// warps turn scores into weights.  A softmax thread owns one token and sums
// its weights per row over all tiles; the sums meet at the end.
//   The running maximum of a row is a reference that weights are relative
// to, common to all tokens: it is set by the first tile and moved only when
// a score passes it by more than 2^60, which fp32 and bf16 hold with no loss
// of precision; so a tile usually needs no maximum, only one vote per 16
// rows that none of its scores is above.
template <int D, int M, int R, int P, bool FOUT>
__global__ void __launch_bounds__(Shape<D, M, R, P>::kThreads, Shape<D, M, R, P>::kResident) tree_kernel(TreeArgs a) {
  using S = Shape<D, M, R, P>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *ref = reinterpret_cast<float *>(smem + S::kStat), *factor = ref + R, *wstat = factor + R;   // wstat[4][R]
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::kBar);
  uint64_t *k_full = bar, *v_full = bar + 1, *s_done = bar + 2, *p_full = bar + 4, *o_done = bar + 6,
           *drained = bar + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 9);
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
    ptx::mbar_init(k_full, kDecodeWarps * 32);
    ptx::mbar_init(v_full, kDecodeWarps * 32);
    ptx::mbar_init(drained, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(p_full + i, S::kSoftWarps * 32);
      ptx::mbar_init(s_done + i, 1);
      ptx::mbar_init(o_done + i, 1);
    }
    ptx::fence_mbar_init();
    *given_up = 0;
  }
  for (int i = threadIdx.x; i < R; i += S::kThreads) ref[i] = -INFINITY;
  // tensor memory is taken after the wait for earlier kernels and before
  // later ones may start: a CTA that waits for another kernel holds none
  if (warp == S::kSoftWarps + kDecodeWarps) {
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

  if (warp == S::kSoftWarps + kDecodeWarps) {
    // ------------------------------------------------------ matrix products
    if (lane == 0 && nt > 0) {
      auto scores = [&](int t) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_bf16(tmem + (t & 1) * R, ptx::desc_sw128(sbase + S::kK + (k / 4) * kAtom + (k % 4) * 32),
                        ptx::desc_sw128(sbase + S::kQ + (k / 4) * (R * 128) + (k % 4) * 32), S::kIdescS, k > 0);
        ptx::mma_commit(s_done + (t & 1));
      };
      bool ok = wait_phase(k_full, 0, given_up, a.status);
      ptx::tc_fence_after();
      if (ok) scores(0);
      for (int t = 0; ok && t < nt; ++t) {
        if (t + 1 < nt) {
          ok = wait_phase(k_full, (t + 1) & 1, given_up, a.status);
          if (!ok) break;
          ptx::tc_fence_after();
          scores(t + 1);
        }
        ok = wait_phase(v_full, t & 1, given_up, a.status) && wait_phase(p_full + (t & 1), (t >> 1) & 1, given_up, a.status);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t pb = sbase + S::kP + (S::kPBufs == 2 ? (t & 1) * S::kPBytes : 0);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          ptx::mma_bf16(tmem_o, ptx::desc_mn<64>(sbase + S::kV + k * 2048, kAtom),
                        ptx::desc_mn<S::kPWidth>(pb + k * 32 * S::kPWidth, S::kPAtom), S::kIdescO, t > 0 || k > 0);
        ptx::mma_commit(o_done + (t & 1));
      }
      if (!ok) {
        // leave no product in flight: a last commit covers all that were issued
        ptx::mma_commit(drained);
        ptx::mbar_wait_cycles(drained, 0, kTreeWait);
      }
    }
    __syncwarp();
  } else if (warp >= S::kSoftWarps) {
    // ------------------------------------------------- fetching and decoding
    constexpr int BL = D / kBlock;                   // blocks of a cache row
    const int w = warp - S::kSoftWarps, q4 = lane >> 3;
    const int blk = q4 % BL, sub = q4 / BL;
    constexpr int kRows = 32 * 4 / BL;               // rows per iteration of the four warps
    constexpr int kIt = kTile / kRows;
    const int row_in = w * (8 * 4 / BL) + sub * 8 + (lane & 7);
    // chunk of 16 bytes c of atom A of row r: 8 lanes on 8 rows hit 8 banks groups
    const uint32_t base = (blk / 2) * kAtom, chunk0 = (blk & 1) * 4;
    uint4 raw[2][kIt][M / 4];
    uint32_t sc[2][kIt];
    int64_t at[kIt];
    auto locate = [&](int t) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int p = (tile0 + t) * kTile + it * kRows + row_in;
        const int64_t slot = p < range.total ? slot_of(a, b, p) : -1;
        at[it] = slot < 0 ? -1 : slot * a.c.n_kvh + g;
      }
    };
    auto fetch = [&](int sv) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        if (at[it] >= 0) {
          const uint8_t *c = a.c.codes[sv] + at[it] * a.c.code_pitch[sv] + blk * (kBlock * M / 8);
#pragma unroll
          for (int i = 0; i < M / 4; ++i) raw[sv][it][i] = load_stream(c + 16 * i);
          sc[sv][it] = __ldg(a.c.scales[sv] + at[it] * a.c.scale_pitch[sv] + blk);
        } else {
#pragma unroll
          for (int i = 0; i < M / 4; ++i) raw[sv][it][i] = make_uint4(0, 0, 0, 0);
          sc[sv][it] = 0;
        }
      }
    };
    auto decode = [&](int sv, uint32_t dst) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int r = it * kRows + row_in;
        uint8_t *rowp = smem + dst + base + r * 128;
        const BlockScale<M> bs(sc[sv][it]);
        const uint32_t *wd = reinterpret_cast<const uint32_t *>(&raw[sv][it][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(rowp + (((chunk0 + j) ^ (r & 7)) << 4)) =
              decode8<M>(wd[j * M / 4], M == 8 ? wd[j * M / 4 + 1] : 0, bs);
      }
      ptx::fence_async_shared();
    };
    if (nt > 0) {
      locate(0);
      fetch(0);
      fetch(1);
      // q: row c of the tile, 16-byte chunks, zero where there is no such row
      for (int i = threadIdx.x - S::kSoftWarps * 32; i < R * (D / 8); i += kDecodeWarps * 32) {
        const int c = i / (D / 8), e = i - c * (D / 8);
        const int rr = row0 + c, di = rr / a.rep, h = rr - di * a.rep;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (di < sq.n)
          v = *reinterpret_cast<const uint4 *>(a.q + (sq.first + di) * a.ldqt + (g * a.rep + h) * a.ldqh + e * 8);
        *reinterpret_cast<uint4 *>(smem + S::kQ + (e / 8) * (R * 128) + c * 128 + (((e & 7) ^ (c & 7)) << 4)) = reorder8<M>(v);
      }
    }
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const int u = t - 1;
      if (t > 0) ok = wait_phase(s_done + (u & 1), (u >> 1) & 1, given_up, a.status);
      if (!ok) break;
      decode(0, S::kK);
      ptx::mbar_arrive(k_full);
      if (t + 1 < nt) {
        locate(t + 1);
        fetch(0);
      }
      if (t > 0) ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
      if (!ok) break;
      decode(1, S::kV);
      ptx::mbar_arrive(v_full);
      if (t + 1 < nt) fetch(1);
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2, w4 = warp & 3;
    const int tok = w4 * 32 + lane, col0 = grp * 64;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    // the swizzle of a row of 128, 64 or 32 bytes
    const int pswz = S::kPWidth == 64 ? tok & 7 : S::kPWidth == 32 ? (tok >> 1) & 3 : (tok >> 2) & 1;
    float sum[S::kCols];
#pragma unroll
    for (int k = 0; k < S::kCols; ++k) sum[k] = 0.f;
    bool ok = true;
    for (int t = 0; t < nt && ok; ++t) {
      ok = wait_phase(s_done + (t & 1), (t >> 1) & 1, given_up, a.status);
      if (t >= S::kPBufs) {
        const int u = t - S::kPBufs;
        ok = ok && wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
      }
      ptx::tc_fence_after();
      const int p = (tile0 + t) * kTile + tok;
      const bool masked = (tile0 + t + 1) * kTile > range.open;
      uint8_t *prow = smem + S::kP + (S::kPBufs == 2 ? (t & 1) * S::kPBytes : 0) + tok * (2 * S::kPWidth);
#pragma unroll
      for (int c0 = 0; c0 < S::kCols; c0 += 16) {
        uint32_t s[16];
        ptx::tmem_ld16(tmem + lanes + (t & 1) * R + col0 + c0, s);
        uint32_t see = 0xFFFFu;
        if (masked) {
          see = 0;
          if (p < sq.ctx) {
            see = 0xFFFFu;
          } else if (p < range.total) {
            const int j = p - sq.ctx;
            int i = (row0 + col0 + c0) / a.rep, h = row0 + col0 + c0 - i * a.rep;
            bool sees = false, fresh = true;
            for (int k = 0; k < 16; ++k) {
              if (fresh)
                sees = i < sq.n && (a.mask ? (a.mask[(sq.first + i) * a.ldm + (j >> 5)] >> (j & 31)) & 1u : j <= i);
              see |= static_cast<uint32_t>(sees) << k;
              fresh = ++h == a.rep;
              if (fresh) {
                h = 0;
                ++i;
              }
            }
          }
        }
        ptx::tmem_wait_ld();
        float v[16], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = fmaf(__uint_as_float(s[k]), a.scale_log2, -ref[col0 + c0 + k]);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = (see >> k) & 1u ? v[k] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, v[k]);
        if (any_of(grp, top > kSlack || !ok)) {
          // a reference is overtaken (or not set yet): move those of these 16
          // columns to the larger of themselves and the tile's maximum
          bool stop = !ok;
          if (t > 0 && !stop) {
            const int u = t - 1;
            stop = !wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
            ptx::tc_fence_after();
          }
          if (any_of(grp, stop)) {
            ok = false;
            break;
          }
          ptx::tmem_ld16(tmem + lanes + (t & 1) * R + col0 + c0, s);
          ptx::tmem_wait_ld();
          float mine = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            v[k] = (see >> k) & 1u ? __uint_as_float(s[k]) * a.scale_log2 : -INFINITY;
            float m = v[k];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == k) mine = m;
          }
          if (lane < 16) wstat[w4 * R + col0 + c0 + lane] = mine;
          group_sync(grp);
          if (w4 == 0 && lane < 16) {
            const int c = col0 + c0 + lane;
            const float old = ref[c];
            const float m = fmaxf(fmaxf(fmaxf(wstat[c], wstat[R + c]), fmaxf(wstat[2 * R + c], wstat[3 * R + c])), old);
            factor[c] = m == old ? 1.f : exp2f(old - m);
            ref[c] = m;
          }
          group_sync(grp);
          float f[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            f[k] = factor[col0 + c0 + k];
            sum[c0 + k] *= f[k];
            v[k] = (see >> k) & 1u ? v[k] - ref[col0 + c0 + k] : -INFINITY;
          }
          if (t > 0) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
              uint32_t o[16];
              ptx::tmem_ld16(tmem_o + lanes + q * R + col0 + c0, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k]);
              ptx::tmem_st16(tmem_o + lanes + q * R + col0 + c0, o);
            }
            ptx::tmem_wait_st();
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          v[k] = exp2_fast(v[k]);
          sum[c0 + k] += v[k];
        }
        // the weights as P bf16 pieces, each the rounding of what the ones before left
#pragma unroll
        for (int q = 0; q < P; ++q) {
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            o[k] = pack2(v[2 * k], v[2 * k + 1]);
            if (q + 1 < P) {
              v[2 * k] -= __uint_as_float(o[k] << 16);
              v[2 * k + 1] -= __uint_as_float(o[k] & 0xFFFF0000u);
            }
          }
          const int cc = q * R + col0 + c0;
          uint8_t *pr = prow + (cc / S::kPWidth) * S::kPAtom;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4 *>(pr + ((((cc % S::kPWidth) / 8 + k) ^ pswz) << 4)) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (!ok) break;
      ptx::fence_async_shared();
      ptx::tc_fence_before();
      ptx::mbar_arrive(p_full + (t & 1));
    }
    // the sums over the tokens: lanes, then warps, in a fixed order
#pragma unroll
    for (int c0 = 0; c0 < S::kCols; c0 += 16) {
      float mine = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float v = sum[c0 + k];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == k) mine = v;
      }
      if (lane < 16) wstat[w4 * R + col0 + c0 + lane] = mine;
    }
    group_sync(grp);
    if (nt > 0) {
      const int u = nt - 1;
      ok = ok && wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
      ptx::tc_fence_after();
    }
    // out: thread = position tok of the head, one column after the other
    const int e = true_position<M>(tok);
    const int64_t heads = a.n_qh;
#pragma unroll
    for (int c0 = 0; c0 < S::kCols; c0 += 16) {
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
      int i = (row0 + col0 + c0) / a.rep, h = row0 + col0 + c0 - i * a.rep;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (i < sq.n) {
          const int c = col0 + c0 + k;
          const float l = wstat[c] + wstat[R + c] + wstat[2 * R + c] + wstat[3 * R + c];
          const float y = l == 0.f ? 0.f : o[k] / l;
          const int64_t row = sq.first + i, head = g * a.rep + h;
          const float lse2 = l == 0.f ? -INFINITY : ref[c] + log2f(l);
          if (a.splits == 1) {
            if (tok < D) {
              const int64_t z = row * a.ldot + head * a.ldoh + e;
              if constexpr (FOUT) static_cast<float *>(a.out)[z] = y;
              else static_cast<__nv_bfloat16 *>(a.out)[z] = __float2bfloat16(y);
            }
            if (a.lse && tok == 0) a.lse[row * heads + head] = lse2 * kLn2;
          } else {
            const int64_t z = (sp * a.rows + row) * heads + head;
            if (tok < D) a.part[z * D + e] = y;
            if (tok == 0) a.part_lse[z] = lse2;
          }
        }
        if (++h == a.rep) {
          h = 0;
          ++i;
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == S::kSoftWarps + kDecodeWarps) ptx::tmem_dealloc(tmem, S::kTmem);
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
