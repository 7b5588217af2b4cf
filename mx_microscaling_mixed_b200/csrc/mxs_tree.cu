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

struct Meta;

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
  int32_t row_tiles, ctas;
  float *part, *part_lse;  // unfinished items' normalised outputs and base-2 lse: [CTA][first, last][column]([D])
  int32_t out_vec;         // out's rows allow 16-byte stores
  Meta *meta;       // [CTA]; NULL where no item has more than one tile
  int *status;
};

// What a CTA says of its first item, for joining.
struct Meta {
  int first, n;            // the sequence's rows
  int rt, g, tile, tiles;  // the item, its tile where the CTA begins, its tiles
  int total, parts;        // tiles of the call, CTAs with work
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
constexpr int kTreeWait = 2000000000;            // cycles (about 1 s)
// Limit of the matrix warp's waits, which stop all other roles
// (mxs_set_wait_limit lowers it for a diagnostic run).
__device__ int g_tree_wait = kTreeWait;

// Waits for a barrier's phase; gives up when the limit ran out or another
// role has given up.
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *given_up, int *status) {
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait_for(bar, parity, 20000)) {
    if (*given_up) return false;
    if (clock64() - t0 > kTreeWait) {
      *given_up = 1;
      atomicExch(status, static_cast<int>(MXS_ERR_TIMEOUT));
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *given_up, int *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_long(bar, parity, given_up, status);
}
// A suspended wait may outlast a short limit: the matrix warp looks behind
// each tile at what its waits and the products issued after them took.
// (At each of the warp's waits the look took 4 % of the wide form;
// the limit read in the other roles' waits too, 3 % of 7-token trees.)
__device__ __forceinline__ bool in_time(uint32_t &since, uint32_t limit, volatile int *given_up, int *status) {
  const uint32_t now = clock(), took = now - since;
  since = now;
  if (took <= limit) return true;
  *given_up = 1;
  atomicExch(status, static_cast<int>(MXS_ERR_TIMEOUT));
  return false;
}
// Leaves no product in flight, whichever role gave up and when (a softmax
// warp may, on the last products, after all of them were issued): a last
// commit covers all that the warp issued, and the tensor memory is freed
// after this wait.
__device__ __forceinline__ void drain(uint32_t leader, uint64_t *bar, int *status) {
  ptx::mma_commit_by(leader, bar);
  if (!ptx::mbar_wait_cycles(bar, 0, kTreeWait)) atomicExch(status, static_cast<int>(MXS_ERR_TIMEOUT));
}
// One arrival for a warp whose lanes have each made their writes visible:
// arrivals of single lanes on one barrier go through one after the other.
__device__ __forceinline__ void arrive_warp(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
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
// The same for the 256 softmax threads of a half in tree_rows_kernel.
__device__ __forceinline__ bool any_of256(int half, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(half + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void half_sync(int half) {
  asm volatile("barrier.cta.sync %0, 256;" ::"r"(half + 1) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// (x, y) = (s, t) * scale + (r, q), two at once; s and t as bits.
__device__ __forceinline__ void scale_shift(float &x, float &y, uint32_t s, uint32_t t, float scale, float r, float q) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(__uint_as_float(s)), "f"(__uint_as_float(t)), "f"(scale), "f"(r), "f"(q));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The factors of a block by its scale byte come from a table in shared
// memory (a dozen instructions per block otherwise).
template <int M>
constexpr int kTableEntry = M == 4 ? 8 : 16;
template <int M, int THREADS>
__device__ __forceinline__ void fill_table(uint8_t *table) {
  for (uint32_t i = threadIdx.x; i < 256; i += THREADS) {
    const BlockScale<M> k = scale_factors<M>(min(i, kTopScale));
    if constexpr (M == 4) *reinterpret_cast<uint2 *>(table + 8 * i) = make_uint2(k.s, k.c);
    else *reinterpret_cast<uint4 *>(table + 16 * i) = make_uint4(k.s, k.c, k.s16, 0);
  }
}
template <int M>
__device__ __forceinline__ BlockScale<M> block_scale(const uint8_t *table, uint32_t b) {
  if constexpr (M == 4) {
    const uint2 t = *reinterpret_cast<const uint2 *>(table + 8 * b);
    return {t.x, t.y};
  } else {
    const uint4 t = *reinterpret_cast<const uint4 *>(table + 16 * b);
    return {t.x, t.y, t.z};
  }
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

// How a CTA's shared memory is laid out for R columns (query rows), P bf16
// pieces of a weight: what has to be there once first, then a second place
// for what waits most, while there is room.
template <int D, int M, int R, int P>
struct Shape {
  static constexpr int kSoftWarps = 8;                       // two groups of four
  // For each of K and V.  (Eight took a quarter longer: 7-token trees over 32 contexts of up to 8191 tokens of 8 bits.)
  static constexpr int kFetchWarps = 4;
  static constexpr int kMmaWarp = kSoftWarps + 2 * kFetchWarps;
  static constexpr int kThreads = (kMmaWarp + 1) * 32;
  // 64 columns: the softmax warps need 120 registers; 96 a thread at the launch, 256 x (120 - 96) = 256 x (96 - 72) moved
  static constexpr bool kMoveRegisters = R == 64;
  static constexpr int kCols = R / 2;                        // columns of a softmax group
  static constexpr int kN = R * P;                           // columns of the output product
  static constexpr int kKV = kTile * D * 2;
  static constexpr int kPWidth = R < 64 ? R : 64;            // columns in a row of a swizzle atom of the weights
  static constexpr int kPAtom = kTile * kPWidth * 2;
  static constexpr int kPBytes = kTile * kN * 2;
  static constexpr int kCodeRow = D * M / 8;                 // bytes
  static constexpr int kRawTensor = kTile * (kCodeRow + 4);  // codes and scale words of a tile as fetched
  static constexpr int kRaw = 2 * kRawTensor;
  static constexpr int kQBytes = R * D * 2, kAccBytes = P > 1 ? R * D * 4 : 0;
  static constexpr int kSmall = 6 * R * 4 + R * 8 + 32 * 8 + 256 + 256 * kTableEntry<M>;
  static constexpr int kRoom = 227 * 1024 - 1024 - kSmall;
  static constexpr int kOnce = 2 * kKV + kPBytes + kQBytes + kAccBytes + 2 * kRaw;
  static constexpr bool kFits = kOnce <= kRoom;
  static constexpr int kPBufs = kOnce + kPBytes <= kRoom ? 2 : 1;
  static constexpr int kWithP = kOnce + (kPBufs - 1) * kPBytes;
  static constexpr int kStagesV = kWithP + kKV <= kRoom ? 2 : 1;
  static constexpr int kWithV = kWithP + (kStagesV - 1) * kKV;
  static constexpr int kStagesK = kWithV + kKV <= kRoom ? 2 : 1;
  static constexpr int kWithK = kWithV + (kStagesK - 1) * kKV;
  static constexpr int kRings = kWithK + kRaw <= kRoom ? 3 : 2;          // fetched tiles
  static constexpr int kK = 0, kV = kStagesK * kKV, kP = kV + kStagesV * kKV, kQ = kP + kPBufs * kPBytes;
  static constexpr int kAcc = kQ + kQBytes;                  // fp32 sums of output periods, [column][place]
  static constexpr int kRawAt = kAcc + kAccBytes;
  static constexpr int kStat = kRawAt + kRings * kRaw;       // per column: reference, factor, 4 maxima or sums
  static constexpr int kPlace = kStat + 6 * R * 4;           // per column: where its output goes (64 bits)
  static constexpr int kBar = kPlace + R * 8;
  static constexpr int kStart = kBar + 32 * 8;               // where the CTA's work begins
  static constexpr int kTable = kStart + 256;                // factors by scale byte
  static constexpr int kEnd = kTable + 256 * kTableEntry<M>;
  static constexpr int kBytes = kEnd + 1024;
  // (heads of 64: the output product reads 64 places that nobody uses behind V's: P is there)
  static_assert(kV + kStagesV * kKV + kAtom <= kEnd, "within the CTA's shared memory");
  static constexpr int kTmem = 2 * R + kN <= 64 ? 64 : 2 * R + kN <= 128 ? 128 : 2 * R + kN <= 256 ? 256 : 512;
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kTile >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | (static_cast<uint32_t>(R >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (3u << 15) | (static_cast<uint32_t>(kN >> 3) << 17);
};

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

// The tiles of a call in one line: row tile after row tile of sequence after
// sequence, all K/V heads of each.  The CTAs take equal stretches of it, of
// whatever items they belong to; an item that reaches over a CTA's end leaves
// partial results, joined afterwards.
struct Stretch {
  int size, more;            // tiles of a CTA, CTAs with one more
  __device__ __forceinline__ Stretch(int total, int parts) : size(total / parts), more(total - size * parts) {}
  __device__ __forceinline__ int begin(int c) const { return c * size + min(c, more); }
  __device__ __forceinline__ int cta_of(int tile) const {
    const int edge = more * (size + 1);
    return tile < edge ? tile / (size + 1) : more + (tile - edge) / size;
  }
};
struct Walk {
  int b, rt, g;              // the item
  int tile, tiles;           // the first tile here and the item's tiles
  int left;                  // tiles of the CTA from here on
  Sequence sq;
  TileRange range;
  __device__ __forceinline__ int count() const { return min(tiles - tile, left); }
  __device__ __forceinline__ bool whole() const { return tile == 0 && left >= tiles; }
  __device__ __forceinline__ void measure(const TreeArgs &a, int R) {
    range = tile_range(a, sq, rt * R, R);
    tiles = rt * R < sq.n * a.rep ? (range.total + kTile - 1) / kTile : 0;
  }
  __device__ __forceinline__ void load(const TreeArgs &a, int R, bool report) {
    sq = sequence_of(a, b, report);
    measure(a, R);
  }
  __device__ __forceinline__ void next_pair(const TreeArgs &a, int R) {
    do {
      if (++rt == a.row_tiles) {
        rt = 0;
        if (++b == a.B) {
          left = 0;          // (cannot be: the tiles were counted)
          return;
        }
      }
      load(a, R, false);
    } while (tiles == 0);
  }
  __device__ __forceinline__ void next(const TreeArgs &a, int R) {
    left -= count();
    tile = 0;
    if (left <= 0 || ++g < a.c.n_kvh) return;
    g = 0;
    next_pair(a, R);
  }
};

// Finds the CTA's work: every thread counts the tiles of a run of (sequence,
// row tile) pairs, one of them comes upon the CTA's first tile.
template <int R, int THREADS>
__device__ __forceinline__ void find_work(const TreeArgs &a, int *smem) {
  // smem: 8 ints of the result, then one per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = THREADS / 32;
  const uint32_t pairs = static_cast<uint32_t>(a.B) * a.row_tiles;
  const uint32_t per = (pairs + THREADS - 1) / THREADS;
  const uint32_t i0 = min(pairs, per * threadIdx.x), i1 = min(pairs, i0 + per);
  Walk w;
  int mine = 0;
  auto take = [&](uint32_t i, bool report) {
    w.b = static_cast<int>(i / a.row_tiles);
    w.rt = static_cast<int>(i - static_cast<uint32_t>(w.b) * a.row_tiles);
    w.load(a, R, report && blockIdx.x == 0 && w.rt == 0);
    return w.tiles * a.c.n_kvh;
  };
  for (uint32_t i = i0; i < i1; ++i) mine += take(i, true);
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) smem[8 + warp] = before;
  if (threadIdx.x == 0) smem[0] = 0;                 // (no work unless found)
  __syncthreads();
  int sums = lane < kWarps ? smem[8 + lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += v;
  }
  const int total = __shfl_sync(0xffffffffu, sums, 31);
  const int earlier = __shfl_sync(0xffffffffu, sums, max(warp - 1, 0));
  before += (warp > 0 ? earlier : 0) - mine;
  const int parts = min(a.ctas, total);
  if (static_cast<int>(blockIdx.x) < parts) {
    const Stretch st(total, parts);
    const int begin = st.begin(blockIdx.x);
    if (begin >= before && begin < before + mine) {
      int at = before, n = mine;
      for (uint32_t i = i0; i < i1; ++i) {
        if (per > 1) n = take(i, false);
        if (begin < at + n) break;
        at += n;
      }
      w.g = (begin - at) / w.tiles;
      w.tile = begin - at - w.g * w.tiles;
      smem[0] = st.begin(blockIdx.x + 1) - begin;
      smem[1] = w.b;
      smem[2] = w.rt;
      smem[3] = w.g;
      smem[4] = w.tile;
      smem[5] = w.sq.first;
      smem[6] = w.sq.n;
      smem[7] = w.sq.ctx;
      if (a.meta) a.meta[blockIdx.x] = Meta{w.sq.first, w.sq.n, w.rt, w.g, w.tile, w.tiles, total, parts};
    }
  } else if (threadIdx.x == 0 && a.meta) {
    a.meta[blockIdx.x] = Meta{0, 0, 0, 0, 0, 0, total, parts};
  }
}
__device__ __forceinline__ Walk start_walk(const TreeArgs &a, const int *smem, int R) {
  Walk w;
  w.left = smem[0];
  w.b = smem[1];
  w.rt = smem[2];
  w.g = smem[3];
  w.tile = smem[4];
  w.sq = Sequence{smem[5], smem[6], smem[7]};
  w.tiles = 0;
  if (w.left > 0) w.measure(a, R);
  return w;
}

// Asynchronous copies, zeros where there is nothing real.  (Not ordered with
// ordinary accesses by the compiler: a ring's place is handed over by
// barriers, and the copies may go between the arithmetic of another.)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0));
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0));
}

// The fetching and decoding role of a warp: RW rows of every tile of K or of
// V.  Copies of the next tiles are on their way into its own part of a ring.
// `before` runs ahead of the wait for a tile's copies, `ready` waits for its
// place in shared memory and says whether to go on.
template <typename S, int D, int M, int R, int W, typename Before, typename Ready>
__device__ __forceinline__ void fetch_tiles(const TreeArgs &a, const int *start, uint8_t *smem, int isv, int wt, int lane,
                                            uint64_t *full, Before before, Ready ready) {
  constexpr int RW = kTile / W, kRings = S::kRings, kStages[2] = {S::kStagesK, S::kStagesV};
  constexpr int CR = S::kCodeRow, kChunks = CR / 16;         // 16-byte chunks of a row
  constexpr int BL = D / kBlock;                             // blocks of a row
  const uint32_t sbase = ptx::smem_addr(smem);
  const int total = start[0], NS = isv ? kStages[1] : kStages[0];
  const uint32_t raw = S::kRawAt + isv * S::kRawTensor + wt * RW * (CR + 4);
  // chunk c of row r lies at chunk c ^ (r / (8 / kChunks)) % kChunks, so that 8 rows' meet no bank conflict
  const uint8_t *codes = a.c.codes[isv], *scales = a.c.scales[isv];
  const int64_t code_pitch = a.c.code_pitch[isv], scale_pitch = a.c.scale_pitch[isv];

  struct Look {
    int page, off, g;                                      // off: -1 where there is no such token
  };
  Walk f = start_walk(a, start, R);                        // of the tile looked up last
  int ft = 0;
  auto look_up = [&]() {                                   // the page of this lane's row of the next tile
    Look k{0, -1, f.g};
    if (f.left <= 0) return k;
    const int p = (f.tile + ft) * kTile + wt * RW + lane % RW, real = min(p, f.range.total - 1);
    const uint32_t pg = page_of(a, real);
    k.page = a.pages[f.b * a.ldp + pg];
    k.off = p == real ? static_cast<int>(p - pg * a.page_size) : -1;
    if (++ft == f.count()) {
      ft = 0;
      f.next(a, R);
    }
    return k;
  };
  bool bad = false;
  const int in8 = lane / kChunks, swz = (in8 & 7) / (8 / kChunks) % kChunks;
  auto fetch = [&](int n, const Look &k) {                 // copies of tile n, looked up before
    const uint32_t to = sbase + raw + n % kRings * S::kRaw;
    const int64_t slot = static_cast<int64_t>(k.page) * a.page_size + k.off;
    const bool real = k.off >= 0 && k.page >= 0 && slot < a.c.n_slots;
    bad |= !real && k.off >= 0;
    const int64_t row = real ? slot * a.c.n_kvh + k.g : 0;
    if (lane < RW) copy4(to + RW * CR + 4 * lane, scales + row * scale_pitch, real);
    // (the lowest bit of an address says that the row is there)
    const uint64_t addr = reinterpret_cast<uint64_t>(codes) + static_cast<uint64_t>(row * code_pitch) + real;
    constexpr int kCopies = RW * kChunks / 32;
    uint64_t from[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) from[i] = __shfl_sync(0xffffffffu, addr, i * (32 / kChunks) + in8);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      // rows lane / kChunks of the i-th 32 / kChunks rows, chunk lane % kChunks
      const int rr = i * (32 / kChunks) + in8, c = lane % kChunks;
      const int sw = kChunks == 8 ? ((i & 1) * 4 + in8) & 7 : swz;
      copy16(to + rr * CR + ((c ^ sw) << 4), reinterpret_cast<const uint8_t *>(from[i] & ~uint64_t{1}) + 16 * c,
             from[i] & 1);
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  const int blk = (lane >> 3) % BL, row_in = (lane >> 3) / BL * 8 + (lane & 7);
  constexpr int kRows = 32 / BL, kIt = RW / kRows;         // rows per step of a warp, steps
  // where this lane reads and writes: rows step by multiples of 8, the swizzles stay
  const int r8 = lane & 7;
  uint32_t src[M / 4], dst[4];
#pragma unroll
  for (int i = 0; i < M / 4; ++i) src[i] = row_in * CR + ((blk * (M / 4) + i ^ (r8 / (8 / kChunks)) % kChunks) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[i] = (blk / 2) * kAtom + (wt * RW + row_in) * 128 + (((blk & 1) * 4 + i ^ r8) << 4);
  Walk w = start_walk(a, start, R);
  Look ahead[kRings];
#pragma unroll
  for (int n = 0; n < kRings; ++n) ahead[n] = look_up();
#pragma unroll
  for (int n = 0; n < kRings - 1; ++n) {
    if (n < total) fetch(n, ahead[n]);
    commit();
  }
  Look next = ahead[kRings - 1];
  bool ok = true;
  int n = 0;
  while (ok && w.left > 0) {
    const int nt = w.count();
    for (int t = 0; t < nt; ++t, ++n) {
      before(w, t);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRings - 2) : "memory");
      __syncwarp();
      ok = ready(w, t, n);
      if (!ok) break;
      fetch(n + kRings - 1, next);                         // (nothing behind the last tile)
      const uint8_t *from = smem + raw + n % kRings * S::kRaw;
      uint8_t *to = smem + (isv ? S::kV : S::kK) + n % NS * S::kKV;
      // (all loads first: the compiler may not take one past another row's stores)
      uint4 code[kIt][M / 4];
      uint32_t byte[kIt];
      BlockScale<M> bs[kIt];
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        byte[it] = from[RW * CR + 4 * row_in + blk + it * kRows * 4];
#pragma unroll
        for (int i = 0; i < M / 4; ++i) code[it][i] = *reinterpret_cast<const uint4 *>(from + src[i] + it * kRows * CR);
      }
#pragma unroll
      for (int it = 0; it < kIt; ++it) bs[it] = block_scale<M>(smem + S::kTable, byte[it]);
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const uint32_t *wd = reinterpret_cast<const uint32_t *>(&code[it][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(to + dst[j] + it * kRows * 128) =
              decode8<M>(wd[j * M / 4], M == 8 ? wd[j * M / 4 + 1] : 0, bs[it]);
      }
      commit();
      ptx::fence_async_shared();
      arrive_warp(full + n % NS, lane);                      // (and the ring's place may be written again)
      next = look_up();
    }
    if (ok) w.next(a, R);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (bad) record_bad_index(a.status);
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 8) {
    ptx::tmem_ld8(addr, r);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 16) ptx::tmem_ld16(addr + i, *reinterpret_cast<uint32_t(*)[16]>(&r[i]));
  }
  ptx::tmem_wait_ld();
}

}  // namespace

// A persistent grid: CTA = a stretch of the line of tiles, one tile of 128
// tokens of a (sequence, row tile, K/V head) after the other.  Tokens are the
// 128 rows of the matrix instruction, query rows its columns, so that the
// work follows the number of rows (16 to 64 of them) while a cache tile is
// decoded once for all of them:
//   S^T [token][row] = K Q^T     A = K  (token x d, K-major),  B = Q
//   O^T [d][row]    += V^T P^T   A = V  (token x d, stored along d), B = P
// Both accumulate in tensor memory.  Eight warps fetch (asynchronous copies,
// a tile or two ahead) and decode the cache into shared memory, half K and
// half V; one warp issues the products; eight warps turn scores into weights, four
// for each half of the columns.  A softmax thread owns one token and sums its
// weights per row over all tiles; the sums meet at an item's end.
//   The running maximum of a row is a reference that weights are relative
// to, common to all tokens: it is set by an item's first tile and moved only
// when a score passes it by more than 24 (weights of 2^24), which fp32 and
// bf16 hold with no loss of precision; so a tile usually needs no maximum
// over its tokens, only one vote that none of its scores is above.
//   The tensor core's fp32 sums are rounded towards zero at every step: an
// fp32 output is taken out of tensor memory every kPeriod tiles and summed
// outside it (7-token trees over 8191 tokens: 3.5e-6 of the exact result
// without that, 0.9e-6 with it).  A bf16 output stays there: the error is
// small next to the output's own rounding up to some 2^18 tokens of one CTA.
//   Weights enter the product with V as P bf16 pieces: one for a bf16 output,
// each weight off by up to 2^-8 of itself, which adds as much as the output's
// rounding does (2.3e-3 of the result in all, 1.7e-3 with fp32 weights);
// three for an fp32 output, 24 bits.  With three, trees of 16 take 43.6 us
// where one takes 36.7, and the products of the wide form would triple; a
// caller who needs the difference asks for fp32.
//   Trees of up to 16 tokens over 8 contexts of up to 4096 (64 rows of 128,
// 4 bits): 36 us, of which 10.8 tiles per SM are 16 (2900 cycles each) and
// finding the work, the first tile and joining the rest; the cache's 29.6 MB
// need 4.5.  7-token trees over 32 contexts of up to 8191 (21 rows of 64,
// 8 bits, fp32 output): 149 us, issue slots 0.62 busy, DRAM 0.50; 211 MB need
// 32, and 583 are read.
template <int D, int M, int R, int P, bool FOUT>
__global__ void __launch_bounds__(Shape<D, M, R, P>::kThreads, 1) tree_kernel(TreeArgs a) {
  using S = Shape<D, M, R, P>;
  constexpr int C = S::kCols, SK = S::kStagesK, SV = S::kStagesV;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler keeps to shared-memory instructions)
  uint8_t *smem = smem_raw + (-ptx::smem_addr(smem_raw) & 1023u);
  // (ref: the references, negated)
  float *ref = reinterpret_cast<float *>(smem + S::kStat), *factor = ref + R, *wstat = factor + R;   // wstat[4][R]
  int64_t *place = reinterpret_cast<int64_t *>(smem + S::kPlace);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::kBar);
  uint64_t *s_done = bar, *p_full = bar + 2, *o_done = bar + 4, *k_full = bar + 6, *v_full = bar + 8, *drained = bar + 12;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 10);
  volatile int *given_up = reinterpret_cast<int *>(tmem_slot + 1);
  int *start = reinterpret_cast<int *>(smem + S::kStart);
  const int warp = ptx::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(k_full + i, S::kFetchWarps);
      ptx::mbar_init(v_full + i, S::kFetchWarps);
      ptx::mbar_init(s_done + i, 1);
      ptx::mbar_init(p_full + i, S::kSoftWarps);
      ptx::mbar_init(o_done + i, 1);
    }
    ptx::mbar_init(drained, 1);
    ptx::fence_mbar_init();
    *given_up = 0;
  }
  for (int i = threadIdx.x; i < R; i += S::kThreads) ref[i] = INFINITY;
  fill_table<M, S::kThreads>(smem + S::kTable);
  pdl_wait();
  // tensor memory is taken after the wait for earlier kernels and before
  // later ones may start: a CTA that waits for another kernel holds none
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, S::kTmem);
    ptx::tmem_relinquish();
  }
  find_work<R, S::kThreads>(a, start);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + 2 * R;
  const uint32_t sbase = ptx::smem_addr(smem);

  if (warp == S::kMmaWarp) {
    // ------------------------------------------------------ matrix products
    // The whole warp goes through them, so that their operands are worked out
    // once for it, and one elected lane issues (from inside a lane's branch
    // each product took over 100 cycles to issue).
    const uint32_t leader = ptx::elect_one();
    auto scores = [&](int n) {                               // waits for K(n); the place of its scores is free
      if (!__all_sync(0xffffffffu, wait_phase(k_full + n % SK, (n / SK) & 1, given_up, a.status))) return false;
      ptx::tc_fence_after();
      const uint64_t kd = ptx::desc_sw128(ptx::uniform(sbase + S::kK + (n % SK) * S::kKV)), qd = ptx::desc_sw128(sbase + S::kQ);
      const uint32_t to = ptx::uniform(tmem + (n & 1) * R);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ptx::mma_bf16_by(leader, to, kd + (((k / 4) * kAtom + (k % 4) * 32) >> 4),
                         qd + (((k / 4) * (R * 128) + (k % 4) * 32) >> 4), S::kIdescS, k > 0);
      ptx::mma_commit_by(leader, s_done + (n & 1));
      return true;
    };
    Walk w = start_walk(a, start, R);
    const int total = start[0];
    const uint32_t limit = g_tree_wait;
    uint32_t since = clock();
    bool late = false;
    bool ok = total == 0 || scores(0);
    for (int n = 0; ok && w.left > 0; w.next(a, R)) {
      const int nt = w.count();
      for (int t = 0; t < nt && ok; ++t, ++n) {
        // (the scores of n + 1 go where those of n - 1 were: their weights have been waited for)
        if (n + 1 < total) ok = scores(n + 1);
        ok = ok && !late && wait_phase(v_full + n % SV, (n / SV) & 1, given_up, a.status) &&
             wait_phase(p_full + (n & 1), (n >> 1) & 1, given_up, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t more = ptx::uniform((P > 1 ? t % kPeriod : t) != 0);
        const uint64_t vd = ptx::desc_mn<64>(ptx::uniform(sbase + S::kV + (n % SV) * S::kKV), kAtom);
        const uint64_t pd = ptx::desc_mn<S::kPWidth>(ptx::uniform(sbase + S::kP + n % S::kPBufs * S::kPBytes), S::kPAtom);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          ptx::mma_bf16_by(leader, ptx::uniform(tmem_o), vd + k * (2048 >> 4), pd + k * (32 * S::kPWidth >> 4), S::kIdescO,
                           k > 0 ? 1u : more);
        ptx::mma_commit_by(leader, o_done + (n & 1));
        late = !in_time(since, limit, given_up, a.status);
      }
    }
    if (total > 0) drain(leader, drained, a.status);
    __syncwarp();
  } else if (warp >= S::kSoftWarps) {
    // ------------------------------------------------- fetching and decoding
    constexpr int W = S::kFetchWarps;
    const int dw = warp - S::kSoftWarps, wt = dw % W, isv = dw / W;
    if constexpr (S::kMoveRegisters) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    constexpr int kQ = (R * D / 8 + W * 32 - 1) / (W * 32);  // 16-byte chunks of q per thread of K's warps
    uint4 qv[kQ];
    auto before = [&](const Walk &w, int t) {
      if (t > 0 || isv) return;
      // q of a new item: row c of the tile, zero where there is no such row
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int j = (i * W + wt) * 32 + lane, c = j / (D / 8), e = j - c * (D / 8);
        const int rr = w.rt * R + c, di = rr / a.rep, h = rr - di * a.rep;
        qv[i] = make_uint4(0, 0, 0, 0);
        if (di < w.sq.n && c < R)
          qv[i] = *reinterpret_cast<const uint4 *>(a.q + (w.sq.first + di) * a.ldqt + (w.g * a.rep + h) * a.ldqh + e * 8);
      }
    };
    auto ready = [&](const Walk &, int t, int n) {
      // the place of tile u is taken; for a new q, every score of the old one has to be there
      const int u = t == 0 && !isv ? n - 1 : n - (isv ? SV : SK);
      bool ok = true;
      if (u >= 0) ok = wait_phase((isv ? o_done : s_done) + (u & 1), (u >> 1) & 1, given_up, a.status);
      if (!__all_sync(0xffffffffu, ok)) return false;
      if (t == 0 && !isv) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int j = (i * W + wt) * 32 + lane, c = j / (D / 8), e = j - c * (D / 8);
          if (c < R)
            *reinterpret_cast<uint4 *>(smem + S::kQ + (e / 8) * (R * 128) + c * 128 + (((e & 7) ^ (c & 7)) << 4)) =
                reorder8<M>(qv[i]);
        }
      }
      return true;
    };
    fetch_tiles<S, D, M, R, W>(a, start, smem, isv, wt, lane, isv ? v_full : k_full, before, ready);
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (S::kMoveRegisters) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    const int grp = warp >> 2, w4 = warp & 3;
    const int tok = w4 * 32 + lane, col0 = grp * C;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    constexpr int CC = C < 16 ? C : 16;
    // the swizzle of a row of 128, 64 or 32 bytes
    const int pswz = S::kPWidth == 64 ? tok & 7 : S::kPWidth == 32 ? (tok >> 1) & 3 : (tok >> 2) & 1;
    float *acc = reinterpret_cast<float *>(smem + S::kAcc) + col0 * D + tok;
    const int e = true_position<M>(tok);
    Walk w = start_walk(a, start, R);
    bool ok = true, first = true;
    int n = 0;
    while (ok && w.left > 0) {
      const int nt = w.count(), row0 = w.rt * R;
      float sum[C];
#pragma unroll
      for (int k = 0; k < C; ++k) sum[k] = 0.f;
      for (int t = 0; t < nt; ++t, ++n) {
        ok = wait_phase(s_done + (n & 1), (n >> 1) & 1, given_up, a.status);
        ptx::tc_fence_after();
        const bool masked = (w.tile + t + 1) * kTile > w.range.open;
        // bit lane of shfl(seen(), k): does this token's column k see it
        auto seen = [&] {
          return seen_tokens(a, w.sq, (row0 + col0 + lane % C) / a.rep, (w.tile + t) * kTile + w4 * 32 - w.sq.ctx);
        };
        uint32_t s[C];
        tmem_load(tmem + lanes + (n & 1) * R + col0, s);
        float v[C], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < C; k += 4) {
          const float4 r = *reinterpret_cast<const float4 *>(ref + col0 + k);
          scale_shift(v[k], v[k + 1], s[k], s[k + 1], a.scale_log2, r.x, r.y);
          scale_shift(v[k + 2], v[k + 3], s[k + 2], s[k + 3], a.scale_log2, r.z, r.w);
        }
        if (masked) {
          const uint32_t mine = seen();
#pragma unroll
          for (int k = 0; k < C; ++k) v[k] = __shfl_sync(0xffffffffu, mine, k) >> lane & 1u ? v[k] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < C; k += 2) top = max3(top, v[k], v[k + 1]);
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = exp2_fast(v[k]);
        // (the vote below also carries a wait that ran out: all of the group leave together)
        if (n >= S::kPBufs) {
          const int u = n - S::kPBufs;
          ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status) && ok;
        }
        const bool flush = P > 1 && t > 0 && t % kPeriod == 0;
        if (any_of(grp, top > kSlack || !ok || flush)) {
          // rare: a reference is overtaken (or not set yet), or an output period ends
          if (t > 0 && ok) {
            const int u = n - 1;
            ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
            ptx::tc_fence_after();
          }
          if (any_of(grp, !ok)) {
            ok = false;
            break;
          }
          tmem_load(tmem + lanes + (n & 1) * R + col0, s);
#pragma unroll
          for (int k = 0; k < C; ++k) v[k] = __uint_as_float(s[k]) * a.scale_log2;
          if (masked) {
            const uint32_t mine = seen();
#pragma unroll
            for (int k = 0; k < C; ++k) v[k] = __shfl_sync(0xffffffffu, mine, k) >> lane & 1u ? v[k] : -INFINITY;
          }
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
            const float old = -ref[c];
            float m = fmaxf(fmaxf(wstat[c], wstat[R + c]), fmaxf(wstat[2 * R + c], wstat[3 * R + c]));
            m = m - old > kSlack || old == -INFINITY ? m : old;
            factor[c] = m == old ? 1.f : exp2f(old - m);
            ref[c] = -m;
          }
          group_sync(grp);
#pragma unroll
          for (int k = 0; k < C; ++k) {
            sum[k] *= factor[col0 + k];
            v[k] = v[k] == -INFINITY ? 0.f : exp2_fast(v[k] + ref[col0 + k]);
          }
          if (t > 0) {
#pragma unroll 1
            for (int c0 = 0; c0 < C; c0 += CC) {
              float part[CC];
#pragma unroll
              for (int k = 0; k < CC; ++k) part[k] = 0.f;
#pragma unroll 1
              for (int q = P - 1; q >= 0; --q) {
                uint32_t o[CC];
                tmem_load(tmem_o + lanes + q * R + col0 + c0, o);
                if (flush) {
#pragma unroll
                  for (int k = 0; k < CC; ++k) part[k] += __uint_as_float(o[k]);
                } else {
#pragma unroll
                  for (int k = 0; k < CC; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[col0 + c0 + k]);
                  if constexpr (CC == 8) ptx::tmem_st8(tmem_o + lanes + q * R + col0 + c0, o);
                  else ptx::tmem_st16(tmem_o + lanes + q * R + col0 + c0, o);
                }
              }
              if (P > 1 && tok < D && (flush || t > kPeriod)) {
#pragma unroll
                for (int k = 0; k < CC; ++k) {
                  float *z = acc + (c0 + k) * D;
                  *z = ((t > kPeriod ? *z : 0.f) + part[k]) * factor[col0 + c0 + k];
                }
              }
            }
            ptx::tmem_wait_st();
          }
          group_sync(grp);                           // (factor and wstat may be written again)
        }
        // the weights as P bf16 pieces, each the rounding of what the ones before left
        uint8_t *prow = smem + S::kP + n % S::kPBufs * S::kPBytes + tok * (2 * S::kPWidth);
#pragma unroll
        for (int k = 0; k < C; k += 2) add2(sum[k], sum[k + 1], v[k], v[k + 1]);
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
        arrive_warp(p_full + (n & 1), lane);
      }
      if (!ok) break;
      // the sums over the tokens: lanes, then warps, in a fixed order
      const float mine = over_lanes(sum, lane, [](float p, float q) { return p + q; });
      if (lane % (32 / C) == 0) wstat[w4 * R + col0 + lane / (32 / C)] = mine;
      const bool whole = w.whole();
      group_sync(grp);
      if (tok < C) {
        const int c = col0 + tok, i = (row0 + c) / a.rep, h = row0 + c - i * a.rep;
        const float l = (wstat[c] + wstat[R + c]) + (wstat[2 * R + c] + wstat[3 * R + c]);
        const float lse2 = l == 0.f ? -INFINITY : log2f(l) - ref[c];
        const int64_t row = w.sq.first + i, head = w.g * a.rep + h;
        factor[c] = l == 0.f ? 0.f : 1.f / l;
        ref[c] = INFINITY;
        int64_t z = -1;
        if (i < w.sq.n) {
          if (whole) {
            z = row * a.ldot + head * a.ldoh;
            if (a.lse) a.lse[row * a.n_qh + head] = lse2 * kLn2;
          } else {
            // a CTA has at most two unfinished items, its first and its last
            z = (static_cast<int64_t>(blockIdx.x) * 2 + !first) * R + c;
            a.part_lse[z] = lse2;
            z *= D;
          }
        }
        place[c] = z;
      }
      group_sync(grp);
      {
        const int u = n - 1;
        ok = wait_phase(o_done + (u & 1), (u >> 1) & 1, given_up, a.status);
        ptx::tc_fence_after();
      }
      if (any_of(grp, !ok)) break;
      // out: thread = position tok of the head, one column after the other
#pragma unroll 1
      for (int c0 = 0; c0 < C; c0 += CC) {
        float o[CC];
#pragma unroll
        for (int k = 0; k < CC; ++k) o[k] = 0.f;
#pragma unroll
        for (int q = P - 1; q >= 0; --q) {
          uint32_t r[CC];
          tmem_load(tmem_o + lanes + q * R + col0 + c0, r);
#pragma unroll
          for (int k = 0; k < CC; ++k) o[k] += __uint_as_float(r[k]);
        }
        if (tok < D) {
#pragma unroll
          for (int k = 0; k < CC; ++k) {
            const int c = col0 + c0 + k;
            if (place[c] < 0) continue;
            float y = o[k];
            if (P > 1 && nt > kPeriod) y += acc[(c0 + k) * D];
            y = factor[c] == 0.f ? 0.f : y * factor[c];
            const int64_t z = place[c] + e;
            if (!whole) a.part[z] = y;
            else if constexpr (FOUT) static_cast<float *>(a.out)[z] = y;
            else static_cast<__nv_bfloat16 *>(a.out)[z] = __float2bfloat16(y);
          }
        }
      }
      first = false;
      w.next(a, R);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, S::kTmem);
}

// Shared memory of tree_rows_kernel, filled like Shape.
template <int D, int M>
struct RowsShape {
  static constexpr int kSoftWarps = 16, kFetchWarps = 4, kMmaWarp = kSoftWarps + 2 * kFetchWarps;
  static constexpr int kThreads = (kMmaWarp + 1) * 32;
  static constexpr int kKV = kTile * D * 2;
  static constexpr int kCodeRow = D * M / 8;
  static constexpr int kRawTensor = kTile * (kCodeRow + 4);
  static constexpr int kRaw = 2 * kRawTensor;
  static constexpr int kQHalf = 128 * D * 2;                 // 128 rows of q
  static constexpr int kSmall = 16 * 8 + 256 + 256 * kTableEntry<M> + 512 * 4;
  static constexpr int kRoom = 227 * 1024 - 1024 - kSmall;
  static constexpr int kOnce = 2 * kKV + 2 * kQHalf + 2 * kRaw;
  static constexpr int kRings = kOnce + kRaw <= kRoom ? 3 : 2;
  static constexpr int kWithRaw = kOnce + (kRings - 2) * kRaw;
  static constexpr int kStagesV = kWithRaw + kKV <= kRoom ? 2 : 1;     // (V is waited for first)
  static constexpr int kWithV = kWithRaw + (kStagesV - 1) * kKV;
  static constexpr int kStagesK = kWithV + kKV <= kRoom ? 2 : 1;
  static constexpr int kK = 0, kV = kStagesK * kKV, kQ = kV + kStagesV * kKV;
  static constexpr int kRawAt = kQ + 2 * kQHalf;
  static constexpr int kBar = kRawAt + kRings * kRaw;
  static constexpr int kStart = kBar + 16 * 8;
  static constexpr int kTable = kStart + 256;
  static constexpr int kSwap = kTable + 256 * kTableEntry<M>;    // a maximum or sum of each softmax thread
  static constexpr int kBytes = kSwap + 512 * 4 + 1024;
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(128 >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | (static_cast<uint32_t>(kTile >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17);
  static constexpr int kTmemO = 2 * kTile, kTmem = 512;
};

// The same for many rows: query rows are the matrix instruction's rows, twice
// 128 of them per CTA, so that a cache tile is decoded once for 256 rows and
// the products run at full width:
//   S [row][token] = Q K^T       A = Q  (row x d, K-major),     B = K
//   O [row][d]    += P V         A = P  (tensor memory, in S's place), B = V
// The two halves take turns: while one's scores become weights the other's
// products run.  Two softmax threads share a row, 64 tokens of a tile and half
// of its output each (one thread with all 128 took 329 us where two take less:
// a half's products wait for its weights, so their latency counts).  The
// maximum that weights are relative to moves, by a vote of the half, when a
// score passes it by more than kSlack.
//   64-token trees over 2 contexts of up to 65536 (512 rows of 128, 4 bits):
// 287 us, tensor pipe 0.45 and exponentials 0.46 busy; 235 GFLOP need 143.
// Each half's chain of scores, weights and product holds it.  Weights are one
// bf16 piece (see tree_kernel): a second would fill the place of the scores
// while half of them are still to be read, and run the output product twice.
template <int D, int M>
__global__ void __launch_bounds__(RowsShape<D, M>::kThreads, 1) tree_rows_kernel(TreeArgs a) {
  using S = RowsShape<D, M>;
  constexpr int R = 256, SK = S::kStagesK, SV = S::kStagesV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-ptx::smem_addr(smem_raw) & 1023u);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::kBar);
  uint64_t *s_done = bar, *p_full = bar + 2, *o_done = bar + 4, *k_full = bar + 6, *v_full = bar + 8, *k_free = bar + 10,
           *v_free = bar + 12, *drained = bar + 14;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 15);
  volatile int *given_up = reinterpret_cast<int *>(tmem_slot + 1);
  int *start = reinterpret_cast<int *>(smem + S::kStart);
  const int warp = ptx::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_done + i, 1);
      ptx::mbar_init(p_full + i, 8);
      ptx::mbar_init(o_done + i, 1);
      ptx::mbar_init(k_full + i, S::kFetchWarps);
      ptx::mbar_init(v_full + i, S::kFetchWarps);
      ptx::mbar_init(k_free + i, 1);
      ptx::mbar_init(v_free + i, 1);
    }
    ptx::mbar_init(drained, 1);
    ptx::fence_mbar_init();
    *given_up = 0;
  }
  fill_table<M, S::kThreads>(smem + S::kTable);
  pdl_wait();
  if (warp == S::kMmaWarp) {
    ptx::tmem_alloc(tmem_slot, S::kTmem);
    ptx::tmem_relinquish();
  }
  find_work<R, S::kThreads>(a, start);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = ptx::smem_addr(smem);
  const int total = start[0];
  // halves of an item that have rows
  auto halves = [&](const Walk &w) { return w.sq.n * a.rep - w.rt * R > 128 ? 2 : 1; };

  if (warp == S::kMmaWarp) {
    // ------------------------------------------------------ matrix products
    const uint32_t leader = ptx::elect_one();
    const uint32_t limit = g_tree_wait;
    uint32_t since = clock();
    bool ok = true;
    auto await = [&](uint64_t *b, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && wait_phase(b, parity, given_up, a.status));
      ptx::tc_fence_after();
      return ok;
    };
    auto scores = [&](int n, int q) {
      const uint64_t qd = ptx::desc_sw128(ptx::uniform(sbase + S::kQ + q * S::kQHalf));
      const uint64_t kd = ptx::desc_sw128(ptx::uniform(sbase + S::kK + n % SK * S::kKV));
      const uint32_t to = ptx::uniform(tmem + q * kTile);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t step = ((k / 4) * kAtom + (k % 4) * 32) >> 4;
        ptx::mma_bf16_by(leader, to, qd + step, kd + step, S::kIdescS, k > 0);
      }
      ptx::mma_commit_by(leader, s_done + q);
    };
    auto output = [&](int n, int q, uint32_t more) {
      const uint64_t vd = ptx::desc_mn<64>(ptx::uniform(sbase + S::kV + n % SV * S::kKV), kAtom);
      const uint32_t from = ptx::uniform(tmem + q * kTile), to = ptx::uniform(tmem + S::kTmemO + q * D);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        ptx::mma_bf16_ts_by(leader, to, from + (k / 4) * 64 + (k % 4) * 8, vd + k * (2048 >> 4), S::kIdescO, k > 0 ? 1u : more);
      ptx::mma_commit_by(leader, o_done + q);
    };
    Walk w = start_walk(a, start, R);
    int n = 0, done[2] = {0, 0};                     // tiles so far, of each half
    if (total > 0 && await(k_full, 0)) {
      const int nq = halves(w);
      for (int q = 0; q < nq; ++q) scores(0, q);
      ptx::mma_commit_by(leader, k_free);
    }
    while (ok && w.left > 0) {
      const int nt = w.count(), nq = halves(w);
      Walk after = w;
      after.next(a, R);
      for (int t = 0; t < nt && ok; ++t, ++n) {
        const int nq2 = t + 1 < nt ? nq : after.left > 0 ? halves(after) : 0;
        await(v_full + n % SV, (n / SV) & 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q < nq && ok && await(p_full + q, done[q] & 1)) {
            ++done[q];
            output(n, q, t > 0);
            if (q == nq - 1) ptx::mma_commit_by(leader, v_free + n % SV);
          }
          // (the next scores of this half go where its weights were: behind their product, in order)
          if (q < nq2 && ok && (q > 0 || await(k_full + (n + 1) % SK, ((n + 1) / SK) & 1))) {
            scores(n + 1, q);
            if (q == nq2 - 1) ptx::mma_commit_by(leader, k_free + (n + 1) % SK);
          }
        }
        ok = __all_sync(0xffffffffu, ok && in_time(since, limit, given_up, a.status));
      }
      w = after;
    }
    if (total > 0) drain(leader, drained, a.status);
    __syncwarp();
  } else if (warp >= S::kSoftWarps) {
    // ------------------------------------------------- fetching and decoding
    constexpr int W = S::kFetchWarps;
    const int dw = warp - S::kSoftWarps, wt = dw % W, isv = dw / W;
    auto before = [](const Walk &, int) {};
    auto ready = [&](const Walk &w, int t, int n) {
      bool ok = true;
      if (isv) {
        if (n >= SV) ok = wait_phase(v_free + n % SV, ((n - SV) / SV) & 1, given_up, a.status);
        return __all_sync(0xffffffffu, ok) != 0;
      }
      const int u = t == 0 ? n - 1 : n - SK;
      if (u >= 0) ok = wait_phase(k_free + u % SK, (u / SK) & 1, given_up, a.status);
      if (!__all_sync(0xffffffffu, ok)) return false;
      if (t == 0) {
        // q of a new item, zero where there is no such row; negated for a negative scale
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        constexpr int B = 8, kQ = R * D / 8 / (W * 32);
#pragma unroll 1
        for (int i0 = 0; i0 < kQ; i0 += B) {
          uint4 v[B];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const int j = ((i0 + i) * W + wt) * 32 + lane, c = j / (D / 8), e = j - c * (D / 8);
            const int rr = w.rt * R + c, di = rr / a.rep, h = rr - di * a.rep;
            v[i] = make_uint4(0, 0, 0, 0);
            if (di < w.sq.n)
              v[i] = *reinterpret_cast<const uint4 *>(a.q + (w.sq.first + di) * a.ldqt + (w.g * a.rep + h) * a.ldqh + e * 8);
          }
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const int j = ((i0 + i) * W + wt) * 32 + lane, c = j / (D / 8), e = j - c * (D / 8);
            v[i] = reorder8<M>(v[i]);
            *reinterpret_cast<uint4 *>(smem + S::kQ + (c / 128) * S::kQHalf + (e / 8) * kAtom + (c % 128) * 128 +
                                       (((e & 7) ^ (c & 7)) << 4)) =
                make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
          }
        }
      }
      return true;
    };
    fetch_tiles<S, D, M, R, W>(a, start, smem, isv, wt, lane, isv ? v_full : k_full, before, ready);
  } else {
    // -------------------------------------------------------------- softmax
    const int q = warp >> 3, part = (warp >> 2) & 1, tok = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // this thread's 64 scores, with its weights in their first 32 columns, and its half of the output
    const uint32_t tmem_s = tmem + lanes + q * kTile + part * 64, tmem_o = tmem + lanes + S::kTmemO + q * D + part * (D / 2);
    float *mine = reinterpret_cast<float *>(smem + S::kSwap) + (warp >> 2) * 128 + tok;
    const float *other = reinterpret_cast<float *>(smem + S::kSwap) + ((warp >> 2) ^ 1) * 128 + tok;
    const float scale = fabsf(a.scale_log2);
    Walk w = start_walk(a, start, R);
    bool ok = true, first = true;
    int done = 0;                                    // tiles of this half
    for (; ok && w.left > 0; first = false, w.next(a, R)) {
      if (q >= halves(w)) continue;
      const int nt = w.count(), rr = w.rt * R + q * 128 + tok, i = rr / a.rep, h = rr - i * a.rep;
      float m = -INFINITY, l0 = 0.f, l1 = 0.f;
      for (int t = 0; t < nt; ++t, ++done) {
        ok = wait_phase(s_done + q, done & 1, given_up, a.status);
        if (done > 0) ok = wait_phase(o_done + q, (done - 1) & 1, given_up, a.status) && ok;
        ptx::tc_fence_after();
        const bool masked = (w.tile + t + 1) * kTile > w.range.open;
        const int j0 = (w.tile + t) * kTile + part * 64 - w.sq.ctx;
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t s[32];
          tmem_load(tmem_s + c, s);
          if (masked) {
            const uint32_t see = seen_tokens(a, w.sq, i, j0 + c);
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1u ? s[k] : 0xFF800000u;
          }
#pragma unroll
          for (int k = 0; k < 32; k += 2) top = max3(top, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
        }
        top = top == -INFINITY ? top : top * scale;
        // (the vote also carries a wait that ran out: all of the half leave together)
        if (any_of256(q, top > m + kSlack || (m == -INFINITY && top != m) || !ok)) {
          *mine = ok ? top : NAN;
          half_sync(q);
          const float both = fmaxf(top, *other);
          if (any_of256(q, !ok)) {
            ok = false;
            break;
          }
          const bool up = both > m + kSlack || (m == -INFINITY && both != m);
          if (__any_sync(0xffffffffu, up)) {
            const float f = up ? exp2f(m - both) : 1.f;
            l0 *= f;
            l1 *= f;
            if (up) m = both;
            if (t > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                tmem_load(tmem_o + c, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                ptx::tmem_st16(tmem_o + c, o);
              }
            }
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t s[32];
          tmem_load(tmem_s + c, s);
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; k += 2) scale_shift(v[k], v[k + 1], s[k], s[k + 1], scale, shift, shift);
          if (masked) {
            const uint32_t see = seen_tokens(a, w.sq, i, j0 + c);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = (see >> k) & 1u ? v[k] : -INFINITY;
          }
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            v[2 * k] = exp2_fast(v[2 * k]);
            v[2 * k + 1] = exp2_fast(v[2 * k + 1]);
            add2(l0, l1, v[2 * k], v[2 * k + 1]);
            p[k] = pack2(v[2 * k], v[2 * k + 1]);
          }
          ptx::tmem_st16(tmem_s + c / 2, p);         // (over scores that have been read)
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        arrive_warp(p_full + q, lane);
      }
      if (!ok) break;
      *mine = l0 + l1;
      ok = wait_phase(o_done + q, (done - 1) & 1, given_up, a.status);
      if (any_of256(q, !ok)) break;
      ptx::tc_fence_after();
      // (the same order in both threads)
      const float l = part ? *other + (l0 + l1) : (l0 + l1) + *other, inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
      const bool whole = w.whole(), has = i < w.sq.n;
      const int64_t row = w.sq.first + i, head = w.g * a.rep + h;
      // a CTA has at most two unfinished items, its first and its last
      const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + !first) * R + q * 128 + tok;
      if (has && whole && a.lse && !part) a.lse[row * a.n_qh + head] = lse2 * kLn2;
      if (has && !whole && !part) a.part_lse[slot] = lse2;
      uint16_t *out = static_cast<uint16_t *>(a.out) + row * a.ldot + head * a.ldoh + part * (D / 2);
      // (unfinished: chunks of four positions, [chunk][row])
      float4 *left = reinterpret_cast<float4 *>(a.part) +
                     ((static_cast<int64_t>(blockIdx.x) * 2 + !first) * (D / 4) + part * (D / 8)) * R + q * 128 + tok;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t o[16];
        tmem_load(tmem_o + c, o);
        if (!has) continue;
#pragma unroll
        for (int g8 = 0; g8 < 16; g8 += 8) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float z = __uint_as_float(o[g8 + k]);
            y[true_position<M>(k)] = inv == 0.f ? 0.f : z * inv;
          }
          if (!whole) {
            left[(c + g8) / 4 * R] = make_float4(y[0], y[1], y[2], y[3]);
            left[((c + g8) / 4 + 1) * R] = make_float4(y[4], y[5], y[6], y[7]);
          } else if (a.out_vec) store8<false>(out, c + g8, y);
          else
#pragma unroll
            for (int k = 0; k < 8; ++k) store1<false>(out, c + g8 + k, y[k]);
        }
      }
      half_sync(q);                                  // (the sums have been read)
      ptx::tc_fence_before();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == S::kMmaWarp) ptx::tmem_dealloc(tmem, S::kTmem);
}

// Joins an item's partial results, weighted by 2^(lse_j - lse) in the order
// of the CTAs.  Block (c, chunk of 8 W columns) takes the item that CTA c found
// begun by the CTA before it, if that was the item's first; a warp takes W
// columns, whose loads are in flight together.
template <int R>
constexpr int kJoinColumns = R >= 64 ? 2 : 1;
template <int D, int R, bool FOUT>
__global__ void __launch_bounds__(256) tree_combine_kernel(TreeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = D / 32, W = kJoinColumns<R>;
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
  const Meta m = a.meta[c];
  if (c >= m.parts || m.tile == 0) return;
  const Stretch st(m.total, m.parts);
  const int begin = st.begin(c), before = begin - st.begin(c - 1);
  if (m.tile > before) return;                       // an earlier CTA began it
  const int col = (blockIdx.y * 8 + (threadIdx.x >> 5)) * W;
  const int columns = min(W, m.n * a.rep - m.rt * R - col);
  if (columns <= 0) return;
  // parts: CTA c - 1 (its first or its last item), then the first items of c, c + 1, ... up to the item's end
  const int n = st.cta_of(begin - m.tile + m.tiles - 1) - c + 2;
  // (columns behind the last row: read, as the workspace has them, and not used)
  const int64_t slot0 = ((static_cast<int64_t>(c) - 1) * 2 + (m.tile < before)) * R + col;
  const int64_t slot1 = static_cast<int64_t>(c) * 2 * R + col - 2 * R;
  auto part_of = [&](int j) { return j == 0 ? slot0 : slot1 + j * (2 * R); };
  float top[W], near[W];                             // near: part `lane`'s
  bool nan[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    top[w] = near[w] = -INFINITY;
    nan[w] = false;
  }
  for (int j = lane; j < n; j += 32) {
    const float *l = a.part_lse + part_of(j);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float x = l[w];
      if (j < 32) near[w] = x;
      nan[w] |= x != x;
      top[w] = fmaxf(top[w], x);
    }
  }
  float total[W], acc[W][E];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    nan[w] = __any_sync(0xffffffffu, nan[w]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], o));
    total[w] = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) acc[w][k] = 0.f;
  }
  for (int j0 = 0; j0 < n; j0 += 32) {
    float weight[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (j0 > 0) near[w] = j0 + lane < n ? a.part_lse[part_of(j0 + lane) + w] : -INFINITY;
      weight[w] = top[w] == -INFINITY ? 0.f : exp2f(near[w] - top[w]);
    }
    const int m32 = min(32, n - j0);
#pragma unroll 8 / W
    for (int j = 0; j < m32; ++j) {
      const float *p = a.part + part_of(j0 + j) * D + lane * E;
      float v[W][E];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if constexpr (E == 4) *reinterpret_cast<float4 *>(v[w]) = *reinterpret_cast<const float4 *>(p + w * D);
        else *reinterpret_cast<float2 *>(v[w]) = *reinterpret_cast<const float2 *>(p + w * D);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = __shfl_sync(0xffffffffu, weight[w], j);
        total[w] += f;
#pragma unroll
        for (int k = 0; k < E; ++k) acc[w][k] = fmaf(f, v[w][k], acc[w][k]);
      }
    }
  }
  int i = (m.rt * R + col) / a.rep, h = m.rt * R + col - i * a.rep;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w >= columns) break;
    const int64_t row = m.first + i, head = m.g * a.rep + h;
    const float inv = nan[w] ? NAN : total[w] == 0.f ? 0.f : 1.f / total[w];
    const int64_t at = row * a.ldot + head * a.ldoh + lane * E;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float y = total[w] == 0.f && !nan[w] ? 0.f : acc[w][k] * inv;
      if constexpr (FOUT) static_cast<float *>(a.out)[at + k] = y;
      else static_cast<__nv_bfloat16 *>(a.out)[at + k] = __float2bfloat16(y);
    }
    if (a.lse && lane == 0)
      a.lse[row * a.n_qh + head] = nan[w] ? NAN : total[w] == 0.f ? -INFINITY : (top[w] + log2f(total[w])) * kLn2;
    if (++h == a.rep) {
      h = 0;
      ++i;
    }
  }
}

// The same behind tree_rows_kernel, whose partial outputs lie in chunks of
// four positions, [chunk][row]: lane = row in the reads here as in the writes
// there (row after row instead, 16 bytes of 32 rows per instruction, the
// chunked prompt of 211 tokens took 73 us).  Block (c, 32 rows, 64
// positions); a warp takes two chunks, four parts in flight.
template <int D>
__global__ void __launch_bounds__(256) tree_rows_combine_kernel(TreeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int R = 256, C = 2;
  const int c = blockIdx.x + 1, warp = blockIdx.z * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Meta m = a.meta[c];
  if (c >= m.parts || m.tile == 0) return;
  const Stretch st(m.total, m.parts);
  const int begin = st.begin(c), before = begin - st.begin(c - 1);
  if (m.tile > before) return;                       // an earlier CTA began it
  const int row0 = blockIdx.y * 32, r = row0 + lane, rows = m.n * a.rep - m.rt * R;
  if (row0 >= rows) return;
  const int n = st.cta_of(begin - m.tile + m.tiles - 1) - c + 2;
  auto slot_of = [&](int j) -> int64_t {
    return j == 0 ? (static_cast<int64_t>(c) - 1) * 2 + (m.tile < before) : (static_cast<int64_t>(c) + j - 1) * 2;
  };
  // (rows behind the last: read, as the workspace has them, and not used)
  float top = -INFINITY;
  bool nan = false;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const float l = a.part_lse[slot_of(j) * R + r];
    nan |= l != l;
    top = fmaxf(top, l);
  }
  float total = 0.f, acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const int64_t slot = slot_of(j);
    const float l = a.part_lse[slot * R + r], w = top == -INFINITY ? 0.f : exp2f(l - top);
    const float4 *p = reinterpret_cast<const float4 *>(a.part) + (slot * (D / 4) + warp * C) * R + r;
    total += w;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const float4 v = p[k * R];
      acc[4 * k] = fmaf(w, v.x, acc[4 * k]);
      acc[4 * k + 1] = fmaf(w, v.y, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(w, v.z, acc[4 * k + 2]);
      acc[4 * k + 3] = fmaf(w, v.w, acc[4 * k + 3]);
    }
  }
  if (r >= rows) return;
  const int i = (m.rt * R + r) / a.rep, h = m.rt * R + r - i * a.rep;
  const int64_t row = m.first + i, head = m.g * a.rep + h;
  const float inv = nan ? NAN : total == 0.f ? 0.f : 1.f / total;
  uint16_t *out = static_cast<uint16_t *>(a.out) + row * a.ldot + head * a.ldoh + warp * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = inv == 0.f ? 0.f : acc[k] * inv;
  if (a.out_vec) store8<false>(out, 0, acc);
  else
#pragma unroll
    for (int k = 0; k < 8; ++k) store1<false>(out, k, acc[k]);
  if (a.lse && warp == 0)
    a.lse[row * a.n_qh + head] = nan ? NAN : total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
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

// How a call is cut: columns of a row tile, row tiles, CTAs, and what
// unfinished items need.  As many columns as a K/V group has rows, up to 64:
// a cache tile is decoded once for all of them.  (An fp32 output's weights and
// sums over an 8-bit cache of d = 128 leave shared memory for 32.)
struct Cut {
  int R, pieces;
  int64_t row_tiles, tiles, ctas, part_bytes, lse_bytes, meta_bytes;
  size_t bytes() const { return static_cast<size_t>(part_bytes + lse_bytes + meta_bytes); }
};
Cut tree_cut(const TreeArgs &a, bool fout, int sms) {
  Cut c{};
  c.pieces = fout ? 3 : 1;
  const int64_t group_rows = static_cast<int64_t>(a.max_q) * a.rep;
  // (bf16 outputs of more rows: tree_rows_kernel, 256 rows of its own kind)
  const int most = fout && a.c.d == 128 && a.c.bits == 8 ? 32 : 64;
  c.R = group_rows <= 16 ? 16 : group_rows <= 32 ? 32 : group_rows <= 64 || fout ? most : 256;
  c.row_tiles = (group_rows + c.R - 1) / c.R;
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(a.max_len) + kTile - 1) / kTile);
  const __int128 all = static_cast<__int128>(tiles) * c.row_tiles * a.c.n_kvh * a.B;
  c.tiles = all > INT32_MAX ? INT64_MAX : static_cast<int64_t>(all);
  c.ctas = std::min<int64_t>(sms, c.tiles);
  if (tiles > 1) {
    const int64_t n = c.ctas * 2 * c.R;
    c.part_bytes = n * a.c.d * 4;
    c.lse_bytes = round_up(n * 4, 256);
    c.meta_bytes = c.ctas * static_cast<int64_t>(sizeof(Meta));
  }
  return c;
}

template <int D, int M, int R, int P, bool FOUT>
mxs_status launch_tree(const TreeArgs &a, cudaStream_t s) {
  using S = Shape<D, M, R, P>;
  static_assert(S::kFits && S::kBytes <= 227 * 1024, "a CTA's shared memory");
  if (!ensure_smem(tree_kernel<D, M, R, P, FOUT>, S::kBytes)) return MXS_ERR_CUDA;
  launch_pdl(tree_kernel<D, M, R, P, FOUT>, dim3(static_cast<unsigned>(a.ctas)), dim3(S::kThreads), S::kBytes, s, a);
  count_launch();
  if (a.meta && a.ctas > 1) {
    launch_pdl(tree_combine_kernel<D, R, FOUT>, dim3(static_cast<unsigned>(a.ctas - 1), R / (8 * kJoinColumns<R>)), dim3(256), 0, s, a);
    count_launch();
  }
  return cuda_status(cudaGetLastError());
}
template <int D, int M>
mxs_status launch_rows(const TreeArgs &a, cudaStream_t s) {
  using S = RowsShape<D, M>;
  static_assert(S::kOnce <= S::kRoom && S::kBytes <= 227 * 1024, "a CTA's shared memory");
  if (!ensure_smem(tree_rows_kernel<D, M>, S::kBytes)) return MXS_ERR_CUDA;
  launch_pdl(tree_rows_kernel<D, M>, dim3(static_cast<unsigned>(a.ctas)), dim3(S::kThreads), S::kBytes, s, a);
  count_launch();
  if (a.meta && a.ctas > 1) {
    launch_pdl(tree_rows_combine_kernel<D>, dim3(static_cast<unsigned>(a.ctas - 1), 256 / 32, D / 64), dim3(256), 0, s, a);
    count_launch();
  }
  return cuda_status(cudaGetLastError());
}
template <int D, int M>
mxs_status launch_shape(const TreeArgs &a, const Cut &c, cudaStream_t s) {
  if (c.pieces == 1) {
    if (c.R == 256) return launch_rows<D, M>(a, s);
    if (c.R == 16) return launch_tree<D, M, 16, 1, false>(a, s);
    if (c.R == 32) return launch_tree<D, M, 32, 1, false>(a, s);
    return launch_tree<D, M, 64, 1, false>(a, s);
  }
  if (c.R == 16) return launch_tree<D, M, 16, 3, true>(a, s);
  if constexpr (D == 128 && M == 8) {
    return launch_tree<D, M, 32, 3, true>(a, s);
  } else {
    if (c.R == 32) return launch_tree<D, M, 32, 3, true>(a, s);
    return launch_tree<D, M, 64, 3, true>(a, s);
  }
}

}  // namespace

bool set_tree_wait(long long cycles) {
  const int v = static_cast<int>(cycles <= 0 ? kTreeWait : std::min<long long>(cycles, kTreeWait));
  return cudaMemcpyToSymbol(g_tree_wait, &v, sizeof(v)) == cudaSuccess;
}

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
  *bytes = c.bytes();
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
  if (c.tiles > INT32_MAX) return MXS_ERR_SHAPE;
  if (c.bytes() > 0 && (!ws || ws_bytes < c.bytes() || (reinterpret_cast<uintptr_t>(ws) & 255u)))
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
  a.out_vec = aligned16(out) && ldot % 8 == 0 && ldoh % 8 == 0;
  a.lse = lse;
  a.row_tiles = static_cast<int32_t>(c.row_tiles);
  a.ctas = static_cast<int32_t>(c.ctas);
  if (c.bytes() > 0) {
    a.part = static_cast<float *>(ws);
    a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + c.part_bytes);
    a.meta = reinterpret_cast<Meta *>(static_cast<uint8_t *>(ws) + c.part_bytes + c.lse_bytes);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64) return a.c.bits == 4 ? launch_shape<64, 4>(a, c, s) : launch_shape<64, 8>(a, c, s);
  return a.c.bits == 4 ? launch_shape<128, 4>(a, c, s) : launch_shape<128, 8>(a, c, s);
}
