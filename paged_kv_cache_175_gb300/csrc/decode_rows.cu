// Attention of many query rows per cached row on the fifth-generation tensor cores: a sequence's drafted tokens
// times the query heads of a group over the paged bf16 cache, or times all heads over the latent cache.
//
// Mathematics: one pass over the cached rows with a running softmax in base 2.  Everything is kept transposed,
// cached rows on the M side of the tensor core and query rows on its N side: with 16 to 64 query rows N is
// what may be small, and M = 128 (64) cached rows or channels fills the tensor core's lanes.
//   S^T[rows of the tile][R]   = K Q^T                 (both K-major, as they lie in memory)
//   O^T[channels][HL R]       += V^T [P_1 | P_2 ..]^T  (both MN-major, as they lie in shared memory)
// K and V of a latent cache are the same rows, which are loaded once: V is the first channels of the K slots.  P is
// taken as HL bf16 parts, which are columns of one product and are added in the epilogue (64 query rows over 512 latent
// channels: two products into the same columns).
//
// Work partition: the line of all (sequence, kv head, group of row tiles, tile of cached rows), in that order, is
// cut into equal pieces, one for each team of C CTAs, where a segment (all tiles of one row tile) counts as a few tiles more than
// it has, for what its end costs; the members of a team take C row tiles of the same cached rows at the same time, so
// those come from HBM once.  A CTA finds its piece from the lengths by a
// block-wide scan.  A segment that a piece boundary cuts leaves partial softmax states, which a
// second kernel joins; a piece holds at most two cut segments, its first and its last.
//
// A CTA of 12 warps runs these roles, joined by mbarriers with bounded waits:
//   warps 0, 3  producers: keys and query rows, and values (latent cache: a half of a tile's chunks each), by TMA
//   warp 1      owner of the tensor memory; issues the first product into one of the S buffers
//   warp 2      issues the second product
//   warps 4-11  softmax and epilogue, in two groups of four warps.  K and V pools: the groups take alternate tiles, each
//               with an O accumulator of its own; latent cache: both take every tile, half of the query rows each
//
// What bounds it (GPU time; R query rows per CTA):
//   64 trees of up to 16 tokens over 0.5-4K rows, 8 kv heads of 4 x 128 (620 MB): 110 us, 5.6 TB/s: HBM, then the segments' ends.  The
//     same of up to 8 tokens: 101 us.
//   8 trees of up to 64 over 8-32K, 8 x 8 heads (512 rows, 207 GFLOP): 390 us, 530 TFLOP/s: shared memory and HBM.  A tile of 128
//     rows takes 96 KB written to shared memory (P among them) and 112 read by its products, 1625 clocks at 128 bytes each, of the 2200 that
//     there are for each tile of a CTA; HBM is 70% busy, since the caches are read 3.2 times over.  (128 query rows per CTA, with one
//     part of p, took 489 us where 64 took 398: they leave two S buffers and three key stages.)
//   64 x 0.5-4K latent tokens of 16 heads (173 MB): 41 us, 4.2 TB/s: HBM for 28 of them, then setup, first loads and the join.
//   32 x 2-16K latent tokens of 128 heads (82 GFLOP): 144 us, 567 TFLOP/s: shared memory for three quarters of it, 88 KB written and
//     341 read per tile of 64 rows, 3430 of the 4640 clocks that there are for each tile of a CTA.  What the others go to was not measured; the
//     products, the softmax and the copies of a tile wait on one another.
//   300 trees of up to 4 over 1-300 rows (2400 segments): 77 us: the ends of 16 segments per CTA, about 8000 clocks each: masks, softmax,
//     second product and epilogue, in series.
//   One tree of 8 over 333 rows: 10.8 us; one latent token of 16 heads over 301: 11.7: setup 1.5 us, loads 2, masks and softmax 2,
//     epilogue 1, the join 2, and code that is run once and cold.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "drafts.cuh"
#include "nvtx_range.h"
#include "umma.cuh"

namespace pkv {

// A segment that a piece boundary cuts for the first time, for the kernel that joins the parts.
struct RowsCut {
  int parts, first;              // pieces (0: nothing to join); partial of the first piece (0 or 1)
  int q0, n, g, rg, pad0, pad1;
};

struct RowsArgs {
  const int32_t *bt, *ctx, *q_start;
  const int64_t* mask;
  int max_blocks, max_ctx, mask_words, n_tok, batch, n_h, n_kv, G, num_blocks, n_each, bs_log2;
  // A row tile: latent cache: R of a sequence's tokens times heads, wherever that cuts a token.  K and V pools: tpt
  // tokens of gt heads, or where a group has more than R heads one token's heads in hc parts.
  int gt, tpt, hc;
  int last_steps;                // 16-channel steps of a latent cache's position chunk
  int C, P;                      // members of a team, teams
  float scale_log2;
  void* out;
  int out_f32;
  int32_t* err;
  RowsCut* cuts;                 // [P]
  float *ws_ml, *ws_o;           // [P * C][2][R][2] and [P * C][2][R][DV]
};

// Where a CTA stands on the line.
struct RowsCursor {
  Drafts d;
  int s, g, rg, t, nt, rt;       // sequence, kv head, group of row tiles, tile; tiles of a segment, row tiles
  int at_start;                  // still in the segment that the piece starts in
  int whole_from;                // the segment began in this piece
  long long left;                // the piece's share of the line from here on (this tile included)
};

// KC: 64-channel chunks of a key; VT: M tiles of VM channels of a value; R: query rows; HL: bf16 parts of p.
// PP: the two softmax groups take alternate tiles, each with an O accumulator of its own; else both take every tile,
// half of the query rows each (a latent cache's O leaves no room in tensor memory for a second one).
template <int KC_, int VT_, int VM_, bool SHARED_, int R_, int HL_>
struct RowsCfg {
  static constexpr int KC = KC_, VT = VT_, VM = VM_, R = R_, HL = HL_;
  static constexpr bool SHARED = SHARED_, PP = !SHARED;
  static constexpr int TT = SHARED ? 64 : 128;                // cached rows of a tile
  static constexpr int MT = TT / 64;
  // What a segment's end (its masked tile, its epilogue, the next queries) weighs on the line, in tiles: with 0 a CTA of many short
  // segments ended last.  When it was chosen: 64 trees of 16 126 us with 0, 113 with 2, 108 with 4, 109 with 6; 128 x 16-1K latent
  // tokens of 16 heads 29.6 with 0, 26.7 with 1, 28.4 with 3, and of 128 heads 56.3, 51.3, 50.1.
  static constexpr int END = PP ? (R == 64 ? 4 : 3) : (R == 64 ? 2 : 1);
  static constexpr int DV = VT * VM, VC = DV / 64;
  static constexpr int CHUNK = TT * 128;
  // Bytes from 8 rows of a slot to the next 8: a copy brings a block's rows of all of a slot's chunks, 1024 bytes of each
  // chunk for every 8 rows.
  static constexpr int GS = SHARED ? 2048 : KC * 1024;
  // 64 query rows of 512 latent channels: 72 KB of queries, and an O that leaves tensor memory for one part of p.  The second
  // part is then a product of its own into the same columns, from one buffer for all tiles.
  static constexpr bool FULL = SHARED && KC == 9 && R == 64;
  static constexpr int HO = FULL ? 1 : HL;                    // parts of p that are columns of one product
  static constexpr int N2 = R * HO;                           // columns of the second product
  static constexpr int QCH = R * 128, QBUF = KC * QCH;
  static constexpr int PAT = (N2 + 63) / 64, PBUF = PAT * CHUNK;
  // Rings, from what 227 KB hold.  K and V pools: NK stages of a tile's keys and NV of its values, which are held for less of
  // a tile's way: with 64 query rows of 128 channels, where that way and not the memory sets the pace, 4 and 2, and one buffer of
  // query rows (8 x 8-32K tokens, 512 rows: 388 us, and 452 with 3 and 2 and two such buffers).  Latent cache: NK slots of two
  // chunks, which the second product frees one after another, and NP slots of the position chunk.  The tile's P takes
  // the place of its keys (of their position chunk), which the first product is the only one to read.
  static constexpr int KPART = KC * CHUNK > PBUF + 3072 ? KC * CHUNK : PBUF + 3072;   // P and the scratch behind it
  static constexpr int KST = SHARED ? 2 * CHUNK : KPART, VST = VC * CHUNK;
  static constexpr int PST = SHARED ? PBUF : KST;
  static constexpr int NQ = (SHARED && (KC == 9 ? R > 16 : R == 64)) || (KC == 2 && R == 64) ? 1 : 2;
  static constexpr int NK = SHARED ? (FULL || PAT > 1 ? 8 : 9) : (KC == 1 || R == 64 ? 4 : 3), NV = SHARED ? 1 : (KC == 1 ? 4 : (R == 64 ? 2 : 3));
  static constexpr int NP = SHARED ? (FULL ? 2 : 3) : NK;     // tiles whose P there is room for
  static constexpr int NM = SHARED ? (KC == 9 ? 3 : 8) : NK;  // metadata of tiles: of all that the ring may hold a part of
  static constexpr int NS = PP ? 4 : 2, NG = PP ? 2 : 1;      // S buffers; accumulators of a segment
  static constexpr int NO = VT * N2 * NG * 2 + NS * R <= 512 && !(PP && R == 64) ? 2 : 1;
  static constexpr int S_COL = VT * N2 * NG * NO, NCOL = S_COL + NS * R;
  static constexpr uint32_t TMEM_COLS = NCOL <= 64 ? 64 : (NCOL <= 128 ? 128 : (NCOL <= 256 ? 256 : 512));
  static constexpr int P_OFF = SHARED ? NK * KST : 0, V_OFF = NK * KST, L_OFF = P_OFF + NP * PST,
                       Q_OFF = NK * KST + (SHARED ? NP * PST + (FULL ? PBUF : 0) : NV * VST), W_OFF = Q_OFF + NQ * QBUF, M_OFF = W_OFF + (SHARED ? 28 * R + 16 : 0);   // W: scratch
  static constexpr bool F32 = HL == 3;                        // output type
};

struct RowsMeta {
  int flags, k;                  // F_ and G_ flags; number of the segment in the piece
  int tile0, ctx, n, q0;         // first cached row of the tile; the sequence
  int t0, h0, g;                 // first token of the row tile and its first head of the group; kv head
  int invalid, part;             // blocks of the tile with a bad id; partial state of a cut segment
  int rows;                      // query rows of the row tile: the first ones
};
// Exponents (base 2) up to this are taken against an offset as it is: p is held in bf16 and fp32, whose range is 2^127, and
// is as exact at 2^32 as at 1; what an offset this far below the maximum takes from the other end, 2^-94, is nothing.
constexpr float kRowsLazy = 32.f;
// The lowest offset, of a query row that has seen no score above it: a number, so that what is subtracted is what a state says,
// and a row whose scores so far were minus infinities (weight 0) goes on from there.  Any other score against it is raised.
constexpr float kRowsLowest = -3.402823466e38f;
// An exponent is a score times the scale less the offset in one operation, where the offset is such a product rounded: half a step
// of it stays, which is below 1 up to this size.  A segment with a larger offset rounds its other products likewise.
constexpr float kRowsFar = 16777216.f;
// For a softmax group: its first and its last tile of the segment; a segment of one tile.  (F_END: no tile, but the end.)
enum : int { G_FIRST = 64, G_LAST = 128, G_SOLO = 256 };

template <class X>
struct RowsShared {
  // What has landed, by stage (latent cache: either half of a tile's chunks, by its metadata); slots of keys, or stages; values; P, by its slot;
  // slots of position chunks; the products of P by the tile's parity
  uint64_t kfull[X::SHARED ? 2 * X::NM : X::NK], kempty[X::NK], vfull[X::NV], vempty[X::NV], pfull[X::NP], pslot[X::SHARED ? X::NP : 1], pempty[2],
      qfull[X::NQ], qempty[X::NQ], sfull[X::NS], sempty[X::NS], ofull[X::NG], oempty[X::NO], joined[X::NG], drain;
  RowsMeta meta[X::NM];          // of tile i: entry i % NM
  uint32_t tmem;
  int any;
  volatile int abort_flag;
  volatile int bad[X::NG][2];                                     // of each group of waiting warps, by the parity of its barriers
  RowsCut first;                 // the piece's first segment; parts: tiles ahead of the piece, first: of the segment
  long long W;
  float offset[X::NG][X::R];     // of each query row: what its exponents are taken against
  // Of a segment's end, by its O buffer: offset and sum of each query row in a group's tiles, factors of the output (of
  // either accumulator), and output rows
  float2 sum[X::PP ? X::NO : 1][X::NG][X::PP ? X::R : 1];
  union {
    std::conditional_t<X::PP, float2, float> factor[X::NO][X::R];
    RowsCursor cur;                // of the setup: the member's first tile (both producers have read it before any product)
  };
  union {
    int row[X::NO][X::R];
    long long scan[12];            // of the setup
  };
};
// What the warps of a tile share for a moment: behind its P, or in a place of its own.
template <class X>
struct RowsScratch {
  float red[4][X::R];                                         // each warp's part of a query row's maximum or sum
  float factor[X::R];                                         // of a rescale
  unsigned long long win[X::MT][X::R], seen[X::MT][2];        // cached rows attended to, by each query row and by any of a warp's
};

static __device__ __noinline__ long long div_far(long long x, long long y) { return x / y; }
// Quotient of numbers that are hardly ever beyond 32 bits, where a division takes a third of the time.
__device__ __forceinline__ long long div_pos(long long x, long long y) {
  return (x | y) >> 32 ? div_far(x, y) : (long long)((unsigned)x / (unsigned)y);
}
// Piece p of a line of W tiles in P pieces starts here: the first W % P pieces are one tile longer.
struct RowsLine {
  long long W, each, longer;
  int P;
  __device__ __forceinline__ RowsLine(long long w, int most) : W(w), P((int)(w < most ? w : most)) {
    each = P ? div_pos(W, P) : 0;
    longer = W - each * P;
  }
  __device__ __forceinline__ long long start(int p) const { return p * each + (p < longer ? p : longer); }
  __device__ __forceinline__ int piece(long long pos) const {
    const long long head = longer * (each + 1);
    return (int)(pos < head ? div_pos(pos, each + 1) : longer + div_pos(pos - head, each));
  }
};
template <class X>
__device__ __forceinline__ int row_tiles(const RowsArgs& a, int n) {
  return X::SHARED ? (int)(((long long)n * a.G + X::R - 1) / X::R) : (n + a.tpt - 1) / a.tpt * a.hc;
}
template <class X>
__device__ __forceinline__ long long line_length(const RowsArgs& a, const Drafts& d) {
  constexpr int tt = X::TT;
  const int rt = row_tiles<X>(a, d.n);
  return d.ctx > 0 ? (long long)a.n_kv * ((rt + a.C - 1) / a.C) * ((d.ctx + tt - 1) / tt + X::END) : 0;
}

// Behind a segment's last tile, or where the member has no row tile: the next segment in which it has one (left is 0: the
// piece has none).  By value, so that a cursor stays in registers between segments.
template <class X>
__device__ __noinline__ RowsCursor next_segment(RowsCursor c, const RowsArgs& a, int member) {
  while (c.left > 0) {
    if (c.t >= c.nt) {
      c.t = 0;
      c.at_start = 0;
      c.whole_from = 1;
      c.left -= X::END;
      if (c.left <= 0) break;
      if (++c.rg * a.C >= c.rt) {
        c.rg = 0;
        if (++c.g >= a.n_kv) {
          c.g = 0;
          int flags = 0;
          do {
            if (++c.s >= a.batch) {
              c.left = 0;
              return c;
            }
            c.d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, c.s, flags);
            c.nt = (c.d.ctx + X::TT - 1) / X::TT;
            c.rt = row_tiles<X>(a, c.d.n);
          } while (c.nt == 0 || c.rt == 0);
        }
      }
    }
    if (c.rg * a.C + member < c.rt) return c;
    c.left -= c.nt - c.t;
    c.t = c.nt;
  }
  c.left = 0;
  return c;
}
__device__ __forceinline__ float sum_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }   // a sum that is no number stays one

// Token (of its sequence, -1: none) and head of the group of query row c of a row tile; `in` is row_in(a, c).
template <class X>
__device__ __forceinline__ int2 row_in(const RowsArgs& a, int c) {
  if constexpr (X::SHARED) return make_int2(0, c);
  return make_int2(c < a.gt * a.tpt ? c / a.gt : 1 << 30, c % a.gt);
}
template <class X>
__device__ __forceinline__ int2 query_of(const RowsArgs& a, int n, int t0, int h0, int2 in) {
  int h = h0 + in.y;                                          // a latent cache's tile may begin inside a token
  long long t = (long long)t0 + in.x;
  if constexpr (X::SHARED) {
    t += h / a.G;
    h %= a.G;
  }
  return make_int2(t < n && h < a.G ? (int)t : -1, h);
}
template <class X>
__device__ __forceinline__ void tile_of(const RowsArgs& a, int rt, int& t0, int& h0) {
  if constexpr (X::SHARED) {
    const long long r = (long long)rt * X::R;
    t0 = (int)(r / a.G);
    h0 = (int)(r - (long long)t0 * a.G);
  } else {
    t0 = rt / a.hc * a.tpt;
    h0 = rt % a.hc * a.gt;
  }
}
__device__ __forceinline__ void store_out(const RowsArgs& a, long long at, float v) {
  if (a.out_f32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ unsigned long long ones_below(int b) { return b <= 0 ? 0ull : (b >= 64 ? ~0ull : (1ull << b) - 1); }

// Which of the 64 cached rows from `first` on, in the tile `mt`, token i of its sequence attends to.
static __device__ __noinline__ unsigned long long attended(const RowsArgs& a, const RowsMeta& mt, int i, int first) {
  const int o = mt.ctx - mt.n - first;                        // the first drafted token's row, from `first`
  unsigned long long w;
  if (!a.mask) {
    w = ones_below(o + i + 1);
  } else {
    w = ones_below(o);
    const int64_t* m = a.mask + (size_t)(mt.q0 + i) * a.mask_words;
    if (o < 64 && o >= 0) w |= (unsigned long long)m[0] << o;
    if (o < 0) {
      const int q = -o >> 6, r = -o & 63;
      if (q < a.mask_words) w |= (unsigned long long)m[q] >> r;
      if (r && q + 1 < a.mask_words) w |= (unsigned long long)m[q + 1] << (64 - r);
    }
  }
  w &= ones_below(mt.ctx - first);
  // rows of blocks with a bad id
  unsigned bad = (unsigned)mt.invalid >> ((first - mt.tile0) >> a.bs_log2);
  for (int b = 0; bad && b < 64 >> a.bs_log2; ++b, bad >>= 1)
    if (bad & 1) w &= ~(ones_below(1 << a.bs_log2) << (b << a.bs_log2));
  return w;
}

// A wait whose polling is out of line: the roles' loops have to fit the instruction cache together.  It gives up after its
// limit, or when another role has (`stop`).
static __device__ __noinline__ bool rows_poll(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* stop) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (stop && *stop) return false;
    if ((it & 255u) == 0 && global_timer_ns() - t0 > limit_ns) return false;
  }
  return false;
}
// Of a whole warp, whose lanes leave it together: what follows (elect.sync, tensor memory) wants a converged warp.
__device__ __forceinline__ bool rows_wait(uint64_t* bar, int round, const volatile int* stop) {
  const bool done = mbar_try_wait(bar, round & 1) || rows_poll(bar, round & 1, 2000000000ull, stop);
  const bool all = __all_sync(FULL_MASK, done);
  __syncwarp();
  return all;
}
// The lane that issues copies and products, of a converged warp.  What it runs is a straight line, and loops are the whole
// warp's: a rolled loop around tcgen05.mma and its commits in one lane alone ended in an illegal instruction.
__device__ __forceinline__ bool elected() {
  __syncwarp();
  return elect_one();
}

template <class X>
__global__ void __launch_bounds__(384, 1)
    decode_rows_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ CUtensorMap tmq, const __grid_constant__ RowsArgs a) {
  constexpr int TT = X::TT, R = X::R, HL = X::HL, HO = X::HO, N2 = X::N2, KC = X::KC, VT = X::VT, MT = X::MT, DV = X::DV;
  constexpr int NK = X::NK, NV = X::NV, NM = X::NM, NP = X::NP, NO = X::NO, NS = X::NS, NG = X::NG, NQ = X::NQ;
  constexpr int NF = X::SHARED ? NM : NK;                     // full barriers
  constexpr bool PP = X::PP;
  extern __shared__ __align__(1024) uint8_t sm[];
  RowsShared<X>& sh = *reinterpret_cast<RowsShared<X>*>(sm + X::M_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / a.C, member = blockIdx.x % a.C;
  if (smem_u32(sm) & 1023u) {              // the descriptors and the swizzle count on it, and there is no room to align it here
    if (threadIdx.x == 0) set_err(a.err, PKV_DEV_TIMEOUT);
    return;
  }

  if (warp == 1) tmem_alloc(&sh.tmem, X::TMEM_COLS);
  if (warp == 2) {
    constexpr int SW = PP ? 4 : 8;         // softmax warps of a tile
    for (uint64_t* b = sh.kfull + lane; b <= &sh.drain; b += 32) {
      int count = 1;
      if (X::SHARED && b < sh.kempty) count = ((smem_u32(b) - smem_u32(sh.kfull)) & 8u) ? VT / 2 + 1 : VT / 2;
      if ((b >= sh.sempty && b < sh.sempty + NS) || (b >= sh.pfull && b < sh.pfull + NP)) count = SW;
      if (b >= sh.oempty && b < sh.oempty + NO) count = 8;
      if (PP && b >= sh.joined && b < sh.joined + NG) count = 4;
      if (b == &sh.drain) count = 2;
      mbar_init(b, count);
    }
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.any = 0;
    sh.W = 0;
    for (int j = 0; j < 2 * NG; ++j) sh.bad[j >> 1][j & 1] = 0;
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    prefetch_tensormap(&tmq);
  }
  // query rows past a tile's own hold zeros until the end
  if constexpr (!X::SHARED)
    for (int i = threadIdx.x; i < NQ * X::QBUF / 16; i += 384) reinterpret_cast<uint4*>(sm + X::Q_OFF)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  grid_dep_wait();
  grid_dep_launch();

  // ------------------------------- the piece -------------------------------
  // Thread i sums the line over sequences [i per, (i + 1) per); a scan over the CTA gives every thread where its
  // sequences begin and the line's length, and the thread whose sequences hold the piece's start walks them.
  {
    const int per = (a.batch + 383) / 384, s0 = threadIdx.x * per, s1 = min(s0 + per, a.batch);
    long long mine = 0;
    int flags = 0;
    Drafts d = {};
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, s, flags);
      mine += line_length<X>(a, d);
    }
    if (flags && blockIdx.x == 0) set_err(a.err, flags);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(FULL_MASK, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    long long before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      const long long y = sh.scan[w];
      if (w < warp) before += y;
      W += y;
    }
    before += incl - mine;
    const RowsLine line(W, a.P);
    const long long pstart = line.start(team);
    if (team < line.P && pstart >= before && pstart < before + mine) {
      RowsCursor c;
      long long off = pstart - before;
      c.s = s0;
      c.d = d;                             // with a sequence per thread it is the one
      if (per > 1)
#pragma unroll 1
        for (;; ++c.s) {
          c.d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, c.s, flags);
          const long long len = line_length<X>(a, c.d);
          if (off < len || c.s + 1 >= s1) break;
          off -= len;
        }
      c.nt = max(1, (c.d.ctx + TT - 1) / TT);
      c.rt = row_tiles<X>(a, c.d.n);
      const int groups = max(1, (c.rt + a.C - 1) / a.C);
      const long long seg_at = div_pos(off, c.nt + X::END);   // segment of the sequence
      const int x = (int)(off - seg_at * (c.nt + X::END));    // where in it: behind its tiles, the piece begins with the next one
      c.t = min(x, c.nt);
      c.g = (int)div_pos(seg_at, groups);
      c.rg = (int)(seg_at - (long long)c.g * groups);
      c.at_start = 1;
      c.whole_from = x == 0;
      c.left = line.start(team + 1) - pstart + (x - c.t);
      sh.first = RowsCut{x < c.nt ? x : 0, c.nt, c.d.q0, c.d.n, c.g, c.rg, 0, 0};
      sh.W = W;
      if (c.t >= c.nt || c.rg * a.C + member >= c.rt) c = next_segment<X>(c, a, member);
      sh.cur = c;
      if (c.left > 0) {
        prefetch_l2(a.bt + (size_t)c.s * a.max_blocks + ((c.t * TT) >> a.bs_log2));
        sh.any = 1;
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (sh.any && (warp == 0 || warp == 3)) {
    // ------------------------------- producers -------------------------------
    // Both walk the piece.  Warp 0 loads the queries, the tile's metadata and its keys, or the first half of a latent
    // cache's chunks; warp 3 the values, or the other half and the position chunk.  The whole warp runs the loop
    // and one lane (elect_one) issues the copies in unrolled runs: about 30 clocks each, where a lane per copy
    // or a loop around one takes 60 to 90, which bounded the kernel with blocks of 16.
    const bool lead = warp == 0;
    const int bsz = 1 << a.bs_log2, nbt = TT >> a.bs_log2;    // rows of a block, blocks of a tile
    const uint64_t pol = policy_evict_first();
    RowsCursor c = sh.cur;
    int k = 0, kq = -1, i = 0;
    bool ok = true;
    auto ids_at = [&](int s, int ctx, int from) {             // block ids, one per lane
      return from + lane < (ctx + bsz - 1) >> a.bs_log2 ? a.bt[(size_t)s * a.max_blocks + from + lane] : -1;
    };
    int win_first = ids_at(c.s, c.d.ctx, c.t * nbt);          // the first 32 of the segment that comes next
#pragma unroll 1
    for (;; ++k) {
      // A segment: `count` tiles of it from c.t on.  Lane l keeps word l of its metadata (RowsMeta), of which a tile changes few.
      const int count = c.left < c.nt - c.t ? (int)c.left : c.nt - c.t, all_blocks = (c.d.ctx + bsz - 1) >> a.bs_log2;
      const int whole = c.whole_from && c.t + count == c.nt ? F_WHOLE : 0;
      int t0, h0;
      tile_of<X>(a, c.rg * a.C + member, t0, h0);
      int word = 0;
      if (lane == 1) word = k;
      if (lane == 3) word = c.d.ctx;
      if (lane == 4) word = c.d.n;
      if (lane == 5) word = c.d.q0;
      if (lane == 6) word = t0;
      if (lane == 7) word = h0;
      if (lane == 8) word = c.g;
      if (lane == 10) word = blockIdx.x * 2 + (c.at_start ? 0 : 1);
      if (lane == 11) word = X::SHARED ? (c.d.n - t0) * a.G - h0 : (a.hc > 1 ? a.G - h0 : min(a.tpt, c.d.n - t0) * a.gt);
      int blk0 = c.t * nbt, wfrom = blk0, win = win_first, win_next = ids_at(c.s, c.d.ctx, blk0 + 32);
      // The segment's query rows.  With one buffer for them they come behind the first tile, which need not wait for the
      // last segment's products.
      auto queries = [&] {
        const int qb = k % NQ;
        ok = k < NQ || rows_wait(&sh.qempty[qb], k / NQ - 1, &sh.abort_flag);
        if (!ok) return;
        if (elected()) mbar_arrive_expect_tx(&sh.qfull[qb], (uint32_t)KC * 128u * (uint32_t)(X::SHARED ? R : a.gt * a.tpt));
#pragma unroll 1
        for (int ch = 0; ch < KC; ++ch)
          if (elected())
            tma_load_3d(sm + X::Q_OFF + qb * X::QBUF + ch * X::QCH, &tmq, ch * 64, X::SHARED ? (c.d.q0 + t0) * a.n_h + h0 : c.g * a.G + h0,
                        X::SHARED ? 0 : c.d.q0 + t0, &sh.qfull[qb], pol);
        kq = k;
        __syncwarp();
      };
      if (NQ > 1 && lead) queries();
      RowsCursor next = c;
#pragma unroll 1
      for (int j = 0; j < count && ok; ++j, ++i, blk0 += nbt) {
        if (blk0 >= wfrom + 32) {
          win = win_next;
          wfrom += 32;
          win_next = ids_at(c.s, c.d.ctx, wfrom + 32);
        }
        const int phys = __shfl_sync(FULL_MASK, win, (blk0 - wfrom + lane) & 31);
        const unsigned used = (1u << min(all_blocks - blk0, nbt)) - 1;
        const unsigned valid = __ballot_sync(FULL_MASK, (unsigned)phys < (unsigned)a.num_blocks) & used;
        const uint32_t rows_bytes = (uint32_t)__popc(valid) << a.bs_log2;   // rows that are copied
        constexpr int MB = TT / 16;
        int ids[MB];
#pragma unroll
        for (int b = 0; b < MB; ++b) ids[b] = __shfl_sync(FULL_MASK, phys, b);
        if (lead) {
          const bool last = j + 1 == count, next_last = PP && j + 2 == count;
          const int flags = (j == 0 ? F_FIRST : 0) | (last ? F_LAST : 0) | whole | (j < (PP ? 2 : 1) ? G_FIRST : 0) |
                            (last || next_last ? G_LAST : 0) | (count == 1 ? G_SOLO : 0);
          if (lane == 0) word = flags;
          if (lane == 2) word = blk0 << a.bs_log2;
          if (lane == 9) word = (int)(used & ~valid);
          if (lane == 9 && word) set_err(a.err, PKV_DEV_BAD_BLOCK);
        }
        // One fill of a slot: all of its chunks of each block, from chunk c0 on.  (The copies' bytes are counted behind them: the
        // phase waits for this arrival.)
        const int step = X::GS / 8 << a.bs_log2, group = c.g << (a.bs_log2 - 3);
        auto fill = [&](uint8_t* dst, uint64_t* full, const CUtensorMap* tm, int c0, bool tells) {
          auto box = [&](int b) {
            if ((valid >> b) & 1) tma_load_5d(dst + b * step, tm, 0, 0, c0, group, ids[b], full, pol);
          };
          if (elected()) {
            box(0);
            if (MB == 8 || nbt > 1) {
              box(1);
              if (nbt > 2) {
                box(2);
                box(3);
                if (MB == 8 && nbt > 4) {
#pragma unroll
                  for (int b = 4; b < MB; ++b) box(b);
                }
              }
            }
          }
          if (tells && lane < (int)(sizeof(RowsMeta) / 4)) reinterpret_cast<int*>(&sh.meta[i % NM])[lane] = word;
          if (elected()) mbar_arrive_expect_tx(full, rows_bytes * (X::GS / 8));
          __syncwarp();
        };
        if constexpr (X::SHARED) {
          uint64_t* full = &sh.kfull[2 * (i % NM) + (lead ? 0 : 1)];
#pragma unroll 1
          for (int v = 0; v < VT / 2 && ok; ++v) {
            const int vt = lead ? v : VT / 2 + v, use = i * VT + vt, slot = use % NK;
            ok = use < NK || rows_wait(&sh.kempty[slot], use / NK - 1, &sh.abort_flag);
            if (!ok) break;
            fill(sm + slot * X::KST, full, &tmk, 2 * vt, lead && v == 0);
          }
          if (ok && !lead) {
            ok = i < NP || rows_wait(&sh.pslot[i % NP], i / NP - 1, &sh.abort_flag);
            if (ok) {                      // the position chunk (tmv: its rows may be narrower than a chunk)
              uint8_t* dst = sm + X::P_OFF + (i % NP) * X::PST;
              auto box = [&](int b) {
                if ((valid >> b) & 1) tma_load_3d(dst + (b * 128 << a.bs_log2), &tmv, VT * 128, group * 8, ids[b], full, pol);
              };
              if (elected()) {
                box(0);
                if (nbt > 1) {
                  box(1);
                  if (nbt > 2) {
                    box(2);
                    box(3);
                  }
                }
                mbar_arrive_expect_tx(full, rows_bytes * 128);
              }
              __syncwarp();
            }
          }
        } else {
          const int depth = lead ? NK : NV, st = i % depth;
          ok = i < depth || rows_wait(lead ? &sh.kempty[st] : &sh.vempty[st], i / depth - 1, &sh.abort_flag);
          if (ok)
            fill(sm + (lead ? st * X::KST : X::V_OFF + st * X::VST), lead ? &sh.kfull[st] : &sh.vfull[st], lead ? &tmk : &tmv, 0, lead);
        }
        if (NQ == 1 && lead && j == 0 && ok) queries();
        if (j + 1 == count) {              // on to the next segment, with its block ids on the way meanwhile
          next.t += count;
          next.left -= count;
          if (next.left > 0) next = next_segment<X>(next, a, member);
          if (next.left > 0) win_first = ids_at(next.s, next.d.ctx, next.t * nbt);
        }
      }
      c = next;
      if (!ok || c.left <= 0) break;
    }
    // Behind the last tile, an end for each softmax group.
    if (ok && lead) {
#pragma unroll 1
      for (int z = 0; z < NG && ok; ++z, ++i) {
        const int use = X::SHARED ? i * VT : i, slot = use % NK;
        ok = use < NK || rows_wait(&sh.kempty[slot], use / NK - 1, &sh.abort_flag);
        if (!ok) break;
        if (lane == 0) {
          sh.meta[i % NM].flags = F_END;
          mbar_arrive_n(&sh.kfull[X::SHARED ? 2 * (i % NM) : slot], X::SHARED ? VT / 2 : 1);
        }
        __syncwarp();
      }
    }
    ok = __all_sync(FULL_MASK, ok);
    if (!ok && lane == 0) {
      set_err(a.err, PKV_DEV_TIMEOUT);
      sh.abort_flag = 1;
    }
    // After a timeout: let the loads already issued land before the CTA leaves (bounded).
    if (sh.abort_flag && lane == 0) {
      bool live = true;
      for (int j = max(0, i - NF); j <= i && live; ++j) live = rows_poll(&sh.kfull[X::SHARED ? 2 * (j % NF) : j % NF], (j / NF) & 1, 20000000ull, nullptr);
      live = true;
      constexpr int ND = X::SHARED ? NM : NV;
      for (int j = max(0, i - ND); j <= i && live; ++j)
        live = rows_poll(X::SHARED ? &sh.kfull[2 * (j % NF) + 1] : &sh.vfull[j % NV], (j / ND) & 1, 20000000ull, nullptr);
      if (kq >= 0) rows_poll(&sh.qfull[kq % NQ], (kq / NQ) & 1, 20000000ull, nullptr);
    }
    __syncwarp();
  } else if (sh.any && warp == 1) {
    // ------------------------- first-product issuer -------------------------
    constexpr uint32_t IQK = umma_idesc_bf16(TT, R, 0, 0);
    constexpr uint32_t HI = (uint32_t)(umma_desc_k(16, 1024) >> 32), HIK = (uint32_t)(umma_desc_k(16, X::GS) >> 32);
    const uint32_t sbase = (uint32_t)umma_desc_k(16, 1024) + (smem_u32(sm) >> 4);
    const uint32_t tm = __shfl_sync(FULL_MASK, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int k0 = X::SHARED ? i * VT : i, sb = i % NS;     // first slot of the tile's keys
      ok = rows_wait(&sh.kfull[X::SHARED ? 2 * (i % NF) : i % NF], i / NF, &sh.abort_flag);
      if (!ok) break;
      const RowsMeta& mt = sh.meta[i % NM];
      const int flags = __shfl_sync(FULL_MASK, mt.flags, 0), k = __shfl_sync(FULL_MASK, mt.k, 0), qb = k % NQ;
      if (flags & F_END) break;
      ok = (!(flags & F_FIRST) || rows_wait(&sh.qfull[qb], k / NQ, &sh.abort_flag)) && (i < NS || rows_wait(&sh.sempty[sb], i / NS - 1, &sh.abort_flag));
      if (!ok) break;
      const uint32_t qa = sbase + ((X::Q_OFF + qb * X::QBUF) >> 4), d = tm + X::S_COL + R * sb;
      tc_fence_after();
      // Chunks [ch0, ch0 + NC) of the keys, at ka, four steps of 16 channels each.  Loops are the warp's; what the elected
      // lane runs is a straight line.
      auto chunks = [&](uint32_t ka, int ch0, int steps, auto chunks_of) {
        constexpr int NC = decltype(chunks_of)::value;
        const uint32_t qc = qa + ch0 * (X::QCH >> 4), first = ch0 == 0 ? 0u : 1u;
        if (elected()) {
#pragma unroll
          for (int ch = 0; ch < NC; ++ch)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              if (ks < steps)
                umma_bf16_lo(d, ka + ch * (1024 >> 4) + ks * 2, X::SHARED && NC == 1 ? HI : HIK, qc + ch * (X::QCH >> 4) + ks * 2, HI, IQK, ch + ks ? 1u : first);
        }
        __syncwarp();
      };
      if constexpr (X::SHARED) {
        // the halves of its chunks as they land
#pragma unroll 1
        for (int u = 0; u < VT / 2; ++u) chunks(sbase + ((k0 + u) % NK * X::KST >> 4), 2 * u, 4, std::integral_constant<int, 2>());
        ok = rows_wait(&sh.kfull[2 * (i % NF) + 1], i / NF, &sh.abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = VT / 2; u < VT; ++u) chunks(sbase + ((k0 + u) % NK * X::KST >> 4), 2 * u, 4, std::integral_constant<int, 2>());
        chunks(sbase + ((X::P_OFF + (i % NP) * X::PST) >> 4), KC - 1, a.last_steps, std::integral_constant<int, 1>());
      } else {
        chunks(sbase + ((i % NK) * X::KST >> 4), 0, 4, std::integral_constant<int, KC>());
      }
      if (elected()) {
        umma_commit(&sh.sfull[sb]);
        if (flags & F_LAST) umma_commit(&sh.qempty[qb]);
      }
      __syncwarp();
    }
    ok = __all_sync(FULL_MASK, ok);
    if (elected()) {
      if (!ok) {
        set_err(a.err, PKV_DEV_TIMEOUT);
        sh.abort_flag = 1;
      }
      // every product issued has completed before the tensor memory is released
      umma_commit(&sh.drain);
    }
    rows_wait(&sh.drain, 0, nullptr);
  } else if (sh.any && warp == 2) {
    // ------------------------- second-product issuer ------------------------
    constexpr uint32_t IPV = umma_idesc_bf16(X::VM, N2, 1, 1);
    constexpr uint32_t HI = (uint32_t)(umma_desc_k(X::CHUNK, 1024) >> 32), HIV = (uint32_t)(umma_desc_k(1024, X::GS) >> 32);
    const uint32_t sbase = (uint32_t)umma_desc_k(X::CHUNK, 1024) + (smem_u32(sm) >> 4);
    const uint32_t vbase = (uint32_t)umma_desc_k(1024, X::GS) + (smem_u32(sm) >> 4);
    const uint32_t tm = __shfl_sync(FULL_MASK, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int pb = i % NP, k0 = i * VT;
      ok = rows_wait(&sh.kfull[X::SHARED ? 2 * (i % NF) : i % NF], i / NF, &sh.abort_flag);
      if (!ok) break;
      const RowsMeta& mt = sh.meta[i % NM];
      const int flags = __shfl_sync(FULL_MASK, mt.flags, 0), k = __shfl_sync(FULL_MASK, mt.k, 0), ob = k % NO;
      if (flags & F_END) break;
      ok = rows_wait(X::SHARED ? &sh.kfull[2 * (i % NF) + 1] : &sh.vfull[i % NV], X::SHARED ? i / NF : i / NV, &sh.abort_flag) && rows_wait(&sh.pfull[pb], i / NP, &sh.abort_flag);
      if (!ok) break;
      const int nks = __shfl_sync(FULL_MASK, (min(TT, mt.ctx - mt.tile0) + 15) >> 4, 0);
      ok = !(flags & F_FIRST) || k < NO || rows_wait(&sh.oempty[ob], k / NO - 1, &sh.abort_flag);
      if (!ok) break;
      tc_fence_after();
      __syncwarp();
      const uint32_t pa = sbase + ((X::P_OFF + pb * X::PST) >> 4), acc0 = flags & G_FIRST ? 0u : 1u;
      const uint32_t d = tm + (ob * NG + (PP ? i & 1 : 0)) * VT * N2;
#pragma unroll 1
      for (int vt = 0; vt < VT; ++vt) {
        const int slot = X::SHARED ? (k0 + vt) % NK : i % NV;
        const uint32_t vb = vbase + ((X::SHARED ? slot * X::KST : X::V_OFF + slot * X::VST) >> 4);
        if (elected()) {
#pragma unroll
          for (int kk = 0; kk < TT / 16; ++kk)
            if (kk < nks) umma_bf16_lo(d + vt * N2, vb + kk * (2 * X::GS >> 4), HIV, pa + kk * 128, HI, IPV, kk ? 1u : acc0);
          if constexpr (X::FULL) {
#pragma unroll
            for (int kk = 0; kk < TT / 16; ++kk)
              if (kk < nks) umma_bf16_lo(d + vt * N2, vb + kk * (2 * X::GS >> 4), HIV, sbase + (X::L_OFF >> 4) + kk * 128, HI, IPV, 1u);
          }
          umma_commit(X::SHARED ? &sh.kempty[slot] : &sh.vempty[slot]);
        }
        __syncwarp();
      }
      if (elected()) {
        umma_commit(X::SHARED ? &sh.pslot[pb] : &sh.kempty[pb]);
        umma_commit(&sh.pempty[i & 1]);
        if (flags & F_LAST) {              // for the groups that had tiles of the segment
          if (!PP || (i & 1) == 0 || !(flags & G_SOLO)) umma_commit(&sh.ofull[0]);
          if (PP && ((i & 1) == 1 || !(flags & G_SOLO))) umma_commit(&sh.ofull[NG - 1]);
        }
      }
      __syncwarp();
    }
    ok = __all_sync(FULL_MASK, ok);
    if (elected()) {
      if (!ok) {
        set_err(a.err, PKV_DEV_TIMEOUT);
        sh.abort_flag = 1;
      }
      umma_commit(&sh.drain);
    }
    rows_wait(&sh.drain, 0, nullptr);
  } else if (warp >= 4) {
    // -------------------------- softmax and epilogue ------------------------
    // Warp w reaches the tensor-memory lanes of quarter w % 4: in S^T the cached rows 16 MT wq + ..., in fragments of
    // 16 rows x 8 query rows, in O^T the channels 32 wq + lane.
    constexpr int RC = PP ? R : R / 2;     // query rows of a group in a tile
    constexpr int NC = RC / 4;             // of a thread: 2 (lane % 4) + {0, 1} of every eight
    constexpr int CB = RC >= 16 ? 2 : 1;   // fragments at a time
    constexpr int NW = PP ? 128 : 256;     // threads that share a tile
    const int wq = warp & 3, gi = (warp - 4) >> 2, hb = PP ? 0 : RC * gi;
    const int wg = PP ? gi : 0, tid = (threadIdx.x - 128) & (NW - 1);
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    const int r0 = 16 * MT * wq + (lane >> 2), c0 = hb + 2 * (lane & 3);   // this thread's first cached row and query row
    float* off = sh.offset[wg];            // offsets of the query rows, the lowest where there is none yet
    float l[NC];                           // this thread's rows' share of the sums of its query rows
    bool unset = false;                    // a query row may have no offset yet
    bool far = false;                      // a query row's offset is beyond kRowsFar
    static_assert(NW % R == 0, "a thread's query row in every pass");
    const int2 mine = row_in<X>(a, tid % R);
    // Barriers among the threads of a tile.  A failed (timed-out) wait makes `bad` true for its warp, which raises a flag ahead
    // of the next barrier; behind that all of them see it and leave together, so no thread is left at a barrier.  The
    // flag goes by the barrier's parity, since a warp may be one barrier ahead of another.
    bool bad = false, gone = false;
    int turn = 0, joins = 0, ends = 0;     // barriers, exchanges and segments so far
    auto sync = [&](bool pred) {
      if (bad) sh.bad[wg][turn & 1] = 1;
      __syncwarp();
      const bool any = named_bar_or(1 + wg, NW, pred || bad);
      if (any && sh.bad[wg][turn & 1]) gone = true;
      ++turn;
      return any;
    };
    auto wait = [&](uint64_t* bar, int round) {               // nothing but that a wait failed, or one of another role did, ends it early
      if (!bad) bad = !rows_wait(bar, round, &sh.abort_flag);
    };

#pragma unroll 1
    for (int i = PP ? gi : 0; sh.any; i += PP ? 2 : 1) {
      const int pb = i % NP, sb = i % NS, k0 = X::SHARED ? i * VT : i;
      // A barrier tells a phase from the one before it only by parity, and this group may not have waited for that.  It is
      // over, though: behind the group's last tile the keys of the tiles before it had landed, and behind this one's
      // scores the tile whose slot they took was done with.
      wait(&sh.kfull[X::SHARED ? 2 * (i % NF) : i % NF], i / NF);   // the metadata, which stay until P is there
      if (bad) {
        sync(true);
        break;
      }
      const RowsMeta& mt = sh.meta[i % NM];
      const int flags = mt.flags, ob = mt.k % NO;
      if (flags & F_END) {
        sync(false);                       // with a warp whose wait for it has failed
        break;
      }
      const bool special = mt.tile0 + TT > mt.ctx - mt.n || mt.invalid;
      // what query row (tid + e NW) % R attends to in word (tid + e NW) / R of the tile's rows
      constexpr int WN = (R * MT + NW - 1) / NW;
      unsigned long long win[WN];
      if (special) {
#pragma unroll
        for (int e = 0; e < WN; ++e) {
          win[e] = 0;
          const int w = (tid + e * NW) / R;
          if (w < MT) {
            const int tok = query_of<X>(a, mt.n, mt.t0, mt.h0, mine).x;
            if (tok >= 0) win[e] = attended(a, mt, tok, mt.tile0 + 64 * w);
          }
        }
        __syncwarp();
      }
      wait(&sh.sfull[sb], i / NS);                            // the scores, and room for P in place of the keys
      if (bad) {
        sync(true);
        break;
      }
      uint8_t* pbuf = sm + X::P_OFF + pb * X::PST;
      RowsScratch<X>& scr = *reinterpret_cast<RowsScratch<X>*>(X::SHARED ? sm + X::W_OFF : pbuf + X::PBUF);
      const uint32_t st = tmem + lane_off + X::S_COL + R * sb + hb, acc = tmem + lane_off + (ob * NG + (PP ? gi : 0)) * VT * N2;
      tc_fence_after();
      if (flags & G_FIRST) {
#pragma unroll
        for (int q = 0; q < NC; ++q) l[q] = 0.f;
        if (a.mask && tid < R && !special) {                  // the masks that the segment will end with
          const int tok = query_of<X>(a, mt.n, mt.t0, mt.h0, mine).x;
          if (tok >= 0) prefetch_l2(a.mask + (size_t)(mt.q0 + tok) * a.mask_words);
        }
        __syncwarp();
      }
      // A tile's weights are taken against the running offsets; where an exponent exceeds them by more than kRowsLazy the
      // offsets are raised and the pass is made again.  A segment's first tile starts from the scores of its first row:
      // offsets need not be the maxima, only near them.  Where not all query rows attend to that, the maxima are taken first, and
      // so they are behind such tiles, where a query row may still have no offset, up to one whose first row all attend to.
      const bool sure = mt.tile0 < mt.ctx - mt.n && !(mt.invalid & 1);
      if (flags & G_FIRST) unset = !sure, far = false;
      bool raise = unset;
      unset = unset && !sure;
      // Behind the row tile's own query rows lie other sequences' tokens or other groups' heads, or zeros: their offset is plus
      // infinity, so that their weights are zeros and no offset is raised for them.
      if ((flags & G_FIRST) && sure) {
        if (wq == 0) {
          const int rows = mt.rows;
#pragma unroll 1
          for (int ch = 0; ch < RC / (8 * CB); ++ch) {
            uint32_t sr[4 * CB];
            tmem_ld_frag(st + ch * 8 * CB, sr);
            tmem_wait_ld();
            if (lane < 4) {
#pragma unroll
              for (int b = 0; b < 2 * CB; ++b) {
                const int c = c0 + 8 * (ch * CB + (b >> 1)) + (b & 1);
                const float x = __uint_as_float(sr[4 * (b >> 1) + (b & 1)]) * a.scale_log2;
                off[c] = (fabsf(x) < kRowsFar ? x : kRowsLowest) + (c < rows ? 0.f : INFINITY);   // (the lowest: to be raised)
              }
            }
            __syncwarp();
          }
        }
        if (!special && (sync(false), gone)) break;            // (behind a masked tile's barrier otherwise)
      }
      if (special) {
        // What each query row attends to, and what any of them does.  Scores that do not count become minus infinities (before
        // the scale) where they lie.
#pragma unroll
        for (int e = 0; e < WN; ++e) {
          const int c = (tid + e * NW) % R, w = (tid + e * NW) / R;
          if (w < MT) scr.win[w][c] = win[e];
          // a warp's lanes hold query rows of one word, or of two: an OR of each word's
          const unsigned group = R >= 32 ? FULL_MASK : (0xffffu << (lane & 16));
          const uint32_t lo = __reduce_or_sync(group, (uint32_t)win[e]), hi = __reduce_or_sync(group, (uint32_t)(win[e] >> 32));
          if (w < MT && lane % (R >= 32 ? 32 : 16) == 0) scr.seen[w][R > 32 ? (c >> 5) : 0] = (unsigned long long)hi << 32 | lo;
        }
        if (PP) {                          // the values, of which some are about to be overwritten, behind the group's last product
          if (i >= 2) wait(&sh.pempty[i & 1], i / 2 - 1);
          wait(&sh.vfull[i % NV], i / NV);
        }
        if (sync(false), gone) break;
        const uint32_t none = a.scale_log2 < 0.f ? 0x7f800000u : 0xff800000u;
#pragma unroll 1
        for (int ch = 0; ch < RC / (8 * CB); ++ch) {
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            uint32_t sr[4 * CB];
            const uint32_t at = st + ((uint32_t)(16 * j) << 16) + ch * 8 * CB;
            tmem_ld_frag(at, sr);
            tmem_wait_ld();
            const int first = 16 * MT * wq + 16 * j;          // the fragment's first row: 16 bits of a word
#pragma unroll
            for (int b = 0; b < 2 * CB; ++b) {
              const int c = c0 + 8 * (ch * CB + (b >> 1)) + (b & 1);
              const uint32_t w = reinterpret_cast<const uint16_t*>(&scr.win[first >> 6][c])[(first & 63) >> 4] >> (lane >> 2);
              if (!(w & 1)) sr[4 * (b >> 1) + (b & 1)] = none;
              if (!(w & 256)) sr[4 * (b >> 1) + 2 + (b & 1)] = none;
            }
            __syncwarp();
            tmem_st_frag(at, sr);
          }
        }
        tmem_wait_st();
        // V rows that no query row attends to, and that the product reads with p = 0: they may hold anything
        const int topr = (min(TT, mt.ctx - mt.tile0) + 15) & ~15, row = PP ? tid : tid >> 2;
        unsigned long long seen = scr.seen[row >> 6][0];
        if constexpr (R > 32) seen |= scr.seen[row >> 6][1];
        if (row < topr && !((seen >> (row & 63)) & 1)) {
#pragma unroll 1
          for (int v = PP ? 0 : tid & 3; v < X::VC * 8; v += PP ? 1 : 4) {
            const int ch = v >> 3;
            uint8_t* base = X::SHARED ? sm + ((k0 + (ch >> 1)) % NK) * X::KST + (ch & 1) * 1024 : sm + X::V_OFF + (i % NV) * X::VST + ch * 1024;
            *reinterpret_cast<uint4*>(base + (row >> 3) * X::GS + (row & 7) * 128 + (v & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        __syncwarp();
      }
      float ts[NC];                        // the tile's part of l
      float mul = a.scale_log2;            // of the scores as they lie
      uint32_t second[X::FULL ? NC * MT : 1];                 // second parts of p that wait for their buffer
#pragma unroll 1
      for (;;) {
        if (raise) {
          // the running maxima of the query rows, this tile's among them
#pragma unroll 1
          for (int ch = 0; ch < RC / (8 * CB); ++ch) {
            uint32_t sr[MT][4 * CB];
#pragma unroll
            for (int j = 0; j < MT; ++j) tmem_ld_frag(st + ((uint32_t)(16 * j) << 16) + ch * 8 * CB, sr[j]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2 * CB; ++b) {
              float v = -INFINITY;
#pragma unroll
              for (int jh = 0; jh < 2 * MT; ++jh) v = fmaxf(v, __uint_as_float(sr[jh >> 1][4 * (b >> 1) + 2 * (jh & 1) + (b & 1)]) * mul);
#pragma unroll
              for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, o));
              if (lane < 4) scr.red[wq][c0 + 8 * (ch * CB + (b >> 1)) + (b & 1)] = v;
            }
            __syncwarp();
          }
          if (!(flags & G_FIRST)) wait(&sh.pempty[PP ? i & 1 : (i - 1) & 1], PP ? i / 2 - 1 : (i - 1) / 2);   // for the rescale
          if (sync(false), gone) break;
          bool large = false;
          if (tid < R) {
            const float mx = fmaxf(fmaxf(scr.red[0][tid], scr.red[1][tid]), fmaxf(scr.red[2][tid], scr.red[3][tid]));
            const bool here = tid < mt.rows;
            const float m = flags & G_FIRST ? (here ? kRowsLowest : INFINITY) : off[tid], mn = fmaxf(m, mx);
            scr.factor[tid] = m == mn ? 1.f : ex2(m - mn);
            off[tid] = mn;
            large = here && fabsf(mn) >= kRowsFar && mx > -INFINITY;   // (not the lowest offset, of a row without a score)
          }
          far |= sync(large);
          if (gone) break;
          if (!(flags & G_FIRST)) {
            // the sums and O so far, to which the products of the tiles before have been added: scaled in place
#pragma unroll
            for (int q = 0; q < NC; ++q) l[q] *= scr.factor[c0 + 8 * (q >> 1) + (q & 1)];
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < VT * HO; ++p) {
#pragma unroll 1
              for (int b = 0; b < RC; b += 8) {
                const uint32_t ta = acc + (p / HO) * N2 + (p % HO) * R + hb + b;
                uint32_t o[8];
                tmem_ld8(ta, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scr.factor[hb + b + e]);
                tmem_st8(ta, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        if (far && mul != 1.f) {
          // the products, rounded, in place of the scores
#pragma unroll 1
          for (int ch = 0; ch < RC / (8 * CB); ++ch) {
#pragma unroll 1
            for (int j = 0; j < MT; ++j) {
              uint32_t sr[4 * CB];
              const uint32_t at = st + ((uint32_t)(16 * j) << 16) + ch * 8 * CB;
              tmem_ld_frag(at, sr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4 * CB; ++e) sr[e] = __float_as_uint(__uint_as_float(sr[e]) * mul);
              tmem_st_frag(at, sr);
            }
          }
          tmem_wait_st();
          mul = 1.f;
        }
        // One pass over the tile: weights against the offsets, into P as bf16 parts, and their sums.  Row t of the B operand:
        // 128 bytes per 64 columns (first parts of the query rows, then the next parts), 16-byte chunk c stored at chunk
        // c ^ (t % 8) (128-byte swizzle).
        float top = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < RC / (8 * CB); ++ch) {
          uint32_t sr[MT][4 * CB];
#pragma unroll
          for (int j = 0; j < MT; ++j) tmem_ld_frag(st + ((uint32_t)(16 * j) << 16) + ch * 8 * CB, sr[j]);
          tmem_wait_ld();
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            const int q = 2 * (ch * CB + b);
            const float2 o = *reinterpret_cast<const float2*>(off + c0 + 4 * q);
            float t0 = 0.f, t1 = 0.f;
#pragma unroll
            for (int jh = 0; jh < 2 * MT; ++jh) {
              const int j = jh >> 1, h = jh & 1, row = r0 + 16 * j + 8 * h;
              const float y0 = fmaf(__uint_as_float(sr[j][4 * b + 2 * h]), mul, -o.x);
              const float y1 = fmaf(__uint_as_float(sr[j][4 * b + 2 * h + 1]), mul, -o.y);
              top = fmaxf(top, fmaxf(y0, y1));
              const float p0 = ex2(y0), p1 = ex2(y1);
              const uint32_t hi = pack_bf16(p0, p1);
              uint8_t* prow = pbuf + row * 128 + 4 * (lane & 3);
              auto put = [&](int part, uint32_t v) {
                const int cc = (part * R + hb) / 8 + (q >> 1);
                *reinterpret_cast<uint32_t*>(prow + (cc >> 3) * X::CHUNK + (((cc & 7) ^ (row & 7)) << 4)) = v;
              };
              put(0, hi);
              const float u0 = p0 - bf16_lo(hi), u1 = p1 - bf16_hi(hi);
              const uint32_t lo = pack_bf16(u0, u1);
              if constexpr (X::FULL) second[(q >> 1) * 2 * MT + jh] = lo;
              else put(1, lo);
              if constexpr (HL == 3) put(2, pack_bf16(u0 - bf16_lo(lo), u1 - bf16_hi(lo)));
              t0 += p0;
              t1 += p1;
            }
            ts[q] = t0;
            ts[q + 1] = t1;
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();          // the rows written above, for the tensor core
        if (raise) break;
        raise = sync(top > kRowsLazy);
        if (gone || !raise) break;
      }
      if (gone) break;
      if constexpr (X::FULL) {
        // the buffer is free behind the last tile's products; that they are known to be behind the ones before, see the top
        if (i > 0) wait(&sh.pempty[(i - 1) & 1], (i - 1) / 2);
        if (!bad) {
#pragma unroll
          for (int e = 0; e < NC * MT; ++e) {
            const int q = e / (2 * MT), row = r0 + 8 * (e % (2 * MT)), cc = hb / 8 + q;
            *reinterpret_cast<uint32_t*>(sm + X::L_OFF + row * 128 + 4 * (lane & 3) + ((cc ^ (row & 7)) << 4)) = second[e];
          }
        }
        __syncwarp();
        fence_proxy_async_smem();
      }
      const bool ends_here = flags & G_LAST;
      float2 own = make_float2(0.f, 0.f);  // of query row tid, at the segment's end
      int out_row = -1;
      if (ends_here) {
        // the sums over all cached rows of the group's tiles, while the scratch is there
#pragma unroll
        for (int q = 0; q < NC; ++q) {
          float v = l[q] + ts[q];
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
          if (lane < 4) scr.red[wq][c0 + 8 * (q >> 1) + (q & 1)] = v;
        }
        if (sync(false), gone) break;
        if (tid < R) own = make_float2(off[tid], (scr.red[0][tid] + scr.red[1][tid]) + (scr.red[2][tid] + scr.red[3][tid]));
        fence_proxy_async_smem();          // of the scratch, which lies in a slot that a copy fills again
      }
      const int part = mt.part, q0 = mt.q0, n = mt.n, t0 = mt.t0, h0 = mt.h0, g = mt.g;   // (they may be gone behind P)
      __syncwarp();
      if (lane == 0 && !bad) {
        mbar_arrive(&sh.pfull[pb]);
        mbar_arrive(&sh.sempty[sb]);
      }
#pragma unroll
      for (int q = 0; q < NC; ++q) l[q] += ts[q];

      if (ends_here) {
        // Behind the segment's last product, its output rows.  With two accumulators the groups exchange their states, and
        // each puts together half of the query rows.
        const bool whole = flags & F_WHOLE, pair = PP && !(flags & G_SOLO);
        if (tid < R) {
          const int2 qh = query_of<X>(a, n, t0, h0, mine);
          if (qh.x >= 0) out_row = (q0 + qh.x) * a.n_h + g * a.G + qh.y;
        }
        __syncwarp();
        // (behind this wait the segment before it in this O buffer is done with, in both groups)
        wait(&sh.ofull[wg], ends++);
        if (pair) {
          if (tid < R && !bad) sh.sum[PP ? ob : 0][wg][PP ? tid : 0] = own;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.joined[wg]);
          wait(&sh.joined[NG - 1 - wg], joins++);             // the other group's (a thread reads no more of its own than it wrote)
        }
        if (tid < R && !bad) {
          // an accumulator none of whose rows counted (its sum is 0) has no part in it
          float2 x = own, y = make_float2(0.f, 0.f);
          if (pair) x = sh.sum[PP ? ob : 0][0][PP ? tid : 0], y = sh.sum[PP ? ob : 0][NG - 1][PP ? tid : 0];
          const float M = fmaxf(x.y == 0.f ? -INFINITY : x.x, y.y == 0.f ? -INFINITY : y.x);
          float2 f = make_float2(x.y == 0.f ? 0.f : ex2(x.x - M), y.y == 0.f ? 0.f : ex2(y.x - M));
          const float L = x.y * f.x + y.y * f.y;
          sh.row[ob][tid] = out_row;
          if (whole) {
            const float inv = sum_inverse(L);
            f.x *= inv;
            f.y *= inv;
          } else if (!pair || gi == 0) {
            *reinterpret_cast<float2*>(a.ws_ml + ((size_t)part * R + tid) * 2) = make_float2(M, L);
          }
          if constexpr (PP) {
            if (!pair || tid / (R / 2) == gi) sh.factor[ob][tid] = f;   // a pair's groups each put together half of the query rows
          } else {
            sh.factor[ob][tid] = f.x;
          }
        }
        if (sync(false), gone) break;
        tc_fence_after();
        const int cb = PP ? (pair ? gi * (R / 2) : 0) : hb, cn = PP && !pair ? R : R / 2;
        const uint32_t oa = tmem + lane_off + ob * NG * VT * N2 + (PP && !pair ? gi * VT * N2 : 0);
#pragma unroll 1
        for (int e0 = 0; e0 < VT * cn; e0 += 8) {
          const int vt = e0 / cn, cc = cb + e0 - vt * cn;
          const int chn = vt * X::VM + (X::VM == 128 ? 32 * wq + lane : 16 * wq + lane);
          float v[8];
          uint32_t t[HO][8];
          auto load = [&](int g) {
            __syncwarp();
#pragma unroll
            for (int p = 0; p < HO; ++p) tmem_ld8(oa + (g * VT + vt) * N2 + p * R + cc, t[p]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
              for (int p = HO - 2; p >= 0; --p) t[HO - 1][e] = __float_as_uint(__uint_as_float(t[HO - 1][e]) + __uint_as_float(t[p][e]));
          };
          load(0);
          if constexpr (PP) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(t[HO - 1][e]) * sh.factor[ob][cc + e].x;
            if (pair) {
              load(NG - 1);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaf(__uint_as_float(t[HO - 1][e]), sh.factor[ob][cc + e].y, v[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(t[HO - 1][e]) * sh.factor[ob][cc + e];
          }
          if (X::VM == 64 && lane >= 16) continue;
          if (!whole) {                    // (rows that no query has are written too)
            float* dst = a.ws_o + ((size_t)part * R + cc) * DV + chn;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e * DV] = v[e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int row = sh.row[ob][cc + e];
              if constexpr (X::F32) {
                if (row >= 0) reinterpret_cast<float*>(a.out)[(size_t)row * DV + chn] = v[e];
              } else {
                if (row >= 0) reinterpret_cast<__nv_bfloat16*>(a.out)[(size_t)row * DV + chn] = __float2bfloat16_rn(v[e]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&sh.oempty[ob], PP && !pair ? 2 : 1);
      }
    }
    if (bad && lane == 0) {
      set_err(a.err, PKV_DEV_TIMEOUT);
      sh.abort_flag = 1;
    }
    if (warp == 11) {
      if (lane == 0 && member == 0) {
        // whether the piece's start cuts a segment for the first time, for the kernel that joins the parts
        RowsCut cut = {};
        if (sh.W > 0) {
          const RowsLine line(sh.W, a.P);
          const int t = sh.first.parts, nt = sh.first.first;
          const long long pstart = line.start(team), seg = pstart - t, prev = team > 0 ? line.start(team - 1) : 0;
          if (t > 0 && prev <= seg) {
            cut = sh.first;
            cut.parts = min(line.piece(min(seg + nt, line.W) - 1), line.P - 1) - team + 2;   // up to the last piece that holds a part
            cut.first = prev == seg ? 0 : 1;
          }
        }
        a.cuts[team] = cut;
      }
      __syncwarp();
    }
    // Sequences without cached rows: their tokens' outputs are zeros
#pragma unroll 1
    for (int s = blockIdx.x; s < a.batch; s += gridDim.x) {
      int flags = 0;
      const Drafts d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, s, flags);
      if (d.ctx > 0 || d.n == 0) continue;
      const long long at = (long long)d.q0 * a.n_h * DV, len = (long long)d.n * a.n_h * DV;
#pragma unroll 1
      for (long long e = threadIdx.x - 128; e < len; e += 256) store_out(a, at + e, 0.f);
    }
  }
  // the tensor memory is released once every role is done with it (the issuers waited for their last products)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, X::TMEM_COLS);
}

// ---- parts of cut segments ----------------------------------------------------------------------------
// Joins the parts of a segment that piece boundaries cut, by its first boundary.  Narrow: a warp per query row and boundary,
// all of its channels.  Wide, for few segments of many parts each: a CTA per query row, whose warps take every eighth
// part and meet in shared memory; there a CTA looks its boundary up among all of them, since most cut nothing anew
// and a CTA for each of those, too, cost a short call 2 to 4 us.
template <class X, bool WIDE>
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int R = X::R, DV = X::DV, V = DV < 128 ? 2 : 4, CH = DV / (32 * V);   // channels lane V + 32 V j + ...
  grid_dep_wait();
  grid_dep_launch();
  const int member = blockIdx.x % a.C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ unsigned some[8];
  if constexpr (WIDE) {                    // boundaries with something to join (of at most 256)
    const unsigned mine = __ballot_sync(FULL_MASK, threadIdx.x < a.P && a.cuts[threadIdx.x].parts != 0);
    if (lane == 0) some[warp] = mine;
  }
#pragma unroll 1
  for (int turn = blockIdx.x / a.C;; turn += gridDim.x / a.C) {
    int team = turn;
    if constexpr (WIDE) {
      __syncthreads();
      int left = turn;
      team = -1;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int n = __popc(some[w]);
        if (team < 0 && left < n) team = 32 * w + __fns(some[w], 0, left + 1);
        left -= n;
      }
      if (team < 0) return;
    }
    const RowsCut cut = a.cuts[team];
    if (cut.parts == 0) return;
    const int c = WIDE ? blockIdx.y : blockIdx.y * 8 + warp;
    int t0, h0;
    tile_of<X>(a, cut.rg * a.C + member, t0, h0);
    const int2 qh = query_of<X>(a, cut.n, t0, h0, row_in<X>(a, c));
    if (qh.x < 0) {                          // (of the whole CTA, where it is wide)
      if (WIDE) continue;
      return;
    }
    const long long row = (long long)(cut.q0 + qh.x) * a.n_h + cut.g * a.G + qh.y;
    float M = -INFINITY, L = 0.f, acc[CH][V];
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
    constexpr int AT = DV > 256 ? 2 : 4;     // parts at a time, with all their loads ahead of the first use
#pragma unroll 1
    for (int p0 = WIDE ? warp * AT : 0; p0 < cut.parts; p0 += WIDE ? 8 * AT : AT) {
      float2 ml[AT];
      float o[AT][CH][V];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int p = min(p0 + i, cut.parts - 1);
        const size_t at = (size_t)(((team - 1 + p) * a.C + member) * 2 + (p == 0 ? cut.first : 0)) * R + c;
        ml[i] = *reinterpret_cast<const float2*>(a.ws_ml + 2 * at);
        if (p0 + i >= cut.parts) ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const float* src = a.ws_o + at * DV + lane * V + 32 * V * j;
          if constexpr (V == 4) *reinterpret_cast<float4*>(o[i][j]) = *reinterpret_cast<const float4*>(src);
          else *reinterpret_cast<float2*>(o[i][j]) = *reinterpret_cast<const float2*>(src);
        }
      }
      float top = M;
#pragma unroll
      for (int i = 0; i < AT; ++i) top = fmaxf(top, ml[i].x);
      const float base = top == -INFINITY ? 0.f : top, keep = ex2(M - base);
      L *= keep;
      float w[AT];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        w[i] = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - base);
        L += w[i] * ml[i].y;
      }
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[j][v] *= keep;
#pragma unroll
          for (int i = 0; i < AT; ++i) acc[j][v] += w[i] * o[i][j][v];
        }
      M = top;
    }
    auto store = [&](int ch, const float* x) {
      const size_t at = (size_t)row * DV + ch;
      if constexpr (X::F32) {
        if constexpr (V == 4) *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(x[0], x[1]);
      } else {
        uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at);
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        else *dst = pack_bf16(x[0], x[1]);
      }
    };
    if constexpr (WIDE) {
      __shared__ float2 s_ml[8];
      __shared__ __align__(16) float s_o[8][DV];
      if (lane == 0) s_ml[warp] = make_float2(M, L);
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[warp][lane * V + 32 * V * j + v] = acc[j][v];
      __syncthreads();
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, s_ml[i].x);
      if (top == -INFINITY) top = 0.f;
      float sum = 0.f, f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = ex2(s_ml[i].x - top);
        sum += f[i] * s_ml[i].y;
      }
      const float inv = sum_inverse(sum);
      for (int ch = threadIdx.x * V; ch < DV; ch += 256 * V) {
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[v] = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[v] += f[i] * s_o[i][ch + v];
          x[v] *= inv;
        }
        store(ch, x);
      }
    } else {
      const float inv = sum_inverse(L);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] *= inv;
        store(lane * V + 32 * V * j, acc[j]);
      }
    }
    if (!WIDE) return;
  }
}

// ---- variants ----------------------------------------------------------------------------------------
struct RowsVariant {
  const void *fn, *join[2];
  size_t smem;
  int R, DV;
  bool ready[64];
};

template <class X>
static RowsVariant make_variant() {
  constexpr size_t smem = X::M_OFF + sizeof(RowsShared<X>);
  static_assert(smem <= 232448, "shared memory of one CTA");
  static_assert(sizeof(RowsScratch<X>) <= (X::SHARED ? X::M_OFF - X::W_OFF : X::KPART - X::PBUF), "scratch of a tile");
  static_assert(X::Q_OFF % 1024 == 0 && X::V_OFF % 1024 == 0 && X::P_OFF % 1024 == 0 && X::NCOL <= 512, "descriptor alignment, tensor memory");
  return {(const void*)decode_rows_kernel<X>, {(const void*)rows_join_kernel<X, false>, (const void*)rows_join_kernel<X, true>}, smem, X::R, X::DV, {}};
}
// bf16 outputs take p in two bf16 parts (16 bits), whatever the number of query rows: with one part (8 bits) in the 64-row variants
// 8 trees of 512 rows took 369 us and not 388, 32 latent tokens of 128 heads 123 and not 143, but the error of a sequence's
// output went from 1.7e-3 to 2.3e-3 (relative, 1.7e-3 of it the output's own rounding) and depended on which others were in its batch.
// fp32 outputs take three parts (all 24 bits), with 32 query rows at most: more columns do not fit the tensor memory beside a
// latent cache's O.
static int variant_index(int R, bool f32) { return f32 ? (R == 16 ? 3 : 4) : (R == 16 ? 0 : (R == 32 ? 1 : 2)); }
static RowsVariant* kv_variant(int d, int R, bool f32) {
  static RowsVariant v[2][5] = {
      {make_variant<RowsCfg<1, 1, 64, false, 16, 2>>(), make_variant<RowsCfg<1, 1, 64, false, 32, 2>>(),
       make_variant<RowsCfg<1, 1, 64, false, 64, 2>>(), make_variant<RowsCfg<1, 1, 64, false, 16, 3>>(),
       make_variant<RowsCfg<1, 1, 64, false, 32, 3>>()},
      {make_variant<RowsCfg<2, 1, 128, false, 16, 2>>(), make_variant<RowsCfg<2, 1, 128, false, 32, 2>>(),
       make_variant<RowsCfg<2, 1, 128, false, 64, 2>>(), make_variant<RowsCfg<2, 1, 128, false, 16, 3>>(),
       make_variant<RowsCfg<2, 1, 128, false, 32, 3>>()}};
  return &v[d == 128][variant_index(R, f32)];
}
static RowsVariant* latent_variant(int latent, int R, bool f32) {
  static RowsVariant v[2][5] = {
      {make_variant<RowsCfg<5, 2, 128, true, 16, 2>>(), make_variant<RowsCfg<5, 2, 128, true, 32, 2>>(),
       make_variant<RowsCfg<5, 2, 128, true, 64, 2>>(), make_variant<RowsCfg<5, 2, 128, true, 16, 3>>(),
       make_variant<RowsCfg<5, 2, 128, true, 32, 3>>()},
      {make_variant<RowsCfg<9, 4, 128, true, 16, 2>>(), make_variant<RowsCfg<9, 4, 128, true, 32, 2>>(),
       make_variant<RowsCfg<9, 4, 128, true, 64, 2>>(), make_variant<RowsCfg<9, 4, 128, true, 16, 3>>(),
       make_variant<RowsCfg<9, 4, 128, true, 32, 3>>()}};
  return &v[latent == 512][variant_index(R, f32)];
}

// Query rows of a row tile, and members of a team, from the average of the sequences' query rows per kv head.  Rows that no
// query has cost products and softmax all the same, row tiles loads: 64 trees of 16 rows took 99 us with R = 16, 102
// with 32 and 109 with 64, of 32 rows 102 with 32 and 109 with 64, of 64 rows 111 with 64 and 153 with 32; 64 latent tokens of 16
// heads 41, 43 and 54 with 16, 32 and 64.  Two members read what one CTA loads twice (32 latent tokens of 128 heads 144 us and
// 151, 8 trees of 512 rows 390 and 404), but where the sequences' rows differ one of them may have no tile (12 trees over the latent
// cache 54 and 53; with four members 66, and 412 for the 8 trees).
struct RowsShape {
  int R, C, P;
  long long groups;              // of row tiles, on average
};
static RowsShape rows_shape(int n_tok, int batch, int G, bool f32) {
  const long long rows = ((long long)n_tok * G + batch - 1) / batch;
  RowsShape s;
  s.R = rows <= 16 && G <= 16 ? 16 : (rows <= 32 || f32 ? 32 : 64);
  const long long tiles = (rows + s.R - 1) / s.R;
  s.C = tiles <= 1 ? 1 : 2;
  const int sms = device_sm_count();
  s.P = sms / s.C;
  s.groups = (tiles + s.C - 1) / s.C;
  return s;
}
struct RowsLayout {
  size_t ml, o, total;
};
static RowsLayout rows_layout(const RowsShape& s, int DV) {
  RowsLayout l;
  const size_t parts = (size_t)s.P * s.C * 2 * s.R;
  l.ml = align_up(sizeof(RowsCut) * (size_t)s.P, 256);
  l.o = align_up(l.ml + parts * 2 * sizeof(float), 256);
  l.total = align_up(l.o + parts * DV * sizeof(float), 256);
  return l;
}

// Enough for either output type; 0 without a device.
static size_t most_layout(const RowsShape& x, const RowsShape& y, int DV) {
  if (x.P < 1 || y.P < 1) return 0;
  const size_t a = rows_layout(x, DV).total, b = rows_layout(y, DV).total;
  return a > b ? a : b;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr long long kRowsMaxCtx = 0x7fff0000LL;

static bool valid_step(int n_tok, int batch, const int32_t* q_start, const int64_t* mask, int mask_words, int out_dtype,
                       int max_blocks, int num_blocks) {
  if (n_tok < 0 || batch < 0 || max_blocks < 0 || num_blocks < 0) return false;
  if (out_dtype != PKV_OUT_BF16 && out_dtype != PKV_OUT_F32) return false;
  if (mask && mask_words < 1) return false;
  return q_start || batch == 0 ? true : n_tok % batch == 0;
}
static bool valid_block(int bs) { return bs == 16 || bs == 32 || bs == 64; }
static bool valid_heads(int n_h, int n_kv, int d, int bs) {
  return n_h > 0 && n_kv > 0 && n_h % n_kv == 0 && n_h / n_kv <= 64 && (d == 64 || d == 128) && valid_block(bs);
}
static bool valid_latent(int n_h, int latent, int rope, int bs) {
  return n_h > 0 && n_h <= 1024 && (latent == 256 || latent == 512) && (rope == 32 || rope == 64) && valid_block(bs);
}

// The kernel's attribute, once per device.
static bool rows_ready(RowsVariant* v) {
  static std::mutex lock;
  const std::lock_guard<std::mutex> g(lock);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (v->ready[dev]) return true;
  if (cudaFuncSetAttribute(v->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)v->smem) != cudaSuccess) return false;
  v->ready[dev] = true;
  return true;
}

// What both calls share behind their own checks; w: channels of a key, latent: whether v is the cache k.
static pkv_status rows_attn(const RowsShape& s, RowsVariant* v, bool latent, const void* q, const void* k, const void* vp,
                            const int32_t* bt, int max_blocks, const int32_t* ctx, const int32_t* q_start, const int64_t* mask,
                            int mask_words, float scale, int n_tok, int batch, int n_h, int n_kv, int w, int block_size,
                            int num_blocks, void* out, int out_dtype, void* ws, size_t ws_bytes, int32_t* err, void* stream) {
  if (!q || !k || !vp || !bt || !ctx || !out || !ws) return PKV_EINVAL;
  if (!al16(q) || !al16(k) || !al16(vp) || !al16(out) || (reinterpret_cast<uintptr_t>(mask) & 7u) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return PKV_EINVAL;
  if ((long long)max_blocks * block_size > kRowsMaxCtx || (long long)n_tok * n_h > 0x7fffffffLL) return PKV_ERANGE;
  const RowsLayout lay = rows_layout(s, v->DV);
  if (ws_bytes < lay.total) return PKV_ENOSPC;
  {
    // the output and the workspace are written while the rest is still read
    const size_t out_bytes = (size_t)n_tok * n_h * v->DV * (out_dtype == PKV_OUT_F32 ? 4 : 2);
    const size_t own = lay.total > 256 ? lay.total : 256, pool = (size_t)num_blocks * n_kv * block_size * w * 2;
    const struct { const void* at; size_t bytes; } read[] = {
        {q, (size_t)n_tok * n_h * w * 2}, {k, pool}, {vp, latent ? 0 : pool}, {bt, (size_t)batch * max_blocks * 4}, {ctx, (size_t)batch * 4},
        {q_start, ((size_t)batch + 1) * 4}, {mask, (size_t)n_tok * mask_words * 8}, {err, 4}};
    for (const auto& r : read)
      if (r.bytes && (overlaps(out, out_bytes, r.at, r.bytes) || overlaps(ws, own, r.at, r.bytes))) return PKV_EINVAL;
    if (overlaps(out, out_bytes, ws, own)) return PKV_EINVAL;
  }
  if (s.P < 1 || !rows_ready(v)) {
    record_cuda_error(cudaGetLastError());
    return PKV_ECUDA;
  }
  RowsArgs a = {};
  a.bt = bt; a.ctx = ctx; a.q_start = q_start; a.mask = mask; a.mask_words = mask_words;
  a.max_blocks = max_blocks;
  a.max_ctx = max_blocks * block_size;
  a.n_tok = n_tok; a.batch = batch; a.n_h = n_h; a.n_kv = n_kv; a.G = n_h / n_kv;
  a.num_blocks = num_blocks;
  a.bs_log2 = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
  a.n_each = q_start ? 0 : n_tok / batch;
  a.gt = a.G < s.R ? a.G : s.R;
  a.tpt = s.R / a.gt;
  a.hc = (a.G + a.gt - 1) / a.gt;
  a.last_steps = (w - v->DV) / 16;
  a.C = s.C; a.P = s.P;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.1754944e-38f;      // a masked score times the scale stays an infinity
  a.out = out;
  a.out_f32 = out_dtype == PKV_OUT_F32;
  a.err = err;
  a.cuts = static_cast<RowsCut*>(ws);
  a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.ml);
  a.ws_o = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.o);

  CUtensorMap tmk, tmv, tmq;
  const uint64_t row = (uint64_t)w * 2, rows = (uint64_t)n_kv * block_size, nblk = num_blocks > 0 ? (uint64_t)num_blocks : 1;
  int bad = encode_tensor_map_chunks(&tmk, k, v->DV / 64, rows, nblk, row, latent ? 2 : v->DV / 64, block_size);
  if (latent) {
    bad |= encode_tensor_map_3d(&tmv, k, w, rows, nblk, row, rows * row, 64, block_size);   // for the position chunk
    bad |= encode_tensor_map_3d(&tmq, q, w, (uint64_t)n_tok * n_h, 1, row, row, 64, s.R);
  } else {
    bad |= encode_tensor_map_chunks(&tmv, vp, v->DV / 64, rows, nblk, row, v->DV / 64, block_size);
    bad |= encode_tensor_map_3d(&tmq, q, w, n_h, n_tok, row, n_h * row, 64, a.gt, a.tpt);
  }
  if (bad) return PKV_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* kargs[] = {&tmk, &tmv, &tmq, &a};
  cudaError_t e = launch_pdl(v->fn, dim3(s.P * s.C), dim3(384), v->smem, st, kargs);
  if (e == cudaSuccess) {
    // The pieces over the segments: about the parts that each has, if it has so many tiles.  16 heads over 64K latent tokens:
    // 65 us by a warp per query row, 30 by a CTA; 64 trees of 64 rows: 111 and 156.
    const long long segments = (long long)batch * n_kv * s.groups, tiles = a.max_ctx / (latent ? 64 : 128);
    const bool wide = s.P >= 8 * segments && tiles >= 8 && s.P <= 256;
    void* jargs[] = {&a};
    e = launch_pdl(v->join[wide], dim3((wide ? (int)segments : s.P) * s.C, wide ? s.R : s.R / 8), dim3(256), 0, st, jargs);
  }
  if (e == cudaSuccess) return PKV_OK;
  record_cuda_error(e);
  return PKV_ECUDA;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_tree_workspace_bytes(int batch, int n_tok, int n_h, int n_kv, int head_dim, int block_size) {
  if (batch < 0 || n_tok < 0 || !valid_heads(n_h, n_kv, head_dim, block_size)) return 0;
  if (batch == 0 || n_tok == 0) return 256;
  const RowsShape x = rows_shape(n_tok, batch, n_h / n_kv, false), y = rows_shape(n_tok, batch, n_h / n_kv, true);
  return most_layout(x, y, head_dim);
}

extern "C" pkv_status pkv_paged_tree_attn(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                                          int max_blocks, const int32_t* context_lens, const int32_t* q_start,
                                          const int64_t* tree_mask, int mask_words, float scale, int n_tok, int batch,
                                          int n_h, int n_kv, int head_dim, int block_size, int num_blocks, void* out,
                                          int out_dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                          void* stream) {
  PKV_NVTX("pkv_paged_tree_attn");
  if (!valid_heads(n_h, n_kv, head_dim, block_size) ||
      !valid_step(n_tok, batch, q_start, tree_mask, mask_words, out_dtype, max_blocks, num_blocks))
    return PKV_EINVAL;
  if (n_tok == 0 || batch == 0) return PKV_OK;
  const bool f32 = out_dtype == PKV_OUT_F32;
  const RowsShape s = rows_shape(n_tok, batch, n_h / n_kv, f32);
  RowsVariant* v = kv_variant(head_dim, s.R, f32);
  return rows_attn(s, v, false, q, k_pool, v_pool, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words, scale,
                   n_tok, batch, n_h, n_kv, head_dim, block_size, num_blocks, out, out_dtype, workspace, workspace_bytes, err_flag,
                   stream);
}

extern "C" size_t pkv_latent_workspace_bytes(int batch, int n_tok, int n_h, int latent, int rope, int block_size) {
  if (batch < 0 || n_tok < 0 || !valid_latent(n_h, latent, rope, block_size)) return 0;
  if (batch == 0 || n_tok == 0) return 256;
  return most_layout(rows_shape(n_tok, batch, n_h, false), rows_shape(n_tok, batch, n_h, true), latent);
}

extern "C" pkv_status pkv_paged_latent_attn(const void* q, const void* cache, const int32_t* block_tables, int max_blocks,
                                            const int32_t* context_lens, const int32_t* q_start, const int64_t* tree_mask,
                                            int mask_words, float scale, int n_tok, int batch, int n_h, int latent, int rope,
                                            int block_size, int num_blocks, void* out, int out_dtype, void* workspace,
                                            size_t workspace_bytes, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_paged_latent_attn");
  if (!valid_latent(n_h, latent, rope, block_size) ||
      !valid_step(n_tok, batch, q_start, tree_mask, mask_words, out_dtype, max_blocks, num_blocks))
    return PKV_EINVAL;
  if (n_tok == 0 || batch == 0) return PKV_OK;
  const bool f32 = out_dtype == PKV_OUT_F32;
  const RowsShape s = rows_shape(n_tok, batch, n_h, f32);
  RowsVariant* v = latent_variant(latent, s.R, f32);
  return rows_attn(s, v, true, q, cache, cache, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words, scale, n_tok,
                   batch, n_h, 1, latent + rope, block_size, num_blocks, out, out_dtype, workspace, workspace_bytes, err_flag, stream);
}
