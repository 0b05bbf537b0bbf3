// Attention of many query rows per cached row on the fifth-generation tensor cores: a sequence's drafted tokens
// times the query heads of a group over the paged bf16 cache, or times all heads over the latent cache.
//
// Mathematics: one pass over the cached rows with a running softmax in base 2.  Everything is kept transposed,
// cached rows on the M side of the tensor core and query rows on its N side: with 16 to 64 query rows N is
// what may be small, and M = 128 (64) cached rows or channels fills the tensor core's lanes.
//   S^T[rows of the tile][R]   = K Q^T                 (both K-major, as they lie in memory)
//   O^T[channels][R or 2 R]   += V^T [P_hi | P_lo]^T   (both MN-major, as they lie in shared memory)
// K and V of a latent cache are the same rows, which are loaded once: V is the first channels of the K stage.
//
// Work partition: the line of all (sequence, kv head, group of row tiles, tile of cached rows), in that order, is
// cut into equal pieces, one for each team of C CTAs; the members of a team take C row tiles of
// the same cached rows at the same time, so those come from HBM once.  A CTA finds its piece from the lengths by a
// block-wide scan.  A segment (all tiles of one row tile) that a piece boundary cuts leaves partial softmax states, which a
// second kernel joins; a piece holds at most two cut segments, its first and its last.
//
// A CTA of 12 warps runs these roles, joined by mbarriers with bounded waits:
//   warp 0      K (or latent) tiles into a ring of stages by TMA, and each segment's query rows
//   warp 3      V tiles, in a ring of their own
//   warp 1      owner of the tensor memory; one thread issues the first product into one of two S buffers
//   warp 2      one thread issues the second product
//   warps 4-11  softmax and epilogue, in two groups of four warps that take half of the R query rows each
#include <cmath>
#include <mutex>

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
  int max_blocks, max_ctx, mask_words, n_tok, batch, n_h, n_kv, G, num_blocks, n_each;
  int tile_rows;                 // query rows of a row tile: whole tokens of G heads; R where there is one kv head
  int C, P;                      // members of a team, teams
  float scale_log2;
  void* out;
  int out_f32;
  int32_t* err;
  RowsCut* cuts;                 // [P]
  float *ws_ml, *ws_o;           // [P * C][2][R][2] and [P * C][2][R][DV]
};

// KC: 64-channel chunks of a key; VT: M tiles of VM channels of a value; R: query rows; HL: parts of p (high, low)
template <int BS_, int KC_, int VT_, int VM_, bool SHARED_, int R_, int HL_>
struct RowsCfg {
  static constexpr int BS = BS_, KC = KC_, VT = VT_, VM = VM_, R = R_, HL = HL_;
  static constexpr bool SHARED = SHARED_;
  static constexpr int TT = SHARED ? 64 : 128;                // cached rows of a tile
  static constexpr int MT = TT / 64;
  static constexpr int NBT = TT / BS;
  static constexpr int DV = VT * VM, VC = DV / 64;
  static constexpr int CHUNK = TT * 128;
  static constexpr int KST = KC * CHUNK, VST = SHARED ? 0 : VC * CHUNK;
  static constexpr int N2 = R * HL;                           // columns of the second product
  static constexpr int QCH = R * 128, QBUF = KC * QCH;
  static constexpr int PAT = (N2 + 63) / 64, PBUF = PAT * CHUNK;
  // stages and buffers, from what 227 KB hold
  static constexpr int NQ = SHARED && R == 64 ? 1 : 2;
  static constexpr int NP = SHARED && R >= 32 ? 1 : (SHARED ? 2 : (R == 64 ? 1 : 2));
  static constexpr int NK = 2 * (SHARED ? (KC <= 5 ? 2 : 1) : (KC == 1 ? 2 : 1));
  static constexpr int NV = SHARED ? 0 : (KC == 1 ? 6 : (R == 64 ? 3 : 3));
  static constexpr int NO = VT * N2 * 2 + 2 * R <= 512 ? 2 : 1;
  static constexpr int NCOL = VT * N2 * NO + 2 * R;
  static constexpr uint32_t TMEM_COLS = NCOL <= 64 ? 64 : (NCOL <= 128 ? 128 : (NCOL <= 256 ? 256 : 512));
  static constexpr int S_COL = VT * N2 * NO;                  // S buffers behind the O buffers
  static constexpr int V_OFF = NK * KST, Q_OFF = V_OFF + NV * VST, P_OFF = Q_OFF + NQ * QBUF, M_OFF = P_OFF + NP * PBUF;
};

struct RowsMeta {
  int flags, k;                  // F_ flags; number of the segment in the piece
  int tile0, ctx, n, q0;         // first cached row of the tile; the sequence
  int row0, g;                   // first query row of the row tile (of the n * G or n * n_h ones), kv head
  int invalid, part;             // blocks of the tile with a bad id; partial state of a cut segment
};

enum : int { RB_KFULL = 0, RB_KEMPTY = 4, RB_VFULL = 8, RB_VEMPTY = 14, RB_QFULL = 20, RB_QEMPTY = 22, RB_SFULL = 24, RB_SEMPTY = 26,
             RB_PFULL = 28, RB_PEMPTY = 30, RB_OFULL = 32, RB_OEMPTY = 34, RB_DRAIN = 36, RB_DRAIN_PV = 37, RB_COUNT = 38 };

// Where a CTA stands on the line.
struct RowsCursor {
  Drafts d;
  int s, g, rg, t, nt, rt;       // sequence, kv head, group of row tiles, tile; tiles of a segment, row tiles
  int at_start;                  // still in the segment that the piece starts in
  int whole_from;                // the segment began in this piece
  long long left;                // tiles of the piece from here on (this one included)
};

template <class X>
struct RowsShared {
  static constexpr int R = X::R;
  RowsMeta kmeta[X::NK], vmeta[X::NV > 0 ? X::NV : 1];
  uint64_t bar[RB_COUNT];
  uint32_t tmem;
  int any;
  volatile int abort_flag;
  RowsCursor cur;
  union {
    long long scan[12];                                       // of the setup
    float red[4 * R];                                         // each warp's part of a query row's maximum or sum
  };
  float factor[R];                                            // of each query row: of a rescale, then of the output
  // Attended rows of a tile, by each query row and by any; at a segment's end, behind the vote of the group whose
  // query row c is, win[c] holds its final offset and its output row instead.
  unsigned long long win[X::MT * R], seen[2];
  __device__ float& offset(int c) { return reinterpret_cast<float*>(win + c)[0]; }
  __device__ int& row(int c) { return reinterpret_cast<int*>(win + c)[1]; }
};

__device__ __forceinline__ int row_tiles(const RowsArgs& a, int n) { return (int)(((long long)n * a.G + a.tile_rows - 1) / a.tile_rows); }
__device__ __forceinline__ long long line_length(const RowsArgs& a, const Drafts& d, int tt) {
  const int rt = row_tiles(a, d.n);
  return (long long)a.n_kv * ((rt + a.C - 1) / a.C) * ((d.ctx + tt - 1) / tt);
}

// Moves to the next tile of this member (false: the piece has none left).  Row tiles past the last one are passed over.
template <int TT>
__device__ __forceinline__ bool rows_settle(RowsCursor& c, const RowsArgs& a, int member) {
  while (c.left > 0) {
    if (c.t >= c.nt) {
      c.t = 0;
      c.at_start = 0;
      c.whole_from = 1;
      if (++c.rg * a.C >= c.rt) {
        c.rg = 0;
        if (++c.g >= a.n_kv) {
          c.g = 0;
          int flags = 0;
          do {
            if (++c.s >= a.batch) return false;
            c.d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, c.s, flags);
            c.nt = (c.d.ctx + TT - 1) / TT;
            c.rt = row_tiles(a, c.d.n);
          } while (c.nt == 0 || c.rt == 0);
        }
      }
    }
    if (c.rg * a.C + member < c.rt) return true;
    c.left -= c.nt - c.t;
    c.t = c.nt;
  }
  return false;
}

__device__ __forceinline__ float sum_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }   // a sum that is no number stays one

// Output row of column c of a row tile (-1: none): rows are tokens times the group's heads.
__device__ __forceinline__ long long out_row(const RowsArgs& a, int q0, int n, int g, int row0, int c) {
  const int r = row0 + c;
  if (c >= a.tile_rows || r >= n * a.G) return -1;
  return (long long)(q0 + r / a.G) * a.n_h + g * a.G + r % a.G;
}
__device__ __forceinline__ void store_out(const RowsArgs& a, long long at, float v) {
  if (a.out_f32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ unsigned long long ones_below(int b) { return b <= 0 ? 0ull : (b >= 64 ? ~0ull : (1ull << b) - 1); }

// Which of the 64 cached rows from `first` on token i of a sequence attends to.
__device__ __forceinline__ unsigned long long attended(const RowsArgs& a, const RowsMeta& mt, int i, int first) {
  const int o = mt.ctx - mt.n - first;                        // the first drafted token's row, from `first`
  const unsigned long long cached = ones_below(mt.ctx - first);
  if (!a.mask) return ones_below(o + i + 1) & cached;
  unsigned long long w = 0;
  if (o < 64) {
    const int64_t* m = a.mask + (size_t)(mt.q0 + i) * a.mask_words;
    if (o >= 0) {
      w = (unsigned long long)m[0] << o;
    } else {
      const int q = -o >> 6, r = -o & 63;
      if (q < a.mask_words) w = (unsigned long long)m[q] >> r;
      if (r && q + 1 < a.mask_words) w |= (unsigned long long)m[q + 1] << (64 - r);
    }
  }
  return (ones_below(o) | w) & cached;
}

template <class X>
__global__ void __launch_bounds__(384, 1)
    decode_rows_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ CUtensorMap tmq, const __grid_constant__ RowsArgs a) {
  constexpr int TT = X::TT, BS = X::BS, R = X::R, HL = X::HL, N2 = X::N2, KC = X::KC, VT = X::VT, MT = X::MT, DV = X::DV;
  constexpr int NK = X::NK, NV = X::SHARED ? X::NK : X::NV;
  extern __shared__ __align__(1024) uint8_t sm[];
  RowsShared<X>& sh = *reinterpret_cast<RowsShared<X>*>(sm + X::M_OFF);
  RowsMeta* vmeta = X::SHARED ? sh.kmeta : sh.vmeta;
  uint64_t* bar = sh.bar;
  constexpr int VFULL = X::SHARED ? RB_KFULL : RB_VFULL, VEMPTY = X::SHARED ? RB_KEMPTY : RB_VEMPTY;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / a.C, member = blockIdx.x % a.C;
  if (smem_u32(sm) & 1023u) {              // the descriptors and the swizzle count on it, and there is no room to align it here
    if (threadIdx.x == 0) set_err(a.err, PKV_DEV_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.any = 0;
    for (int b = 0; b < RB_COUNT; ++b)
      mbar_init(&bar[b], (b >= RB_SEMPTY && b < RB_PEMPTY) || b == RB_OEMPTY || b == RB_OEMPTY + 1 ? 8 : 1);   // one arrival per softmax warp
    fence_barrier_init();
    prefetch_tensormap(&tmk);
    if (!X::SHARED) prefetch_tensormap(&tmv);
    prefetch_tensormap(&tmq);
  }
  if (warp == 1) tmem_alloc(&sh.tmem, X::TMEM_COLS);
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
    for (int s = s0; s < s1; ++s) mine += line_length(a, drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, s, flags), TT);
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
    const int Pe = (int)(W < a.P ? W : a.P);
    if (team < Pe) {
      const long long pstart = W * team / Pe, pend = W * (team + 1) / Pe;
      if (pstart >= before && pstart < before + mine) {
        RowsCursor c;
        long long off = pstart - before;
        for (c.s = s0;; ++c.s) {
          c.d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, c.s, flags);
          const long long len = line_length(a, c.d, TT);
          if (off < len || c.s + 1 >= s1) break;
          off -= len;
        }
        c.nt = max(1, (c.d.ctx + TT - 1) / TT);
        c.rt = row_tiles(a, c.d.n);
        const int groups = max(1, (c.rt + a.C - 1) / a.C);
        c.t = (int)(off % c.nt);
        c.rg = (int)(off / c.nt % groups);
        c.g = (int)(off / c.nt / groups);
        c.at_start = 1;
        c.whole_from = c.t == 0;
        c.left = pend - pstart;
        if (member == 0) {
          RowsCut cut = {};
          const long long seg = pstart - c.t, prev = team > 0 ? W * (team - 1) / Pe : 0;
          if (c.t > 0 && prev <= seg) {
            const int last = (int)min(((seg + c.nt) * Pe - 1) / W, (long long)Pe - 1);   // the last piece that holds a part
            cut.parts = last - team + 2;
            cut.first = prev == seg ? 0 : 1;
            cut.q0 = c.d.q0; cut.n = c.d.n; cut.g = c.g; cut.rg = c.rg;
          }
          a.cuts[team] = cut;
        }
        const bool any = rows_settle<TT>(c, a, member);
        sh.cur = c;
        sh.any = any;
      }
    } else if (member == 0 && threadIdx.x == 0) {
      a.cuts[team] = RowsCut{};
    }
  }
  // query rows past a tile's own hold zeros until the end
  if constexpr (!X::SHARED)
    for (int i = threadIdx.x; i < X::NQ * X::QBUF / 16; i += 384) reinterpret_cast<uint4*>(sm + X::Q_OFF)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (sh.any && (warp == 0 || (warp == 3 && !X::SHARED))) {
    // ------------------------------- producers -------------------------------
    const bool kside = warp == 0;
    const int depth = kside ? NK : NV, NC = kside ? KC : X::VC;
    const uint64_t pol = policy_evict_first();
    RowsCursor c = sh.cur;
    int k = -1, kq = -1, i = 0;
    struct Tile {
      RowsMeta m;
      int nblk, phys, first;
    };
    // the tile at the cursor, which then moves on; false when it was the last one
    auto describe = [&](Tile& t) {
      const bool first = k < 0 || c.t == 0;
      if (first) ++k;
      t.first = first;
      t.m.k = k;
      t.m.tile0 = c.t * TT;
      t.m.ctx = c.d.ctx; t.m.n = c.d.n; t.m.q0 = c.d.q0;
      t.m.row0 = (c.rg * a.C + member) * a.tile_rows;
      t.m.g = c.g;
      t.m.part = blockIdx.x * 2 + (c.at_start ? 0 : 1);
      const int blk0 = c.t * X::NBT, nb = (c.d.ctx + BS - 1) / BS;
      t.nblk = min(nb - blk0, X::NBT);
      const int32_t* row = a.bt + (size_t)c.s * a.max_blocks + blk0;
      t.phys = lane < t.nblk ? row[lane] : -1;
      const bool seg_end = c.t + 1 == c.nt;
      t.m.flags = (first ? F_FIRST : 0) | (seg_end || c.left == 1 ? F_LAST : 0) | (seg_end && c.whole_from ? F_WHOLE : 0);
      ++c.t;
      --c.left;
      const bool more = rows_settle<TT>(c, a, member);
      if (!more) t.m.flags |= F_END;
      return more;
    };
    Tile t, tn;
    bool more = describe(t);
    for (;; ++i) {
      bool more2 = false;
      if (more) more2 = describe(tn);                         // its block ids in flight
      const int slot = i % depth, qb = t.m.k % X::NQ;
      uint64_t* fullb = &bar[(kside ? RB_KFULL : VFULL) + slot];
      bool ok = !sh.abort_flag;
      if (ok && i >= depth && lane == 0) ok = mbar_wait(&bar[(kside ? RB_KEMPTY : VEMPTY) + slot], (i / depth - 1) & 1);
      if (ok && kside && t.first && t.m.k >= X::NQ && lane == 0) ok = mbar_wait(&bar[RB_QEMPTY + qb], (t.m.k / X::NQ - 1) & 1);
      ok = __shfl_sync(FULL_MASK, ok, 0);
      if (!ok) {
        if (lane == 0) {
          set_err(a.err, PKV_DEV_TIMEOUT);
          sh.abort_flag = 1;
        }
        break;
      }
      const bool okb = lane < t.nblk && (unsigned)t.phys < (unsigned)a.num_blocks;
      const unsigned invalid = __ballot_sync(FULL_MASK, lane < t.nblk && !okb), valid = __ballot_sync(FULL_MASK, okb);
      uint8_t* st = sm + (kside ? slot * X::KST : X::V_OFF + slot * X::VST);
      if (lane == 0) {
        if (invalid && kside) set_err(a.err, PKV_DEV_BAD_BLOCK);
        t.m.invalid = (int)invalid;
        (kside ? sh.kmeta : vmeta)[slot] = t.m;
        if (kside && t.first) {
          uint8_t* qd = sm + X::Q_OFF + qb * X::QBUF;
          mbar_arrive_expect_tx(&bar[RB_QFULL + qb], (uint32_t)KC * 128u * (uint32_t)a.tile_rows);
          for (int ch = 0; ch < KC; ++ch) {
            if constexpr (X::SHARED) tma_load_3d(qd + ch * X::QCH, &tmq, ch * 64, t.m.q0 * a.n_h + t.m.row0, 0, &bar[RB_QFULL + qb], pol);
            else tma_load_3d(qd + ch * X::QCH, &tmq, ch * 64, t.m.g * a.G, t.m.q0 + t.m.row0 / a.G, &bar[RB_QFULL + qb], pol);
          }
          kq = t.m.k;
        }
        mbar_arrive_expect_tx(fullb, (uint32_t)__popc(valid) * (uint32_t)NC * BS * 128u);
      }
      __syncwarp();
      for (int j0 = 0; j0 < X::NBT * NC; j0 += 32) {          // lane: one box of 64 channels of one block
        const int j = j0 + lane, b = j / NC, ch = j - b * NC;
        const int pb = __shfl_sync(FULL_MASK, t.phys, b & 31);
        if (b < t.nblk && ((valid >> b) & 1))
          tma_load_3d(st + ch * X::CHUNK + b * BS * 128, kside ? &tmk : &tmv, ch * 64, t.m.g * BS, pb, fullb, pol);
      }
      if (!more) {
        ++i;
        break;
      }
      t = tn;
      more = more2;
    }
    // After a timeout: let the loads already issued land before the CTA leaves (bounded).
    if (sh.abort_flag && lane == 0) {
      bool live = true;
      for (int j = i - depth < 0 ? 0 : i - depth; j < i && live; ++j)
        live = mbar_wait(&bar[(kside ? RB_KFULL : VFULL) + j % depth], (j / depth) & 1);
      if (live && kside && kq >= 0) mbar_wait(&bar[RB_QFULL + kq % X::NQ], (kq / X::NQ) & 1);
    }
    __syncwarp();
  } else if (sh.any && warp == 1) {
    // ------------------------- first-product issuer -------------------------
    if (lane == 0) {
      constexpr uint32_t IQK = umma_idesc_bf16(TT, R, 0, 0);
      const uint32_t sbase = smem_u32(sm);
      bool ok = true;
      for (int i = 0;; ++i) {
        const int slot = i % NK, sb = i & 1;
        if (sh.abort_flag || !mbar_wait(&bar[RB_KFULL + slot], (i / NK) & 1)) {
          ok = false;
          break;
        }
        const int flags = sh.kmeta[slot].flags, k = sh.kmeta[slot].k, qb = k % X::NQ;
        if (((flags & F_FIRST) && !mbar_wait(&bar[RB_QFULL + qb], (k / X::NQ) & 1)) ||
            (i >= 2 && !mbar_wait(&bar[RB_SEMPTY + sb], ((i >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t kb = sbase + slot * X::KST, qa = sbase + X::Q_OFF + qb * X::QBUF;
#pragma unroll 4
        for (int ks = 0; ks < KC * 4; ++ks) {
          const uint64_t ad = umma_desc(kb + (ks >> 2) * X::CHUNK + (ks & 3) * 32, 16, 1024, kLayoutSw128);
          const uint64_t bd = umma_desc(qa + (ks >> 2) * X::QCH + (ks & 3) * 32, 16, 1024, kLayoutSw128);
          umma_bf16(tmem + X::S_COL + R * sb, ad, bd, IQK, ks > 0 ? 1u : 0u);
        }
        umma_commit(&bar[RB_SFULL + sb]);
        if (!X::SHARED) umma_commit(&bar[RB_KEMPTY + slot]);
        if (flags & F_LAST) umma_commit(&bar[RB_QEMPTY + qb]);
        if (flags & F_END) break;
      }
      if (!ok) {
        set_err(a.err, PKV_DEV_TIMEOUT);
        sh.abort_flag = 1;
      }
      // every product issued has completed before the tensor memory is released
      umma_commit(&bar[RB_DRAIN]);
      mbar_wait(&bar[RB_DRAIN], 0);
    }
    __syncwarp();
  } else if (sh.any && warp == 2) {
    // ------------------------- second-product issuer ------------------------
    if (lane == 0) {
      constexpr uint32_t IPV = umma_idesc_bf16(X::VM, N2, 1, 1);
      const uint32_t sbase = smem_u32(sm);
      bool ok = true;
      for (int i = 0;; ++i) {
        const int slot = i % NV, pb = i % X::NP;
        if (sh.abort_flag || !mbar_wait(&bar[VFULL + slot], (i / NV) & 1) || !mbar_wait(&bar[RB_PFULL + pb], (i / X::NP) & 1)) {
          ok = false;
          break;
        }
        const RowsMeta& mt = vmeta[slot];
        const int flags = mt.flags, k = mt.k, ob = k % X::NO, nks = (min(TT, mt.ctx - mt.tile0) + 15) >> 4;
        if ((flags & F_FIRST) && k >= X::NO && !mbar_wait(&bar[RB_OEMPTY + ob], (k / X::NO - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t vb = sbase + (X::SHARED ? slot * X::KST : X::V_OFF + slot * X::VST), pa = sbase + X::P_OFF + pb * X::PBUF;
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          for (int kk = 0; kk < nks; ++kk) {
            const uint64_t ad = umma_desc(vb + vt * (X::VM / 64) * X::CHUNK + kk * 2048, X::CHUNK, 1024, kLayoutSw128);
            const uint64_t bd = umma_desc(pa + kk * 2048, X::CHUNK, 1024, kLayoutSw128);
            umma_bf16(tmem + (ob * VT + vt) * N2, ad, bd, IPV, (flags & F_FIRST) && kk == 0 ? 0u : 1u);
          }
        }
        umma_commit(&bar[VEMPTY + slot]);
        umma_commit(&bar[RB_PEMPTY + pb]);
        if (flags & F_LAST) umma_commit(&bar[RB_OFULL + ob]);
        if (flags & F_END) break;
      }
      if (!ok) {
        set_err(a.err, PKV_DEV_TIMEOUT);
        sh.abort_flag = 1;
      }
      umma_commit(&bar[RB_DRAIN_PV]);
      mbar_wait(&bar[RB_DRAIN_PV], 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // Sequences without cached rows: their tokens' outputs are zeros
    for (int s = blockIdx.x; s < a.batch; s += gridDim.x) {
      int flags = 0;
      const Drafts d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, s, flags);
      if (d.ctx > 0 || d.n == 0) continue;
      const long long at = (long long)d.q0 * a.n_h * DV, len = (long long)d.n * a.n_h * DV;
      for (long long e = threadIdx.x - 128; e < len; e += 256) store_out(a, at + e, 0.f);
    }
    // -------------------------- softmax and epilogue ------------------------
    // Group gi takes query rows [hb, hb + R / 2).  Warp w reaches the tensor-memory lanes of quarter w % 4: in
    // S^T the cached rows 16 MT wq + ..., in fragments of 16 rows x 8 query rows, in O^T the channels 32 wq + lane.
    constexpr int RG = R / 2, KB = RG / 8;                    // query rows of a group, fragments
    const int wq = warp & 3, gi = (warp - 4) >> 2, hb = RG * gi;
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    float m[2 * KB], l[2 * KB];                               // offsets and this thread's rows' share of the sums, of its query rows
    // A failed (timed-out) wait makes `bad` true for the whole warp; both groups learn of it at the vote that
    // opens each tile and leave together, so no thread is left at a named barrier.
    bool bad = false;
    int i = 0;
    for (; sh.any;) {
      const int slot = i % NV, sb = i & 1, pb = i % X::NP;
      bool okw = !bad && !sh.abort_flag && mbar_wait(&bar[VFULL + slot], (i / NV) & 1) && mbar_wait(&bar[RB_SFULL + sb], (i >> 1) & 1);
      okw = __all_sync(FULL_MASK, okw);
      if (named_bar_or(1, 256, !okw)) {
        bad = true;
        break;
      }
      const RowsMeta mt = vmeta[slot];
      const int flags = mt.flags, ob = mt.k % X::NO, nrows = min(TT, mt.ctx - mt.tile0);
      const bool special = mt.tile0 + TT > mt.ctx - mt.n || mt.invalid;
      tc_fence_after();
      float x[MT][KB][4];
      {
        uint32_t sr[MT][4 * KB];
#pragma unroll
        for (int j = 0; j < MT; ++j) tmem_ld_frag(tmem + lane_off + ((uint32_t)(16 * j) << 16) + X::S_COL + R * sb + hb, sr[j]);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][b][e] = __uint_as_float(sr[j][4 * b + e]) * a.scale_log2;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[RB_SEMPTY + sb]);       // S buffer sb may be rewritten
      if (flags & F_FIRST) {
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) {
          m[b] = -INFINITY;
          l[b] = 0.f;
        }
      }
      const int r0 = 16 * MT * wq + (lane >> 2), c0 = hb + 2 * (lane & 3);   // this thread's first cached row and query row
      if (special) {
        // what each query row attends to in this tile, and what any of them does
        const int tid = threadIdx.x - 128;
        if (tid < 2) sh.seen[tid] = 0;
        named_bar(6, 256);
        if (tid < R * MT) {
          const int c = tid % R, w = tid / R, r = mt.row0 + c;
          unsigned long long win = 0;
          if (c < a.tile_rows && r < mt.n * a.G) win = attended(a, mt, r / a.G, mt.tile0 + 64 * w);
          for (int b = 0; b < 64 / BS; ++b)
            if ((mt.invalid >> (w * (64 / BS) + b)) & 1) win &= ~(ones_below(BS) << (b * BS));
          sh.win[w * R + c] = win;
          atomicOr(&sh.seen[w], win);
        }
        named_bar(6, 256);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = r0 + 16 * j + 8 * (e >> 1), c = c0 + 8 * b + (e & 1);
              if (!((sh.win[(row >> 6) * R + c] >> (row & 63)) & 1)) x[j][b][e] = -INFINITY;
            }
      }
      bool over = false;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) over |= x[j][b][e] > m[2 * b + (e & 1)] + kLazyMax;
      if (named_bar_or(2 + gi, 128, over)) {
        // raise the group's offsets to the running max
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) {
          float v = -INFINITY;
#pragma unroll
          for (int j = 0; j < MT; ++j) v = fmaxf(v, fmaxf(x[j][b >> 1][b & 1], x[j][b >> 1][2 + (b & 1)]));
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, o));
          if (lane < 4) sh.red[wq * R + c0 + 8 * (b >> 1) + (b & 1)] = v;
        }
        named_bar(4 + gi, 128);
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) {
          const int c = c0 + 8 * (b >> 1) + (b & 1);
          const float mx = fmaxf(fmaxf(sh.red[c], sh.red[R + c]), fmaxf(sh.red[2 * R + c], sh.red[3 * R + c]));
          const float mn = fmaxf(m[b], mx), al = m[b] == -INFINITY ? 0.f : ex2(m[b] - mn);
          m[b] = mn;
          l[b] *= al;
          if (wq == 0 && lane < 4) sh.factor[c] = al;
        }
        named_bar(4 + gi, 128);
        if (!(flags & F_FIRST)) {
          // O accumulated so far: wait for the previous tile's products, then scale the group's columns in place
          bad |= !__all_sync(FULL_MASK, mbar_wait(&bar[RB_PEMPTY + (i - 1) % X::NP], ((i - 1) / X::NP) & 1));
          if (!bad) {
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < VT * HL; ++q) {
#pragma unroll 1
              for (int b = 0; b < KB; ++b) {
                const uint32_t ta = tmem + lane_off + (ob * VT + q / HL) * N2 + (q % HL) * R + hb + 8 * b;
                uint32_t o[8];
                tmem_ld8(ta, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sh.factor[hb + 8 * b + e]);
                tmem_st8(ta, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
      }
      // the P buffer is free once the products that read it last have completed
      if (i >= X::NP) bad |= !__all_sync(FULL_MASK, mbar_wait(&bar[RB_PEMPTY + pb], (i / X::NP - 1) & 1));
      // Row t of the B operand: 128 bytes per 64 columns (high parts of the query rows, then low parts), 16-byte
      // chunk c stored at chunk c ^ (t % 8) (128-byte swizzle).
      uint8_t* pbuf = sm + X::P_OFF + pb * X::PBUF;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = r0 + 16 * j + 8 * h;
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float off = m[2 * b + e] == -INFINITY ? 0.f : m[2 * b + e];
              p[e] = ex2(x[j][b][2 * h + e] - off);
            }
            const uint32_t hi = pack_bf16(p[0], p[1]);
            if constexpr (HL == 1) {                          // the sums take the rounded weights, which the products take
              p[0] = bf16_lo(hi);
              p[1] = bf16_hi(hi);
            }
            l[2 * b] += p[0];
            l[2 * b + 1] += p[1];
            if (!bad) {
              uint8_t* prow = pbuf + row * 128 + 4 * (lane & 3);
              const int ch = (hb >> 3) + b;
              *reinterpret_cast<uint32_t*>(prow + ((ch ^ (row & 7)) << 4)) = hi;
              if constexpr (HL == 2) {
                const uint32_t lo = pack_bf16(p[0] - bf16_lo(hi), p[1] - bf16_hi(hi));
                const int cl = R / 8 + ch;
                *reinterpret_cast<uint32_t*>(prow + (cl >> 3) * X::CHUNK + (((cl & 7) ^ (row & 7)) << 4)) = lo;
              }
            }
          }
      if (special && !bad) {
        // V rows that no query row attends to, and that the product reads with p = 0: they may hold anything
        uint8_t* vst = sm + (X::SHARED ? slot * X::KST : X::V_OFF + slot * X::VST);
        const int top = (nrows + 15) & ~15;
        for (int row = warp - 4; row < top; row += 8)
          if (!((sh.seen[row >> 6] >> (row & 63)) & 1))
            for (int v = lane; v < X::VC * 8; v += 32) *reinterpret_cast<uint4*>(vst + (v >> 3) * X::CHUNK + row * 128 + (v & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();          // the rows written above, for the tensor core
      __syncwarp();
      if (lane == 0 && !bad) mbar_arrive(&bar[RB_PFULL + pb]);

      if (flags & F_LAST) {
        // the segment's sums over all cached rows, and the output rows of its query rows
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) {
          float v = l[b];
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
          if (lane < 4) sh.red[wq * R + c0 + 8 * (b >> 1) + (b & 1)] = v;
          if (wq == 0 && lane < 4) sh.offset(c0 + 8 * (b >> 1) + (b & 1)) = m[b];
        }
        if (wq == 1 && lane < RG) sh.row(hb + lane) = (int)out_row(a, mt.q0, mt.n, mt.g, mt.row0, hb + lane);
        named_bar(4 + gi, 128);
        const bool whole = flags & F_WHOLE;
        if (wq == 0 && lane < RG) {
          const int c = hb + lane;
          const float s = (sh.red[c] + sh.red[R + c]) + (sh.red[2 * R + c] + sh.red[3 * R + c]);
          sh.factor[c] = whole ? sum_inverse(s) : 1.f;
          if (!whole) *reinterpret_cast<float2*>(a.ws_ml + ((size_t)mt.part * R + c) * 2) = make_float2(sh.offset(c), s);
        }
        named_bar(4 + gi, 128);
        bad |= !__all_sync(FULL_MASK, !bad && mbar_wait(&bar[RB_OFULL + ob], (mt.k / X::NO) & 1));
        if (!bad) {
          tc_fence_after();
#pragma unroll 1
          for (int vt = 0; vt < VT; ++vt) {
            const int chn = vt * X::VM + (X::VM == 128 ? 32 * wq + lane : 16 * wq + lane);
            const bool mine = X::VM == 128 || lane < 16;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
              uint32_t t0[8], t1[8];
              const uint32_t oc = tmem + lane_off + (ob * VT + vt) * N2 + hb + 8 * b;
              tmem_ld8(oc, t0);
              if constexpr (HL == 2) tmem_ld8(oc + R, t1);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int c = hb + 8 * b + e, row = sh.row(c);
                float v = __uint_as_float(t0[e]);
                if constexpr (HL == 2) v += __uint_as_float(t1[e]);
                v *= sh.factor[c];
                if (row < 0 || !mine) continue;
                if (whole) store_out(a, (long long)row * DV + chn, v);
                else a.ws_o[((size_t)mt.part * R + c) * DV + chn] = v;
              }
            }
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0 && !bad) mbar_arrive(&bar[RB_OEMPTY + ob]);
        named_bar(4 + gi, 128);            // sums and rows are read before the next segment's
      }
      if (flags & F_END) break;
      ++i;
    }
    if (bad && lane == 0) {
      set_err(a.err, PKV_DEV_TIMEOUT);
      sh.abort_flag = 1;
    }
  }
  // the tensor memory is released once every role is done with it (the issuers waited for their last products)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, X::TMEM_COLS);
}

// ---- parts of cut segments ----------------------------------------------------------------------------
// A CTA per (boundary, member, 8 query rows, 128 channels): a warp per query row joins the parts of its segment.
template <int R, int DV>
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int CB = DV < 128 ? DV : 128, V = CB / 32;        // channels of a CTA, of a lane
  grid_dep_wait();
  grid_dep_launch();
  const int team = blockIdx.x / a.C, member = blockIdx.x % a.C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowsCut cut = a.cuts[team];
  if (cut.parts == 0) return;
  const int c = blockIdx.y * 8 + warp, row0 = (cut.rg * a.C + member) * a.tile_rows;
  const long long row = out_row(a, cut.q0, cut.n, cut.g, row0, c);
  if (row < 0) return;
  auto part = [&](int p) { return (size_t)(((team - 1 + p) * a.C + member) * 2 + (p == 0 ? cut.first : 0)) * R + c; };
  float M = -INFINITY;
  for (int p = lane; p < cut.parts; p += 32) M = fmaxf(M, a.ws_ml[2 * part(p)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
  if (M == -INFINITY) M = 0.f;
  float L = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  const int ch = blockIdx.z * CB + lane * V;
#pragma unroll 8
  for (int p = 0; p < cut.parts; ++p) {
    const size_t at = part(p);
    const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + 2 * at);
    const float w = ex2(ml.x - M);
    L += w * ml.y;
    if constexpr (V == 4) {
      const float4 o = *reinterpret_cast<const float4*>(a.ws_o + at * DV + ch);
      acc[0] += w * o.x; acc[1] += w * o.y; acc[2] += w * o.z; acc[3] += w * o.w;
    } else {
      const float2 o = *reinterpret_cast<const float2*>(a.ws_o + at * DV + ch);
      acc[0] += w * o.x; acc[1] += w * o.y;
    }
  }
  const float inv = sum_inverse(L);
#pragma unroll
  for (int v = 0; v < V; ++v) store_out(a, row * DV + ch + v, acc[v] * inv);
}

// ---- variants ----------------------------------------------------------------------------------------
struct RowsVariant {
  const void *fn, *join;
  size_t smem;
  int R, DV;
  bool ready[64];
};

template <class X>
static RowsVariant make_variant() {
  constexpr size_t smem = X::M_OFF + sizeof(RowsShared<X>);
  static_assert(smem <= 232448, "shared memory of one CTA");
  static_assert(X::Q_OFF % 1024 == 0 && X::P_OFF % 1024 == 0 && X::NCOL <= 512, "descriptor alignment, tensor memory");
  return {(const void*)decode_rows_kernel<X>, (const void*)rows_join_kernel<X::R, X::DV>, smem, X::R, X::DV, {}};
}
template <int BS>
static RowsVariant* kv_variant(int d, int R) {
  static RowsVariant v[2][3] = {
      {make_variant<RowsCfg<BS, 1, 1, 64, false, 16, 2>>(), make_variant<RowsCfg<BS, 1, 1, 64, false, 32, 2>>(),
       make_variant<RowsCfg<BS, 1, 1, 64, false, 64, 2>>()},
      {make_variant<RowsCfg<BS, 2, 1, 128, false, 16, 2>>(), make_variant<RowsCfg<BS, 2, 1, 128, false, 32, 2>>(),
       make_variant<RowsCfg<BS, 2, 1, 128, false, 64, 2>>()}};
  return &v[d == 128][R == 16 ? 0 : (R == 32 ? 1 : 2)];
}
template <int BS>
static RowsVariant* latent_variant(int latent, int R) {
  static RowsVariant v[2][3] = {
      {make_variant<RowsCfg<BS, 5, 2, 128, true, 16, 2>>(), make_variant<RowsCfg<BS, 5, 2, 128, true, 32, 2>>(),
       make_variant<RowsCfg<BS, 5, 2, 128, true, 64, 1>>()},
      {make_variant<RowsCfg<BS, 9, 4, 128, true, 16, 2>>(), make_variant<RowsCfg<BS, 9, 4, 128, true, 32, 2>>(),
       make_variant<RowsCfg<BS, 9, 4, 128, true, 64, 1>>()}};
  return &v[latent == 512][R == 16 ? 0 : (R == 32 ? 1 : 2)];
}

// Query rows of a row tile, and members of a team, from the average of the sequences' query rows per kv head.
struct RowsShape {
  int R, C, P;
};
static RowsShape rows_shape(int n_tok, int batch, int G, int most) {
  const long long rows = ((long long)n_tok * G + batch - 1) / batch;
  RowsShape s;
  s.R = rows <= 16 && G <= 16 ? 16 : (rows <= 32 && G <= 32 ? 32 : 64);
  if (s.R > most) s.R = most;
  const long long tiles = (rows + s.R - 1) / s.R;
  s.C = tiles <= 1 ? 1 : (tiles <= 2 ? 2 : 4);
  const int sms = device_sm_count();
  s.P = sms / s.C;
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
  a.n_each = q_start ? 0 : n_tok / batch;
  a.tile_rows = latent ? s.R : s.R / a.G * a.G;
  a.C = s.C; a.P = s.P;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_dtype == PKV_OUT_F32;
  a.err = err;
  a.cuts = static_cast<RowsCut*>(ws);
  a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.ml);
  a.ws_o = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.o);

  CUtensorMap tmk, tmv, tmq;
  const uint64_t row = (uint64_t)w * 2, rows = (uint64_t)n_kv * block_size, nblk = num_blocks > 0 ? (uint64_t)num_blocks : 1;
  int bad = encode_tensor_map_3d(&tmk, k, w, rows, nblk, row, rows * row, 64, block_size);
  if (latent) {
    tmv = tmk;
    bad |= encode_tensor_map_3d(&tmq, q, w, (uint64_t)n_tok * n_h, 1, row, row, 64, s.R);
  } else {
    bad |= encode_tensor_map_3d(&tmv, vp, w, rows, nblk, row, rows * row, 64, block_size);
    bad |= encode_tensor_map_3d(&tmq, q, w, n_h, n_tok, row, n_h * row, 64, a.G, s.R / a.G);
  }
  if (bad) return PKV_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* kargs[] = {&tmk, &tmv, &tmq, &a};
  cudaError_t e = launch_pdl(v->fn, dim3(s.P * s.C), dim3(384), v->smem, st, kargs);
  if (e == cudaSuccess) {
    void* jargs[] = {&a};
    e = launch_pdl(v->join, dim3(s.P * s.C, s.R / 8, v->DV < 128 ? 1 : v->DV / 128), dim3(256), 0, st, jargs);
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
  const RowsShape s = rows_shape(n_tok, batch, n_h / n_kv, 64);
  return s.P < 1 ? 0 : rows_layout(s, head_dim).total;
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
  const RowsShape s = rows_shape(n_tok, batch, n_h / n_kv, 64);
  RowsVariant* v = block_size == 16 ? kv_variant<16>(head_dim, s.R) : (block_size == 32 ? kv_variant<32>(head_dim, s.R) : kv_variant<64>(head_dim, s.R));
  return rows_attn(s, v, false, q, k_pool, v_pool, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words, scale,
                   n_tok, batch, n_h, n_kv, head_dim, block_size, num_blocks, out, out_dtype, workspace, workspace_bytes, err_flag,
                   stream);
}

// fp32 outputs take p in two parts, which for 64 query rows would not fit the tensor memory: 32 at most.
static RowsShape latent_shape(int n_tok, int batch, int n_h, bool f32) { return rows_shape(n_tok, batch, n_h, f32 ? 32 : 64); }

extern "C" size_t pkv_latent_workspace_bytes(int batch, int n_tok, int n_h, int latent, int rope, int block_size) {
  if (batch < 0 || n_tok < 0 || !valid_latent(n_h, latent, rope, block_size)) return 0;
  if (batch == 0 || n_tok == 0) return 256;
  const RowsShape a = latent_shape(n_tok, batch, n_h, false), b = latent_shape(n_tok, batch, n_h, true);
  if (a.P < 1 || b.P < 1) return 0;
  const size_t x = rows_layout(a, latent).total, y = rows_layout(b, latent).total;
  return x > y ? x : y;
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
  const RowsShape s = latent_shape(n_tok, batch, n_h, out_dtype == PKV_OUT_F32);
  RowsVariant* v = block_size == 16 ? latent_variant<16>(latent, s.R) : (block_size == 32 ? latent_variant<32>(latent, s.R) : latent_variant<64>(latent, s.R));
  return rows_attn(s, v, true, q, cache, cache, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words, scale, n_tok,
                   batch, n_h, 1, latent + rope, block_size, num_blocks, out, out_dtype, workspace, workspace_bytes, err_flag, stream);
}
