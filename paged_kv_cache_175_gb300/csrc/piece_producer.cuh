// The producer warp of the attention kernels whose ring stages hold several consecutive blocks
// of a segment (decode_q8.cu, decode_mass.cu).
#pragma once

#include "decode_common.cuh"

namespace pkv {

// Streams the CTA's piece (len blocks from cursor cur) into a ring of S stages of up to nb
// blocks: per stage the rows and flags go to meta[slot] and lane k calls copy(slot, k, phys, g)
// for the stage's block k, which is to bring block_bytes bytes that complete on full[slot].
// A block id outside the pool becomes a stage of its own without F_VALID and without copies.
// Called by one whole warp; consumers arrive on empty[slot] once a stage is read.
template <class Copy>
__device__ __forceinline__ void produce_piece(const DecodeArgs& a, Cursor& cur, const PieceInfo& pi, int len, int bs16l,
                                              int nb, int S, uint32_t block_bytes, int q_row_bytes, int4* meta,
                                              uint64_t* full, uint64_t* empty, volatile int* abort_flag, Copy copy) {
  const int lane = threadIdx.x & 31, BS = 16 << bs16l;
  int w_seq = -1, w_base = 0, w_phys = -1, n_seq = -1, n_base = 0, n_phys = -1;   // windows of 32 table entries
  int slot = 0, issued = 0, pj = 0;
  uint32_t phase = 0;
  while (pj < len && !__any_sync(FULL_MASK, *abort_flag != 0)) {   // one answer for the warp
    if (cur.s != w_seq || cur.blk < w_base || cur.blk >= w_base + 32) {
      if (cur.s == n_seq && cur.blk >= n_base && cur.blk < n_base + 32) {
        w_seq = n_seq; w_base = n_base; w_phys = n_phys;
      } else {
        w_seq = cur.s; w_base = cur.blk;
        const int b = w_base + lane;
        w_phys = b < cur.nb ? __ldg(a.bt + (size_t)cur.s * a.max_blocks + cur.b0 + b) : -1;
      }
      n_seq = cur.s;
      n_base = w_base + 32 < cur.nb ? w_base + 32 : 0;
      const int b = n_base + lane;
      n_phys = b < cur.nb ? __ldg(a.bt + (size_t)cur.s * a.max_blocks + cur.b0 + b) : -1;
    }
    // lane k's block of the stage: the entry is in this window or, past its end, in the
    // prefetched one (which then starts at w_base + 32, as the block is in the segment)
    const int most = min(min(nb, cur.nb - cur.blk), len - pj);
    const int b = cur.blk + lane;
    const int x = __shfl_sync(FULL_MASK, w_phys, (b - w_base) & 31);
    const int y = __shfl_sync(FULL_MASK, n_phys, (b - n_base) & 31);
    const int phys = b < w_base + 32 ? x : y;
    const unsigned bad = __ballot_sync(FULL_MASK, lane < most && (unsigned)phys >= (unsigned)a.num_blocks);
    const bool ok = !(bad & 1u);
    const int nblk = !ok ? 1 : (bad ? __ffs(bad) - 1 : most);
    bool go = true;
    if (lane == 0) {
      if (issued >= S && !mbar_wait(&empty[slot], phase ^ 1u)) {   // released in the previous pass
        set_err(a.err, PKV_DEV_TIMEOUT);
        *abort_flag = 1;
        go = false;
      }
      const int lb = cur.blk + nblk - 1;                       // the stage's last block
      const int ntok = (nblk - 1) * BS + (lb == cur.nb - 1 ? cur.ctx - (cur.b0 + lb) * BS : BS);
      const int lead = cur.blk == 0 ? window_lead(cur.ctx, a.window, BS) : 0;
      const bool end = pj + nblk >= len;
      int flags = 0;
      if (pj == 0 || cur.blk == 0) flags |= F_FIRST;
      if (end || lb == cur.nb - 1) flags |= F_LAST;
      if (cur.seg_start >= pi.pstart && cur.seg_start + cur.nb <= pi.pend) flags |= F_WHOLE;
      if (end) flags |= F_END;
      if (ok) flags |= F_VALID; else set_err(a.err, PKV_DEV_BAD_BLOCK);
      meta[slot] = make_int4(cur.s, cur.g, cur.blk, pack_rows(ntok, lead, flags));
      if (ok && go) mbar_arrive_expect_tx(&full[slot], (uint32_t)nblk * block_bytes);
      else mbar_arrive(&full[slot]);
      if (flags & F_FIRST) {                                   // warm L2 with the group's queries
        const size_t row = (size_t)a.G * q_row_bytes;
        const char* qp = reinterpret_cast<const char*>(a.q) + ((size_t)cur.s * a.n_kv + cur.g) * row;
        for (size_t off = 0; off < row; off += 128) prefetch_l2(qp + off);
      }
    }
    go = __shfl_sync(FULL_MASK, go, 0);
    if (ok && go && lane < nblk) copy(slot, lane, phys, cur.g);
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
    ++issued;
    pj += nblk;
    cur.blk += nblk - 1;
    if (pj < len) cursor_next(cur, a);
  }
  __syncwarp();
  if (*abort_flag && lane == 0) {
    // let the copies still in flight land before the CTA exits: wait (bounded) for the
    // last stage issued on each slot
    for (int k = 0; k < S && k < issued; ++k) {
      const int last = k + ((issued - 1 - k) / S) * S;
      if (!mbar_wait(&full[k], (last / S) & 1)) break;
    }
  }
}

}  // namespace pkv
