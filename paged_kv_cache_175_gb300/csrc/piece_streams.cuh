// Streams of the attention kernels decode_q8.cu and decode_mass.cu.
//
// A CTA holds NW streams: stream w takes piece blockIdx.x * NW + w of the line of blocks
// (decode_common.cuh) and has a ring of S stages of its own, read by MT consumer warps.  One
// producer warp serves all of them, lane w driving stream w: it walks the stream's piece, reads
// the block-table entries one stage ahead and issues the copies.  The lanes run in step, so a
// stage costs the SM about as many producer instructions for six streams as for one, and only one
// warp's registers are spent on producing.  (With a producer warp per consumer warp half of the
// register file held producers: six or eight consumers per SM at 128 registers, against twelve.)
//
// The unit of the line here is a block of bs = 16 or 32 tokens; a table block of 64 tokens counts
// as two units of 32 (unit u lies in table entry u >> sub).
#pragma once

#include "decode_common.cuh"

namespace pkv {

// Whether the barrier's phase of this parity is over; does not suspend the thread, so a lane whose
// ring is full does not hold up the others.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

struct StreamStart {
  Cursor cur;
  long long pstart, pend;
  int len;                       // units of the stream's piece (0: none)
};

// Called by one whole warp per stream.
__device__ __forceinline__ void stream_setup(const DecodeArgs& a, int piece, int pieces, StreamStart* out) {
  Cursor cur = {};
  PieceInfo pi = {};
  piece_setup(a, piece, pieces, true, cur, pi);
  const int len = piece < pi.P ? (int)(pi.pend - pi.pstart) : 0;
  if ((threadIdx.x & 31) == 0) {
    out->cur = cur;
    out->pstart = pi.pstart;
    out->pend = pi.pend;
    out->len = len;
  }
}

// The producer warp, lanes 0..NW-1 driving one stream each.  nb: units per stage (1 or 2); meta,
// full, empty: [NW][S].  copy(stream, slot, k, phys, u, g) brings unit k of a stage (unit u of its
// sequence, in pool block phys): unit_bytes bytes that complete on full[stream][slot].  A block id
// outside the pool becomes a stage of its own without F_VALID and without copies.  Consumers
// arrive on empty[stream][slot] once a stage is read.
template <class Copy>
__device__ __forceinline__ void produce_streams(const DecodeArgs& a, const StreamStart* starts, int NW, int S, int nb,
                                                int sub, uint32_t unit_bytes, int q_row_bytes, int4* meta, uint64_t* full,
                                                uint64_t* empty, volatile int* abort_flag, Copy copy) {
  const int lane = threadIdx.x & 31, BS = a.block_size;
  StreamStart st = {};
  if (lane < NW) st = starts[lane];
  Cursor cur = st.cur;
  meta += lane * S;
  full += lane * S;
  empty += lane * S;
  int slot = 0, issued = 0, pj = 0, e0 = -1, e1 = -1;
  uint32_t phase = 0;
  auto entries = [&]() {                                       // of the next stage, used a round later
    const int32_t* row = a.bt + (size_t)cur.s * a.max_blocks;
    const int u = cur.b0 + cur.blk;
    e0 = __ldg(row + (u >> sub));
    e1 = nb > 1 && cur.blk + 1 < cur.nb ? __ldg(row + ((u + 1) >> sub)) : -1;
  };
  if (st.len > 0) entries();
  uint32_t spins = 0;
  uint64_t t0 = 0;
  while (__any_sync(FULL_MASK, pj < st.len) && !__any_sync(FULL_MASK, *abort_flag != 0)) {
    bool ready = false;
    if (pj < st.len) ready = issued < S || mbar_test(&empty[slot], phase ^ 1u);   // released in the previous pass
    if (ready) {
      const int most = min(min(nb, cur.nb - cur.blk), st.len - pj);
      const bool ok = (unsigned)e0 < (unsigned)a.num_blocks;
      const int nblk = ok && most > 1 && (unsigned)e1 < (unsigned)a.num_blocks ? 2 : 1;
      const int lb = cur.blk + nblk - 1;                       // the stage's last unit
      const int ntok = (nblk - 1) * BS + (lb == cur.nb - 1 ? cur.ctx - (cur.b0 + lb) * BS : BS);
      const int lead = cur.blk == 0 ? window_lead(cur.ctx, a.window, BS) : 0;
      const bool end = pj + nblk >= st.len;
      int flags = 0;
      if (pj == 0 || cur.blk == 0) flags |= F_FIRST;
      if (end || lb == cur.nb - 1) flags |= F_LAST;
      if (cur.seg_start >= st.pstart && cur.seg_start + cur.nb <= st.pend) flags |= F_WHOLE;
      if (end) flags |= F_END;
      if (ok) flags |= F_VALID; else set_err(a.err, PKV_DEV_BAD_BLOCK);
      meta[slot] = make_int4(cur.s, cur.g, cur.blk, pack_rows(ntok, lead, flags));
      if (ok) {
        mbar_arrive_expect_tx(&full[slot], (uint32_t)nblk * unit_bytes);
        copy(lane, slot, 0, e0, cur.b0 + cur.blk, cur.g);
        if (nblk > 1) copy(lane, slot, 1, e1, cur.b0 + cur.blk + 1, cur.g);
      } else {
        mbar_arrive(&full[slot]);
      }
      if (flags & F_FIRST) {                                   // warm L2 with the group's queries
        const size_t row = (size_t)a.G * q_row_bytes;
        const char* qp = reinterpret_cast<const char*>(a.q) + ((size_t)cur.s * a.n_kv + cur.g) * row;
        for (size_t off = 0; off < row; off += 128) prefetch_l2(qp + off);
      }
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
      ++issued;
      pj += nblk;
      cur.blk += nblk - 1;
      if (pj < st.len) {
        cursor_next(cur, a);
        entries();
      }
      spins = 0;
    } else if (pj < st.len && (++spins & 1023u) == 0) {        // bounded like mbar_wait: about two seconds
      const uint64_t now = global_timer_ns();
      if (spins == 1024u) t0 = now;
      if (now - t0 > 2000000000ull || spins > (1u << 30)) {
        set_err(a.err, PKV_DEV_TIMEOUT);
        *abort_flag = 1;
      }
    }
    __syncwarp();
  }
  if (*abort_flag) {
    // let the copies still in flight land before the CTA exits: wait (bounded) for the last
    // stage issued on each slot
    for (int k = 0; k < S && k < issued; ++k) {
      const int last = k + ((issued - 1 - k) / S) * S;
      if (!mbar_wait(&full[k], (last / S) & 1)) break;
    }
  }
}

}  // namespace pkv
