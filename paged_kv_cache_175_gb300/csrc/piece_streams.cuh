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
#include "stream_plan.cuh"

namespace pkv {

constexpr long long kStreamMaxCtx = 0x7fff0000;               // tokens of a table: token numbers stay in 32 bits

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

// The piece of one stream and its first cursor, called by one whole warp per stream: from the plan
// kernel's tables, or (up to kInlinePlanSeqs sequences) from the context lengths, 32 at a time with all
// loads issued before any is used.
__device__ __forceinline__ void stream_setup(const DecodeArgs& a, int piece, int pieces, StreamStart* out) {
  constexpr int MAXC = kInlinePlanSeqs / 32;
  const int lane = threadIdx.x & 31, chunks = a.inline_plan ? (a.batch + 31) / 32 : 0;
  int ctx[MAXC], incl[MAXC];                                   // units of a chunk's sequences, prefix sums
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    const int s = c * 32 + lane;
    ctx[c] = c < chunks && s < a.batch ? a.ctx_raw[s] : 0;
  }
  bool bad = false;
  long long units = 0;
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    if (c >= chunks) continue;
    bad |= ctx[c] < 0 || ctx[c] > a.max_ctx;
    ctx[c] = clamp_ctx(ctx[c], a.max_ctx);
    incl[c] = span_blocks(ctx[c], a.window, a.block_size);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL_MASK, incl[c], o);
      if (lane >= o) incl[c] += y;
    }
    units += __shfl_sync(FULL_MASK, incl[c], 31);
  }
  if (__any_sync(FULL_MASK, bad) && lane == 0 && blockIdx.x == 0 && threadIdx.x == 0) set_err(a.err, PKV_DEV_BAD_CTX);
  const long long W = (long long)a.n_kv * (a.inline_plan ? units : a.cum[a.batch]);
  const int P = stream_pieces(W, (long long)a.batch * a.n_kv, pieces);
  Cursor cur = {};
  const long long pstart = W * piece / P, pend = W * (piece + 1) / P;
  const int len = piece < P ? (int)(pend - pstart) : 0;
  if (len > 0 && !a.inline_plan) {
    cursor_from_table(cur, piece, pstart, a);
  } else if (len > 0) {
    long long before = 0;                                      // units of earlier chunks
    bool found = false;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      if (c >= chunks || found) continue;
      const int nb = span_blocks(ctx[c], a.window, a.block_size);
      const long long lo = (long long)a.n_kv * (before + incl[c] - nb);
      const unsigned hit = __ballot_sync(FULL_MASK, lo <= pstart && pstart < lo + (long long)a.n_kv * nb);
      if (hit) {
        const int src = __ffs(hit) - 1;
        cur.s = c * 32 + src;
        cur.nb = __shfl_sync(FULL_MASK, nb, src);
        cur.ctx = __shfl_sync(FULL_MASK, ctx[c], src);
        cur.b0 = window_first_block(cur.ctx, a.window, a.block_size);
        const long long off = pstart - __shfl_sync(FULL_MASK, lo, src);
        cur.g = (int)(off / cur.nb);
        cur.blk = (int)(off % cur.nb);
        cur.seg_start = pstart - cur.blk;
        found = true;
        continue;
      }
      before += __shfl_sync(FULL_MASK, incl[c], 31);
    }
  }
  if (lane == 0) {
    out->cur = cur;
    out->pstart = pstart;
    out->pend = pend;
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
    e0 = row[u >> sub];
    e1 = nb > 1 && cur.blk + 1 < cur.nb ? row[(u + 1) >> sub] : -1;
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
