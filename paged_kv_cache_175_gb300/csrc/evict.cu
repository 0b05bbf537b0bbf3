// Eviction from the bf16 cache by accumulated attention weight.
//
// Per (sequence, kv head) with n rows and a budget of K < n: the `recent` newest rows and, of
// the others, those with the largest accounts stay (equal accounts: lowest row first).  Kept rows
// below K stay where they are; the kept rows at or behind K move, in ascending order, into the
// rows below K that were dropped, in ascending order.  Attention does not depend on the order of
// the rows (keys carry their positions), and this moves the fewest rows and lets every move run
// in parallel, sources being at or behind K and destinations below it.  What is newest is known
// from the positions: rows below `kept` have theirs recorded, later rows follow `dropped`.
//
// Select kernel: a cluster of CTAs per (sequence, kv head), each thread holding the keys of R
// consecutive rows in registers (recent rows: the largest key; else the account's bits in an
// order-keeping form), so the accounts are read once, all loads of a thread in flight together.
// Three rounds over 11, 11 and 10 bits of the key build histograms in shared memory, sum them over
// the cluster through distributed shared memory and narrow the K-th largest key; one ordered scan
// then gives every hole and every mover its place in the list (two, when rows with the K-th key
// have to be told apart).  Rows too many for a cluster's registers (over 131072) are read again in
// every round.
// Move kernel: the listed rows of K and V, 16 bytes a lane, spread over the whole GPU.
//
// What bounds it: the select kernel, latency (two or three histogram rounds over a few KB to MB of
// accounts); the move kernel, HBM (4 d bytes read and written per moved row).
// Measured: 64 x 2.1-4K rows cut to 2048, 8 kv heads of 128, 82.6 us (16.7 of them the selection; the
// moves, 367 MB, at 82% of the copy rate); one sequence of 128K rows cut to 32K 58.4 us (23.8; 203 MB at 87%);
// small calls 8.
// Having the move kernel write the movers' accounts and positions, too, from lists took 2 us more in both.
#include <cooperative_groups.h>

#include <cmath>

#include "decode_common.cuh"
#include "nvtx_range.h"

namespace cg = cooperative_groups;

namespace pkv {

struct EvictArgs {
  const float* mass;             // [batch][n_kv] rows of `stride`
  const int32_t* positions;
  const int32_t *kept, *dropped; // [batch]
  float* mass_out;
  int32_t* positions_out;
  int32_t *kept_out, *dropped_out, *new_lens;
  const int32_t *ctx, *keep;
  const int32_t* bt;
  long long stride;
  int batch, n_kv, max_blocks, max_ctx, bs_log2, recent, num_blocks;
  int* counts;                   // workspace: [batch * n_kv] rows to move
  int32_t *dst, *src;            // workspace: [batch * n_kv][max_ctx / 2 + 1]: rows of the moves
  int max_moves;
  uint4 *k_pool, *v_pool;
  int32_t* err;
  int in_place, vec;
};

constexpr int kEvBins = 2048;
constexpr long long kEvMaxRows = 0x7fff0000;                  // row numbers plus a grid's threads stay in 32 bits

// Order-keeping bits of an account: -0 below +0, NaN above everything but the recent rows.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix sum of x over the CTA's threads, in thread order; total gets the sum.
template <int NT, class T>
__device__ __forceinline__ T cta_scan(T x, T* warp_s, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(FULL_MASK, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                                            // warp_s may still be read from the last scan
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  // lane w holds warp w's sum; the warps before this one add up by a masked reduction
  const T v = lane < NT / 32 ? warp_s[lane] : 0;
  T before = lane < warp ? v : 0, all = v;
#pragma unroll
  for (int o = 16; o; o >>= 1) {                              // over the whole warp: every lane gets the sums
    before += __shfl_xor_sync(FULL_MASK, before, o);
    all += __shfl_xor_sync(FULL_MASK, all, o);
  }
  total = all;
  return before + incl - x;
}

template <bool SMALL> struct PairOf { using type = uint32_t; };
template <> struct PairOf<false> { using type = unsigned long long; };

// NT threads of R rows, R a multiple of 4 (0: any number, keys read again whenever they are used).
// CLUSTER: several CTAs may share a (sequence, kv head).
template <int NT, int R, bool CLUSTER>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_select_kernel(const EvictArgs a) {
  grid_dep_wait();                         // launched while the kernel before may still run
  grid_dep_launch();                       // the move kernel's launch overlaps; it waits for this grid
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CLUSTER ? (int)cluster.block_rank() : 0, ranks = CLUSTER ? (int)cluster.num_blocks() : 1;
  // with R > 0 a bin counts at most 16384 rows of the CTA: two bins to a word
  constexpr int kPack = R > 0 ? 1 : 0;
  __shared__ __align__(16) uint32_t hist[2][kEvBins >> kPack];
  // holes and movers travel together, a half of a word each: rows of a CTA fit 15 bits with R > 0
  using Pair = typename PairOf<(R > 0)>::type;
  constexpr int kHalf = 4 * sizeof(Pair);
  __shared__ Pair warp_s[NT / 32];
  __shared__ int sums_s[NT / 32];
  __shared__ Pair share[2];                                   // this CTA's counts, read by the cluster
  __shared__ int pick[3];
  __shared__ uint16_t stage[R > 0 ? NT * R : 1];
  const int sg = blockIdx.x / ranks, s = sg / a.n_kv;
  const int raw = a.ctx[s], n = clamp_ctx(raw, a.max_ctx);
  const int K = max(0, min(a.keep[s], n));
  const int kept = min(max(a.kept[s], 0), n), dropped = a.dropped[s];
  const float* mass = a.mass + (size_t)sg * a.stride;
  const int32_t* posn = a.positions + (size_t)sg * a.stride;
  float* mass_out = a.mass_out + (size_t)sg * a.stride;
  int32_t* pos_out = a.positions_out + (size_t)sg * a.stride;
  if (rank == 0 && sg % a.n_kv == 0 && threadIdx.x == 0) {
    if (raw != n) set_err(a.err, PKV_DEV_BAD_CTX);
    // here and not in the move kernel: an attention call behind this one may read the lengths
    // while the move kernel still runs
    a.new_lens[s] = K;
  }
  // this thread's rows
  const int each = R > 0 ? R : (n + ranks * NT - 1) / (ranks * NT);
  const int r0 = min((long long)n, (long long)(rank * NT + (int)threadIdx.x) * each), r1 = r0 + min(each, n - r0);

  if (K == n) {                                               // nothing to evict (uniform in the cluster)
    if (rank == 0 && threadIdx.x == 0) a.counts[sg] = 0;
    if (!a.in_place)
      for (int r = rank * NT + threadIdx.x; r < n; r += ranks * NT) {
        mass_out[r] = mass[r];
        if (r < kept) pos_out[r] = posn[r];
      }
    return;
  }
  // rows at or behind this position are recent: the newest token is dropped + n - 1
  const int recent_from = dropped + n - min(a.recent, K);
  auto position = [&](int r) { return r < kept ? posn[r] : dropped + r; };
  auto make_key = [&](int r) { return position(r) >= recent_from ? 0xffffffffu : order_bits(mass[r]); };
  uint32_t keys[R > 0 ? R : 1];
  if constexpr (R > 0) {
    if (r0 < r1) {                                            // warps behind the rows skip theirs throughout
      const bool vec = a.vec != 0;                            // rows of the state are 16-byte aligned
      float x[R];
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        if (vec && r0 + i + 4 <= r1) {
          const float4 v = *reinterpret_cast<const float4*>(mass + r0 + i);
          x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i + j] = r0 + i + j < r1 ? mass[r0 + i + j] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        int p[4];
        if (r0 + i >= kept) {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = dropped + r0 + i + j;
        } else if (vec && r0 + i + 4 <= min(r1, kept)) {
          const int4 v = *reinterpret_cast<const int4*>(posn + r0 + i);
          p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = r0 + i + j < r1 ? position(r0 + i + j) : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) keys[i + j] = p[j] >= recent_from ? 0xffffffffu : order_bits(x[i + j]);
      }
    }
  }
  // f(row, key) for this thread's rows in order
  auto rows = [&](auto f) {
    if constexpr (R > 0) {
      if (r1 - r0 == R) {
#pragma unroll
        for (int i = 0; i < R; ++i) f(r0 + i, keys[i]);
      } else if (r0 < r1) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (r0 + i < r1) f(r0 + i, keys[i]);
      }
    } else {
      for (int r = r0; r < r1; ++r) f(r, make_key(r));
    }
  };
  auto meet = [&]() {                                         // barrier of the cluster
    if (ranks == 1) __syncthreads();
    else cluster.sync();
  };

  // ---- the K-th largest key: 11 + 11 + 10 bits from the top ----
  uint32_t prefix = 0, mask = 0;
  int want = K;                                               // of the keys that match prefix, the wanted one's rank
  bool all_equal = true;                                      // every row with the K-th key is kept
  if (K > 0) {
    for (int b = threadIdx.x; b < 2 * (kEvBins >> kPack); b += NT) hist[0][b] = 0;
    __syncthreads();
#pragma unroll
    for (int round = 0; round < 3; ++round) {
      constexpr int kShift[3] = {21, 10, 0};
      const int shift = kShift[round], bins = round == 2 ? 1024 : 2048;
      uint32_t* h = hist[round & 1];
      rows([&](int, uint32_t k) {
        const uint32_t b = (k >> shift) & (bins - 1);
        if ((k & mask) == prefix) atomicAdd(&h[b >> kPack], kPack ? 1u << (16 * (b & 1)) : 1u);
      });
      meet();
      // buffer of the next round but one: its last readers passed the barrier above
      if (round == 1)
        for (int b = threadIdx.x; b < (1024 >> kPack); b += NT) hist[0][b] = 0;
      // CTA 0 of the cluster sums the histograms and finds the bin (every CTA reading all of them
      // took 14 us a round with 64 clusters of eight at work, 70 us in all against 38): warp w takes the w-th run of bins
      // from the top and lane l the l-th run of those; only the warp that holds the wanted rank looks
      // for its bin
      if (rank == 0) {
        constexpr int kRun[3] = {2048 / NT, 2048 / NT, 1024 / NT};
        const int nb = kRun[round], b0 = bins - nb * ((int)threadIdx.x + 1);
        int c[kRun[0]] = {};
        const int w0 = b0 >> kPack, nw = kPack ? (nb + 1) / 2 : nb;   // words of the run
        auto add = [&](int j, uint32_t v) {
          if (!kPack) c[j] += (int)v;
          else if (nb == 1) c[0] += (int)(v >> (16 * (b0 & 1)) & 0xffffu);
          else {
            c[2 * j] += (int)(v & 0xffffu);
            c[2 * j + 1] += (int)(v >> 16);
          }
        };
        if (ranks == 1) {
#pragma unroll
          for (int j = 0; j < nw; ++j) add(j, h[w0 + j]);
        } else {
          constexpr int kGroup = NT == 1024 ? 8 : 4;            // CTAs whose loads are in flight together
          for (int q0 = 0; q0 < ranks; q0 += kGroup) {
            uint32_t d[kGroup][kRun[0]];
#pragma unroll
            for (int q = 0; q < kGroup; ++q) {
              const uint32_t* hq = cluster.map_shared_rank(h, q0 + q < ranks ? q0 + q : 0);
#pragma unroll
              for (int j = 0; j < nw; ++j) d[q][j] = q0 + q < ranks ? hq[w0 + j] : 0u;
            }
#pragma unroll
            for (int q = 0; q < kGroup; ++q)
#pragma unroll
              for (int j = 0; j < nw; ++j) add(j, d[q][j]);
          }
        }
        int sum = 0;
#pragma unroll
        for (int j = 0; j < nb; ++j) sum += c[j];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int warp_sum = __reduce_add_sync(FULL_MASK, sum);
        if (lane == 0) sums_s[warp] = warp_sum;
        __syncthreads();
        const int ahead = __reduce_add_sync(FULL_MASK, lane < warp ? sums_s[lane] : 0);
        if (ahead < want && want <= ahead + warp_sum) {
          int incl = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += y;
          }
          int at = ahead + incl - sum;
#pragma unroll
          for (int j = nb - 1; j >= 0; --j) {
            if (at < want && want <= at + c[j]) {
              pick[0] = b0 + j;
              pick[1] = want - at;
              pick[2] = c[j];
            }
            at += c[j];
          }
        }
      }
      meet();
      const int* found = CLUSTER && ranks > 1 ? cluster.map_shared_rank(pick, 0) : pick;
      const int bin = found[0], rest = found[1], size = found[2];
      prefix |= (uint32_t)bin << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      want = rest;
      all_equal = rest == size;
      // the bin is kept as a whole: its lowest key, the prefix, divides the rows as the K-th would
      // (among a few thousand accounts 22 bits nearly always suffice)
      if (all_equal) break;
    }
  }
  // prefix is the K-th largest key, of the rows equal to it the `want` lowest are kept; or (all_equal)
  // exactly the rows with keys from prefix on are

  // ---- ordered scans ----
  auto widen = [](Pair v) { return (uint64_t)(v >> kHalf) << 32 | (uint32_t)(v & (((Pair)1 << kHalf) - 1)); };
  // sums of share[slot] over the CTAs before this one and over all: lane q asks CTA q
  auto over_cluster = [&](int slot, uint64_t& all) {
    const int lane = threadIdx.x & 31;
    const uint64_t v = lane < ranks ? widen(cluster.map_shared_rank(share, lane)[slot]) : 0;
    uint64_t x = lane < rank ? v : 0;
    all = v;
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      x += __shfl_xor_sync(FULL_MASK, x, o);
      all += __shfl_xor_sync(FULL_MASK, all, o);
    }
    all = __shfl_sync(FULL_MASK, all, 0);
    return __shfl_sync(FULL_MASK, x, 0);                       // at most eight CTAs: lanes 0-7 hold them
  };
  Pair total;
  int e0 = 0;                                                 // rows with the K-th key before this thread's
  if (K > 0 && !all_equal) {
    Pair equal = 0;
    rows([&](int, uint32_t k) { equal += k == prefix; });
    e0 = (int)cta_scan<NT, Pair>(equal, warp_s, total);
    if (threadIdx.x == 0) share[0] = total;
    meet();
    uint64_t all;
    if (ranks > 1) e0 += (int)over_cluster(0, all);
  }
  int e = e0;
  auto stays = [&](uint32_t k) {                              // rows asked in order
    if (K == 0) return false;
    return k > prefix || (k == prefix && (all_equal || e++ < want));
  };
  Pair mine = 0;                                              // holes, and movers in the high half
  uint32_t hole_bits = 0, mover_bits = 0;                     // of this thread's rows (R > 0)
  if constexpr (R > 0) {
    uint32_t st = 0;
    if (K > 0 && r0 < r1) {
#pragma unroll
      for (int i = 0; i < R; ++i) st |= (keys[i] >= prefix ? 1u : 0u) << i;
      if (!all_equal) {                                       // of the equal rows only the first `want` of all
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (keys[i] == prefix && r0 + i < r1 && e++ >= want) st &= ~(1u << i);
      }
    }
    auto low = [](int c) { return c >= R ? (R == 32 ? 0xffffffffu : (1u << R) - 1u) : (c <= 0 ? 0u : (1u << c) - 1u); };
    const uint32_t valid = low(r1 - r0), below = low(K - r0);
    hole_bits = valid & below & ~st;
    mover_bits = valid & ~below & st;
    mine = (Pair)__popc(hole_bits) | (Pair)__popc(mover_bits) << kHalf;
  } else {
    rows([&](int r, uint32_t k) {
      const bool st = stays(k);
      mine += r < K ? (Pair)!st : (Pair)st << kHalf;
    });
  }
  const Pair local = cta_scan<NT, Pair>(mine, warp_s, total);
  uint64_t first = 0, moves_all = widen(total);               // of the cluster, before this CTA; in all
  if (ranks > 1) {
    if (threadIdx.x == 0) share[1] = total;
    meet();
    first = over_cluster(1, moves_all);
  }
  if (rank == 0 && threadIdx.x == 0) a.counts[sg] = (int)(moves_all >> 32);
  int32_t* dst = a.dst + (size_t)sg * a.max_moves;
  int32_t* src = a.src + (size_t)sg * a.max_moves;
  if constexpr (R > 0) {
    // through shared memory, so that the lists leave in whole lines (each thread's own entries lie
    // apart from the next lane's: written directly they took 6 us of a 131072-row selection)
    const int c0 = rank * NT * R, holes = (int)(uint32_t)widen(total), movers = (int)(widen(total) >> 32);
    int h = (int)(uint32_t)widen(local), mv = holes + (int)(widen(local) >> 32);
    for (; hole_bits; hole_bits &= hole_bits - 1) stage[h++] = (uint16_t)(r0 - c0 + __ffs(hole_bits) - 1);
    for (; mover_bits; mover_bits &= mover_bits - 1) stage[mv++] = (uint16_t)(r0 - c0 + __ffs(mover_bits) - 1);
    __syncthreads();
    int32_t *d = dst + (uint32_t)first, *q = src + (first >> 32);
    for (int i = threadIdx.x; i < holes; i += NT) d[i] = c0 + stage[i];
    for (int i = threadIdx.x; i < movers; i += NT) q[i] = c0 + stage[holes + i];
  } else {
    const uint64_t at = widen(local) + first;
    uint32_t h_at = (uint32_t)at, m_at = (uint32_t)(at >> 32);
    e = e0;
    rows([&](int r, uint32_t k) {
      const bool st = stays(k);
      if (r < K) {
        if (!st) dst[h_at++] = r;
      } else if (st) {
        src[m_at++] = r;
      }
    });
  }
  // rows below K: accounts and positions (those of the holes are written again below)
#pragma unroll 4
  for (int r = (a.in_place ? kept : 0) + rank * NT + threadIdx.x; r < K; r += ranks * NT) {
    if (!a.in_place) mass_out[r] = mass[r];
    pos_out[r] = position(r);
  }
  meet();                                                     // the list is whole; no shared memory is read from here on
  const int n_moves = (int)(moves_all >> 32);
#pragma unroll 4
  for (int i = rank * NT + threadIdx.x; i < n_moves; i += ranks * NT) {
    const int to = dst[i], from = src[i];
    const float x = mass[from];
    const int p = position(from);
    mass_out[to] = x;
    pos_out[to] = p;
  }
  if (a.in_place) meet();                                     // every mover's account was read
  for (int r = K + rank * NT + threadIdx.x; r < n; r += ranks * NT) mass_out[r] = 0.f;
}

// Moves the listed rows.  CTAs [sg * split, sg * split + split) share the list of one
// (sequence, kv head); a warp takes four moves at a time, all loads before the stores.
template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a, const int split) {
  constexpr int V = D / 8;                                    // lanes per K (or V) row
  constexpr int U = 4;
  grid_dep_wait();
  const int sg = blockIdx.x / split, part = blockIdx.x % split, s = sg / a.n_kv, g = sg % a.n_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (part == 0 && g == 0 && threadIdx.x == 0) {              // every head of the sequence has read them
    const int n = clamp_ctx(a.ctx[s], a.max_ctx), K = max(0, min(a.keep[s], n));
    a.dropped_out[s] = a.dropped[s] + n - K;
    a.kept_out[s] = K < n ? K : a.kept[s];
  }
  const int count = a.counts[sg];
  const int32_t* dst = a.dst + (size_t)sg * a.max_moves;
  const int32_t* src = a.src + (size_t)sg * a.max_moves;
  const int32_t* bt = a.bt + (size_t)s * a.max_blocks;
  const int low = (1 << a.bs_log2) - 1;
  // a row's K takes V lanes and its V row the V lanes behind them; with D = 64 a warp holds two moves
  constexpr int PER = 32 / (2 * V);
  const int which = lane / (2 * V), half = (lane / V) & 1, vec = lane % V;
  uint4* pool = half ? a.v_pool : a.k_pool;
  auto row = [&](int r, bool& ok) -> uint4* {
    const int phys = bt[r >> a.bs_log2];
    if ((unsigned)phys >= (unsigned)a.num_blocks) {
      set_err(a.err, PKV_DEV_BAD_BLOCK);
      ok = false;
      return pool;
    }
    return pool + ((((size_t)phys * a.n_kv + g) << a.bs_log2) + (r & low)) * V + vec;
  };
  for (int i0 = (part * 8 + warp) * U * PER; i0 < count; i0 += split * 8 * U * PER) {
    uint4 x[U];
    uint4* d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * PER + which;
      d[u] = nullptr;
      if (i < count) {
        bool ok = true;
        uint4* to = row(dst[i], ok);
        const uint4* from = row(src[i], ok);
        if (ok) {
          d[u] = to;
          x[u] = *from;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (d[u]) *d[u] = x[u];
  }
}

static bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bytes && y < x + bytes;
}

struct EvictLayout {
  size_t dst, src, total;
  int max_moves;
};
static EvictLayout evict_layout(int batch, int n_kv, long long max_ctx) {
  EvictLayout w;
  w.max_moves = (int)(max_ctx / 2 + 1);                       // movers and holes lie on both sides of K
  const size_t list = sizeof(int32_t) * (size_t)batch * n_kv * w.max_moves;
  w.dst = align_up(sizeof(int) * (size_t)batch * n_kv, 256);
  w.src = align_up(w.dst + list, 256);
  w.total = align_up(w.src + list, 256);
  return w;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_evict_workspace_bytes(int batch, int n_kv, int block_size, int max_blocks) {
  if (batch < 0 || n_kv <= 0 || max_blocks < 0 || (block_size != 16 && block_size != 32 && block_size != 64)) return 0;
  if ((long long)max_blocks * block_size > kEvMaxRows) return 0;
  const size_t n = evict_layout(batch, n_kv, (long long)max_blocks * block_size).total;
  return n ? n : 256;
}

extern "C" pkv_status pkv_kv_evict(void* k_pool, void* v_pool, const int32_t* block_tables, int max_blocks,
                                   const int32_t* context_lens, const int32_t* keep, int recent, const float* mass,
                                   const int32_t* positions, const int32_t* kept, const int32_t* dropped,
                                   float* mass_out, int32_t* positions_out, int32_t* kept_out, int32_t* dropped_out,
                                   int64_t stride, int32_t* new_lens, int batch, int n_kv, int head_dim, int block_size,
                                   int num_blocks, void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_kv_evict");
  if (batch < 0 || n_kv <= 0 || max_blocks < 0 || num_blocks < 0 || recent < 0) return PKV_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PKV_EINVAL;
  if (block_size != 16 && block_size != 32 && block_size != 64) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  if (!k_pool || !v_pool || !block_tables || !context_lens || !keep || !mass || !positions || !kept || !dropped ||
      !mass_out || !positions_out || !kept_out || !dropped_out || !new_lens || !workspace)
    return PKV_EINVAL;
  for (const void* p : {(const void*)k_pool, (const void*)v_pool})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return PKV_EINVAL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_EINVAL;
  // the state is replaced as a whole or written to another one as a whole
  const bool in_place = mass_out == mass;
  // the lengths are written while these are still read
  for (const int32_t* p : {context_lens, keep, kept, dropped})
    if (new_lens < p + batch && p < new_lens + batch) return PKV_EINVAL;
  if (in_place != (positions_out == positions) || in_place != (kept_out == kept) || in_place != (dropped_out == dropped))
    return PKV_EINVAL;
  const long long max_ctx = (long long)max_blocks * block_size;
  if (max_ctx > kEvMaxRows) return PKV_ERANGE;
  if (stride < max_ctx) return PKV_EINVAL;
  if ((long long)batch * n_kv > 0x7fffffffLL / 64) return PKV_ERANGE;
  const EvictLayout w = evict_layout(batch, n_kv, max_ctx);
  if (workspace_bytes < w.total) return PKV_ENOSPC;
  // no output lies over another, nor a new state over what is still read of the old one
  const size_t lens = sizeof(int32_t) * (size_t)batch;
  const size_t rows = sizeof(float) * ((size_t)((long long)batch * n_kv - 1) * (size_t)stride + (size_t)max_ctx);
  if (overlap(new_lens, kept_out, lens) || overlap(new_lens, dropped_out, lens) || overlap(kept_out, dropped_out, lens) ||
      overlap(mass_out, positions_out, rows))
    return PKV_EINVAL;
  if (!in_place) {
    for (const int32_t* p : {context_lens, keep, kept, dropped})
      if (overlap(kept_out, p, lens) || overlap(dropped_out, p, lens)) return PKV_EINVAL;
    for (const void* p : {(const void*)mass, (const void*)positions})
      if (overlap(mass_out, p, rows) || overlap(positions_out, p, rows)) return PKV_EINVAL;
  }
  char* ws = static_cast<char*>(workspace);
  EvictArgs a = {};
  a.mass = mass; a.positions = positions; a.kept = kept; a.dropped = dropped;
  a.mass_out = mass_out; a.positions_out = positions_out; a.kept_out = kept_out; a.dropped_out = dropped_out;
  a.new_lens = new_lens;
  a.ctx = context_lens; a.keep = keep; a.bt = block_tables;
  a.stride = stride;
  a.batch = batch; a.n_kv = n_kv; a.max_blocks = max_blocks; a.max_ctx = (int)max_ctx;
  a.bs_log2 = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
  a.recent = recent; a.num_blocks = num_blocks;
  a.counts = reinterpret_cast<int*>(ws);
  a.dst = reinterpret_cast<int32_t*>(ws + w.dst);
  a.src = reinterpret_cast<int32_t*>(ws + w.src);
  a.max_moves = w.max_moves;
  a.k_pool = static_cast<uint4*>(k_pool);
  a.v_pool = static_cast<uint4*>(v_pool);
  a.err = err_flag;
  a.in_place = in_place;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count() > 0 ? device_sm_count() : 128;
  const long long pairs = (long long)batch * n_kv;
  a.vec = stride % 4 == 0 && !((reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(positions)) & 15u);
  // A CTA's threads times their rows hold a (sequence, kv head) of up to 4096 rows: few rows per thread,
  // since a thread takes its own in series, in no more threads than stay busy (1000 rows: four rows 8.4
  // us, 16 rows 10.4; 32 pairs of 2000 rows: 512 threads 9.5, 256 threads 11.6, 2048 pairs of them 40.6
  // and 36.7; 512 pairs of up to 4096 rows: 512 x 8 rows 82.8, 256 x 16 rows 84.4, 1024 x 4 rows 89.7).
  // Beyond that a cluster of up to eight CTAs of 512 x 8 rows (8 pairs of 15000: 19.4 us, 256 x 16 24.1;
  // 256 pairs of 9000, where that was better: 41.4 and 39.1), of 1024 x 8 (64 pairs of 60000: 222, 1024 x
  // 16 241) or 1024 x 16 rows; more than 131072 rows are read again in every round.
  // All of this goes by the table's width, the host knowing no lengths: with a table wider than any sequence
  // the clusters hold mostly idle threads (64 x 2.1-4K rows, 8 heads: 83 us with a table of 4096 rows, 109
  // with 8192, 238 with 32768, 457 with 131072).
  const bool few = pairs <= 4LL * sms;
  int threads, ranks = 1;
  const void* fn;
  if (max_ctx <= 1024) {
    threads = 256;
    fn = (const void*)evict_select_kernel<256, 4, false>;
  } else if (max_ctx <= 2048) {
    threads = few ? 512 : 256;
    fn = few ? (const void*)evict_select_kernel<512, 4, false> : (const void*)evict_select_kernel<256, 8, false>;
  } else if (max_ctx <= 4096) {
    threads = 512;
    fn = (const void*)evict_select_kernel<512, 8, false>;
  } else if (max_ctx <= 8 * 4096) {
    threads = 512;
    while (max_ctx > 4096LL * ranks) ranks *= 2;
    fn = (const void*)evict_select_kernel<512, 8, true>;
  } else {
    threads = 1024;
    ranks = 8;
    fn = max_ctx <= 8 * 8192 ? (const void*)evict_select_kernel<1024, 8, true>
         : max_ctx <= 8 * 16384 ? (const void*)evict_select_kernel<1024, 16, true> : (const void*)evict_select_kernel<1024, 0, true>;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * ranks));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* sargs[] = {&a};
  cudaError_t e = cudaLaunchKernelExC(&cfg, fn, sargs);
  if (e == cudaSuccess) {
    long long split = (16LL * sms + pairs - 1) / pairs;       // about 16 CTAs per SM
    const long long most = (w.max_moves + 31) / 32;
    if (split > most) split = most;
    if (split < 1) split = 1;
    int sp = (int)split;
    void* kargs[] = {&a, &sp};
    e = launch_pdl(head_dim == 128 ? (const void*)evict_move_kernel<128> : (const void*)evict_move_kernel<64>,
                   dim3((unsigned)(pairs * split)), dim3(256), 0, st, kargs);
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
