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
// Select kernel: a cluster of CTAs per (sequence, kv head), each holding the keys of an equal
// run of rows in shared memory (recent rows: the largest key; else the account's bits in an
// order-keeping form), so the accounts are read once.  Three rounds over 11, 11 and 10 bits of
// the key build histograms in shared memory, sum them over the cluster through distributed
// shared memory and narrow the K-th largest key; two ordered scans then give every hole and
// every mover its place.  Runs longer than the shared memory are read again from L2 per round.
// Move kernel: the listed rows of K and V, 16 bytes a lane, spread over the whole GPU.
//
// What bounds it: the select kernel, latency (three histogram rounds with cluster barriers over
// a few KB to MB of accounts); the move kernel, HBM (4 d bytes read and written per moved row).
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
  int2* moves;                   // workspace: [batch * n_kv][max_ctx / 2 + 1]: x destination, y source
  int max_moves;
  uint4 *k_pool, *v_pool;
  int32_t* err;
  int staged;                    // keys a CTA holds in shared memory (0: none)
  int in_place;
};

constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;
constexpr int kEvWarps = kEvThreads / 32;

// Order-keeping bits of an account: -0 below +0, NaN above everything but the recent rows.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix sum of x over the CTA's threads, in thread order; total gets the sum.
__device__ __forceinline__ int cta_scan(int x, int* warp_s, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL_MASK, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                                            // warp_s may still be read from the last scan
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w) {
    const int v = warp_s[w];
    if (w < warp) before += v;
    all += v;
  }
  total = all;
  return before + incl - x;
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const EvictArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kEvBins];
  __shared__ int warp_s[kEvWarps];
  __shared__ int share[4];                                    // this CTA's counts, read by the cluster
  __shared__ int pick[2];
  const int sg = blockIdx.x / ranks, s = sg / a.n_kv;
  const int raw = a.ctx[s], n = clamp_ctx(raw, a.max_ctx);
  const int K = max(0, min(a.keep[s], n));
  const int kept = min(max(a.kept[s], 0), n), dropped = a.dropped[s];
  const float* mass = a.mass + (size_t)sg * a.stride;
  const int32_t* posn = a.positions + (size_t)sg * a.stride;
  float* mass_out = a.mass_out + (size_t)sg * a.stride;
  int32_t* pos_out = a.positions_out + (size_t)sg * a.stride;
  const int per = ((n + ranks - 1) / ranks + 3) & ~3;         // rows of a CTA
  const int r0 = min(n, rank * per), r1 = min(n, r0 + per), rows = r1 - r0;
  if (rank == 0 && sg % a.n_kv == 0 && threadIdx.x == 0) {
    if (raw != n) set_err(a.err, PKV_DEV_BAD_CTX);
    // here and not in the move kernel: an attention call behind this one may read the lengths
    // while the move kernel still runs
    a.new_lens[s] = K;
  }

  if (K == n) {                                               // nothing to evict (uniform in the cluster)
    if (rank == 0 && threadIdx.x == 0) a.counts[sg] = 0;
    if (!a.in_place)
      for (int r = r0 + threadIdx.x; r < r1; r += kEvThreads) {
        mass_out[r] = mass[r];
        if (r < kept) pos_out[r] = posn[r];
      }
    return;
  }
  // rows at or behind this position are recent: the newest is dropped + n - 1
  const int recent_from = dropped + n - min(a.recent, K);
  auto position = [&](int r) { return r < kept ? posn[r] : dropped + r; };
  auto make_key = [&](int r) { return position(r) >= recent_from ? 0xffffffffu : order_bits(mass[r]); };
  const bool staged = rows <= a.staged;
  if (staged)
    for (int i = threadIdx.x; i < rows; i += kEvThreads) keys[i] = make_key(r0 + i);
  auto key = [&](int i) { return staged ? keys[i] : make_key(r0 + i); };   // i counts from r0

  // ---- the K-th largest key: 11 + 11 + 10 bits from the top ----
  uint32_t prefix = 0, mask = 0;
  int want = K;                                               // rank of the wanted key among those matching prefix
  if (K > 0) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bins = round == 2 ? 1024 : 2048;
      for (int b = threadIdx.x; b < bins; b += kEvThreads) hist[b] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < rows; i0 += kEvThreads) {
        const int i = i0 + threadIdx.x;
        const uint32_t k = i < rows ? key(i) : 0;
        if (i < rows && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      cluster.sync();
      // thread t: bins from the top, 2 t and 2 t + 1 (1024 bins: bin t)
      const int nb = bins / kEvThreads;
      int c[2] = {0, 0};
      for (int q = 0; q < ranks; ++q) {
        const int* h = cluster.map_shared_rank(hist, q);
        for (int j = 0; j < nb; ++j) c[j] += h[bins - 1 - (threadIdx.x * nb + j)];
      }
      int total;
      const int before = cta_scan(c[0] + c[1], warp_s, total);
      for (int j = 0, at = before; j < nb; at += c[j], ++j)
        if (at < want && want <= at + c[j]) {
          pick[0] = bins - 1 - (threadIdx.x * nb + j);
          pick[1] = want - at;
        }
      cluster.sync();                                         // all have read the histograms; pick is set
      prefix |= (uint32_t)pick[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      want = pick[1];
    }
  }
  // prefix is the K-th largest key; of the rows equal to it the `want` lowest are kept

  // ---- ordered scans: thread t takes the rows [t * each, t * each + each) of the CTA ----
  const int each = (rows + kEvThreads - 1) / kEvThreads | 1;  // odd: threads start in distinct banks
  const int b0 = min(rows, (int)threadIdx.x * each), b1 = min(rows, b0 + each);
  auto cluster_before = [&](int slot) {                       // sum of share[slot] over the CTAs before this one
    int x = 0;
    for (int q = 0; q < rank; ++q) x += cluster.map_shared_rank(share, q)[slot];
    return x;
  };
  int equal = 0, total;
  if (K > 0)
    for (int i = b0; i < b1; ++i) equal += key(i) == prefix;
  int eq_at = cta_scan(equal, warp_s, total);
  if (threadIdx.x == 0) share[0] = total;
  cluster.sync();
  eq_at += cluster_before(0);
  int holes = 0, movers = 0;
  {
    int e = eq_at;
    for (int i = b0; i < b1; ++i) {
      const uint32_t k = key(i);
      const bool stays = K > 0 && (k > prefix || (k == prefix && e < want));
      e += K > 0 && k == prefix;
      if (r0 + i < K) holes += !stays; else movers += stays;
    }
  }
  int h_at = cta_scan(holes, warp_s, total);
  if (threadIdx.x == 0) share[1] = total;
  int m_at = cta_scan(movers, warp_s, total);
  if (threadIdx.x == 0) share[2] = total;
  cluster.sync();
  h_at += cluster_before(1);
  m_at += cluster_before(2);
  int n_moves = 0;
  for (int q = 0; q < ranks; ++q) n_moves += cluster.map_shared_rank(share, q)[2];
  int2* moves = a.moves + (size_t)sg * a.max_moves;
  {
    int e = eq_at;
    for (int i = b0; i < b1; ++i) {
      const uint32_t k = key(i);
      const bool stays = K > 0 && (k > prefix || (k == prefix && e < want));
      e += K > 0 && k == prefix;
      if (r0 + i < K) {
        if (!stays) moves[h_at++].x = r0 + i;
      } else if (stays) {
        moves[m_at++].y = r0 + i;
      }
    }
  }
  if (rank == 0 && threadIdx.x == 0) a.counts[sg] = n_moves;
  // rows below K that stay: their accounts and positions (a hole's come with its mover)
  for (int r = r0 + threadIdx.x; r < min(r1, K); r += kEvThreads) {
    if (!a.in_place) mass_out[r] = mass[r];
    if (!a.in_place || r >= kept) pos_out[r] = position(r);
  }
  __threadfence();
  cluster.sync();                                             // the lists are whole, the rows below K written
  for (int i = rank * kEvThreads + threadIdx.x; i < n_moves; i += ranks * kEvThreads) {
    const int2 mv = moves[i];
    mass_out[mv.x] = mass[mv.y];
    pos_out[mv.x] = position(mv.y);
  }
  if (a.in_place) cluster.sync();                             // every mover's account was read
  for (int r = max(r0, K) + threadIdx.x; r < r1; r += kEvThreads) mass_out[r] = 0.f;
  cluster.sync();                                             // no CTA leaves while its shared memory is read
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
  const int2* moves = a.moves + (size_t)sg * a.max_moves;
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
        const int2 mv = moves[i];
        bool ok = true;
        uint4* to = row(mv.x, ok);
        const uint4* from = row(mv.y, ok);
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

struct EvictLayout {
  size_t moves, total;
  int max_moves;
};
static EvictLayout evict_layout(int batch, int n_kv, long long max_ctx) {
  EvictLayout w;
  w.max_moves = (int)(max_ctx / 2 + 1);                       // movers and holes lie on both sides of K
  w.moves = align_up(sizeof(int) * (size_t)batch * n_kv, 256);
  w.total = align_up(w.moves + sizeof(int2) * (size_t)batch * n_kv * w.max_moves, 256);
  return w;
}

constexpr int kEvStaged = 48 * 1024;                          // keys in shared memory per CTA at most

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_evict_workspace_bytes(int batch, int n_kv, int block_size, int max_blocks) {
  if (batch < 0 || n_kv <= 0 || max_blocks < 0 || (block_size != 16 && block_size != 32 && block_size != 64)) return 0;
  if ((long long)max_blocks * block_size > 0x7fffffffLL) return 0;
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
  if (new_lens == context_lens || new_lens == keep) return PKV_EINVAL;   // both are still read
  if (in_place != (positions_out == positions) || in_place != (kept_out == kept) || in_place != (dropped_out == dropped))
    return PKV_EINVAL;
  const long long max_ctx = (long long)max_blocks * block_size;
  if (max_ctx > 0x7fffffffLL) return PKV_ERANGE;
  if (stride < max_ctx) return PKV_EINVAL;
  if ((long long)batch * n_kv > 0x7fffffffLL / 64) return PKV_ERANGE;
  const EvictLayout w = evict_layout(batch, n_kv, max_ctx);
  if (workspace_bytes < w.total) return PKV_ENOSPC;
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
  a.moves = reinterpret_cast<int2*>(ws + w.moves);
  a.max_moves = w.max_moves;
  a.k_pool = static_cast<uint4*>(k_pool);
  a.v_pool = static_cast<uint4*>(v_pool);
  a.err = err_flag;
  a.in_place = in_place;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count() > 0 ? device_sm_count() : 128;
  const long long pairs = (long long)batch * n_kv;
  // CTAs per (sequence, kv head): enough for about 4096 rows each, while the grid stays within
  // two CTAs per SM; longer rows still take a cluster of up to eight
  int ranks = 1;
  while (ranks < 8 && max_ctx > 4096LL * ranks && (pairs * ranks * 2 <= 2LL * sms || max_ctx > (long long)kEvStaged * ranks)) ranks *= 2;
  long long staged = ((max_ctx + ranks - 1) / ranks + 3) & ~3LL;
  if (staged > kEvStaged) staged = 0;
  a.staged = (int)staged;
  const size_t smem = (size_t)staged * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute((const void*)evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kEvStaged * (int)sizeof(uint32_t));
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * ranks));
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* kargs[] = {&a};
    e = cudaLaunchKernelExC(&cfg, (const void*)evict_select_kernel, kargs);
  }
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
