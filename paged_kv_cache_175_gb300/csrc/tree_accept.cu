// Accepted paths of drafted tokens: their cache rows move to the front of the drafted ones, in all caches
// of a call (every layer's pools) at once.
//
// A thread owns one 16-byte column of a sequence's drafted rows in one cache and head and moves the path's
// rows in ascending order, four loads ahead of four stores.  path[i] >= i, so a row is written only
// once it has been read: the rows still to be read come after path[i], and the thread's column is
// nobody else's.  Rows that stay where they are are not touched.
// What bounds it: four dependent memory round trips (lengths and path, block ids, rows, stores); one launch for
// all layers where a launch per layer would cost that much each.  64 sequences, 8 layers of K and V of 8 x 128: 5.6 us;
// 4 sequences, 40 latent caches: 6.7 us.  Eight loads ahead and CTAs of 256 threads took 7.1 and 7.6: twice the registers,
// and CTAs in two waves.
#include <algorithm>
#include <vector>

#include "drafts.cuh"
#include "nvtx_range.h"

namespace pkv {

constexpr int kAcceptCaches = 256;               // per launch: pointers passed by value
struct AcceptArgs {
  const int32_t *bt, *ctx, *q_start, *path, *n_accept;
  int32_t* new_lens;
  long long columns;                             // per cache: batch * heads * vectors of a row
  int max_blocks, max_ctx, n_each, n_tok, batch, heads, vecs, path_stride, bs_log2, num_blocks, write_lens;
  int32_t* err;
  uint4* caches[kAcceptCaches];
};

constexpr int kAcceptBatch = 4, kAcceptThreads = 128;

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const long long col = (long long)blockIdx.x * kAcceptThreads + threadIdx.x;
  if (col >= a.columns) return;
  const int v = (int)(col % a.vecs), h = (int)(col / a.vecs % a.heads), s = (int)(col / ((long long)a.vecs * a.heads));
  const bool speaks = blockIdx.y == 0 && v == 0 && h == 0;    // one thread per sequence flags and writes its length
  int flags = 0;
  // the path's first rows are asked for with the lengths: how many of them count is known behind both
  int at[kAcceptBatch];
  auto ask = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i) at[i] = i0 + i < a.path_stride ? a.path[(size_t)s * a.path_stride + i0 + i] : -1;
  };
  ask(0);
  int count = a.n_accept[s];
  const Drafts d = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, s, flags);
  const int base = d.ctx - d.n, most = min(d.n, a.path_stride);
  if (base < 0 && count != 0) flags |= PKV_DEV_BAD_TREE;      // (drafted tokens of a padded sequence, of length 0, are none's)
  if (count < 0 || count > most) {
    flags |= PKV_DEV_BAD_TREE;
    count = count < 0 ? 0 : most;
  }
  if (base < 0) count = 0;
  uint4* cache = a.caches[blockIdx.y];
  const int32_t* bt = a.bt + (size_t)s * a.max_blocks;
  const int in = (1 << a.bs_log2) - 1;
  int last = -1, done = 0;
  bool good = true;
  for (int i0 = 0; i0 < count && good; i0 += kAcceptBatch) {
    long long src[kAcceptBatch], dst[kAcceptBatch];            // block ids, then columns of rows in the cache, in vectors
    uint4 x[kAcceptBatch];
    if (i0) ask(i0);
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i) {
      src[i] = dst[i] = -1;                                   // nothing to do
      if (i0 + i >= count || !good) continue;
      good = at[i] > last && at[i] < d.n;
      if (!good) continue;
      last = at[i];
      ++done;
      if (at[i] == i0 + i) continue;
      src[i] = (unsigned)bt[(base + at[i]) >> a.bs_log2];
      dst[i] = (unsigned)bt[(base + i0 + i) >> a.bs_log2];
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i) {
      const bool both = src[i] >= 0 && src[i] < a.num_blocks && dst[i] < a.num_blocks;
      bad |= src[i] >= 0 && !both;
      src[i] = both ? ((((src[i] * a.heads + h) << a.bs_log2) + ((base + at[i]) & in))) * a.vecs + v : -1;
      dst[i] = ((((dst[i] * a.heads + h) << a.bs_log2) + ((base + i0 + i) & in))) * a.vecs + v;
    }
    if (bad) set_err(a.err, PKV_DEV_BAD_BLOCK);
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i)
      if (src[i] >= 0) x[i] = cache[src[i]];
#pragma unroll
    for (int i = 0; i < kAcceptBatch; ++i)
      if (src[i] >= 0) cache[dst[i]] = x[i];
  }
  if (!speaks || !a.write_lens) return;
  if (!good) flags |= PKV_DEV_BAD_TREE;
  if (flags) set_err(a.err, flags);
  a.new_lens[s] = base < 0 ? d.ctx : base + done;
}

}  // namespace pkv

using namespace pkv;

// Whether two of n caches of `bytes` each share memory (one given twice, say, whose rows would move twice).
static bool any_overlap(void* const* caches, int n, uint64_t bytes) noexcept {
  try {
    std::vector<uintptr_t> at(n);
    for (int i = 0; i < n; ++i) at[i] = reinterpret_cast<uintptr_t>(caches[i]);
    std::sort(at.begin(), at.end());
    for (int i = 1; i < n; ++i)
      if (at[i] - at[i - 1] < bytes) return true;
    return false;
  } catch (...) {
    return true;
  }
}

extern "C" pkv_status pkv_kv_tree_accept(void* const* caches, int n_caches, int row_bytes, int heads, const int32_t* block_tables,
                                         int max_blocks, const int32_t* context_lens, const int32_t* q_start, int n_tok,
                                         const int32_t* path, int path_stride, const int32_t* n_accept, int32_t* new_lens,
                                         int batch, int block_size, int num_blocks, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_kv_tree_accept");
  if (n_caches < 1 || row_bytes < 16 || row_bytes % 16 || heads < 1 || max_blocks < 0 || n_tok < 0 || path_stride < 0 || batch < 0 ||
      num_blocks < 0)
    return PKV_EINVAL;
  if (block_size != 16 && block_size != 32 && block_size != 64) return PKV_EINVAL;
  if (batch > 0 && !q_start && n_tok % batch) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  if (!caches || !block_tables || !context_lens || !n_accept || !new_lens || (!path && path_stride > 0)) return PKV_EINVAL;
  for (int i = 0; i < n_caches; ++i)
    if (!caches[i] || (reinterpret_cast<uintptr_t>(caches[i]) & 15u)) return PKV_EINVAL;
  const size_t lens = sizeof(int32_t) * (size_t)batch;
  if (overlaps(new_lens, lens, context_lens, lens) || overlaps(new_lens, lens, n_accept, lens) ||
      overlaps(new_lens, lens, path, lens * path_stride) || overlaps(new_lens, lens, q_start, lens + sizeof(int32_t)))
    return PKV_EINVAL;
  if ((long long)max_blocks * block_size > 0x7fff0000LL) return PKV_ERANGE;
  if (any_overlap(caches, n_caches, std::max<uint64_t>(1, (uint64_t)num_blocks * heads * block_size * row_bytes))) return PKV_EINVAL;
  AcceptArgs a = {};
  a.bt = block_tables; a.ctx = context_lens; a.q_start = q_start; a.path = path; a.n_accept = n_accept;
  a.new_lens = new_lens;
  a.max_blocks = max_blocks;
  a.max_ctx = max_blocks * block_size;
  a.n_each = q_start ? 0 : n_tok / batch;
  a.n_tok = n_tok; a.batch = batch; a.heads = heads;
  a.vecs = row_bytes / 16;
  a.path_stride = path_stride;
  a.bs_log2 = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
  a.num_blocks = num_blocks;
  a.err = err_flag;
  a.columns = (long long)batch * heads * a.vecs;
  const long long grid = (a.columns + kAcceptThreads - 1) / kAcceptThreads;
  if (grid > 0x7fffffffLL) return PKV_ERANGE;
  for (int c0 = 0; c0 < n_caches; c0 += kAcceptCaches) {
    const int n = n_caches - c0 < kAcceptCaches ? n_caches - c0 : kAcceptCaches;
    for (int i = 0; i < n; ++i) a.caches[i] = static_cast<uint4*>(caches[c0 + i]);
    a.write_lens = c0 == 0;
    void* kargs[] = {&a};
    const cudaError_t e = launch_pdl((const void*)tree_accept_kernel, dim3((unsigned)grid, n), dim3(kAcceptThreads), 0,
                                     static_cast<cudaStream_t>(stream), kargs);
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return PKV_ECUDA;
    }
  }
  return PKV_OK;
}
