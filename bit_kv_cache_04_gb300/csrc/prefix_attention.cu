// kvq_prefix_attention: attention of the newest tokens of every sequence where groups of sequences hold the same
// pages for a common prefix.
//
// With P the tokens that a group shares, a row's softmax splits at P:
//   out = (e^a A + e^b B) / (e^a + e^b),
// A and a the output and log-sum over tokens [0, P), B and b over [P, p_i].  All rows of the group see all of [0, P), so
// that part is one unit of (rows of the group) x (prefix): its packed tokens are read and dequantized once instead of once a
// sequence.  Both parts run in one launch of the chunk attention kernel (chunk_kernel.cuh), on one line of tiles cut into equal runs;
// a pass over the rows joins them.
//
// The prefix is what the block table says: the pages that the group's sequences hold in the same places, as far as
// they are quantized in all of them and before every new token, in whole tiles (so that neither part needs a mask
// at the border).  kvq_prefix_plan finds it, on the device.
#include <algorithm>
#include <climits>

#include "chunk_attention.cuh"
#include "kvq_host.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  Layout lo;
  const int32_t* table;
  const int32_t* cu_groups;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int n_groups, total_q, max_q, max_group_q, tile;
  uint32_t* status;
  Segment* segs;  // [n_groups] prefixes, [batch] sequences
};

// One block a group: its sequences' lengths, the pages that they have in common, its segments.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int common, limit, live;
  __shared__ uint32_t bad;
  grid_launch_dependents();
  grid_dependency_wait();
  const int g = blockIdx.x, tid = threadIdx.x, B = a.lo.B, mp = a.lo.max_pages;
  if (tid == 0) {
    common = limit = INT_MAX;
    live = 0;
    bad = 0;
  }
  // the groups cover the batch, in order
  bool wrong = false;
  for (int i = tid; i <= a.n_groups; i += kPlanThreads) {
    const int at = a.cu_groups[i];
    wrong |= i == 0 ? at != 0 : at < a.cu_groups[i - 1];
    if (i == a.n_groups) wrong |= at != B;
  }
  const Segment none{};
  if (__syncthreads_or(wrong)) {  // every block says the same: nothing to do
    for (int b = g * kPlanThreads + tid; b < B; b += a.n_groups * kPlanThreads) a.segs[a.n_groups + b] = none;
    if (tid == 0) {
      a.segs[g] = none;
      atomicOr(a.status, KVQ_DEV_SEQ);
    }
    return;
  }
  const int b0 = a.cu_groups[g], b1 = a.cu_groups[g + 1];
  // sequences: what is in order, and how far a prefix of those with new tokens may go
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], T = a.seq_lens[b];
    const int n = (int)((uint32_t)c1 - (uint32_t)c0);
    Segment s{};
    if (c0 < 0 || c1 < c0 || c1 > a.total_q || n > a.max_q || T < n || T > a.lo.max_T) {
      atomicOr(&bad, KVQ_DEV_LENGTH);
    } else if (n > 0) {
      s.n = n;
      s.T = T;
      s.cu = c0;
      s.b = b;
      atomicMin(&limit, min(q_end_of(a.lo, T), T - n));
      atomicAdd(&live, 1);
    }
    a.segs[a.n_groups + b] = s;
  }
  __syncthreads();
  if (tid == 0) {
    if (g == 0 && a.cu_q[0] != 0) atomicOr(&bad, KVQ_DEV_LENGTH);
    if (live > 1 && !bad && a.cu_q[b1] - a.cu_q[b0] > a.max_group_q) atomicOr(&bad, KVQ_DEV_LENGTH);
  }
  __syncthreads();
  // (with a sequence out of order the rows of the others are not one run: they go without a common prefix)
  const bool share = live > 1 && !bad;
  if (share) {
    // the first page that the group's live sequences do not all hold: a thread compares a page with the first live sequence's
    int first = b0;
    while (a.cu_q[first + 1] == a.cu_q[first]) ++first;
    const int pages = limit / a.lo.pt;
    const int32_t* ref = a.table + (int64_t)first * mp;
    // few pages: threads share a page's sequences
    const int per = max(1, min(b1 - first, kPlanThreads / max(1, pages)));
    for (int64_t e = tid; e < (int64_t)pages * per; e += kPlanThreads) {
      const int j = (int)(e % pages), sub = (int)(e / pages);
      if (j >= *(volatile int*)&common) continue;
      const int p = ref[j];
      bool same = p >= 0 && p < a.lo.n_pages;
#pragma unroll 8
      for (int b = first + 1 + sub; b < b1; b += per) same &= a.table[(int64_t)b * mp + j] == p || a.cu_q[b + 1] == a.cu_q[b];
      if (!same) atomicMin(&common, j);
    }
  }
  __syncthreads();
  if (tid == 0 && bad) atomicOr(a.status, bad);
  const int pages = share ? min(common, limit / a.lo.pt) : 0;
  const int P = (int)((int64_t)pages * a.lo.pt / a.tile) * a.tile;
  if (P > 0)
    for (int b = b0 + tid; b < b1; b += kPlanThreads)
      if (a.segs[a.n_groups + b].n) a.segs[a.n_groups + b].from = P;  // (written by this thread)
  if (tid == 0) {
    Segment s{};
    if (P > 0) {
      int first = b0;
      while (a.cu_q[first + 1] == a.cu_q[first]) ++first;
      s.n = a.cu_q[b1] - a.cu_q[b0];
      s.T = P;
      s.cu = a.cu_q[b0];
      s.b = first;
      s.shared = 1;
    }
    a.segs[g] = s;
  }
}

// Workspace: that of the chunk attention, segments, two parts of every row.
struct PrefixWs {
  size_t segs, rows, total, zeroed;
};
PrefixWs prefix_ws(const kvq_config* c, int n_groups, int64_t rows) {
  PrefixWs w{};
  w.segs = align_up(chunk_workspace_bytes(c, &w.zeroed));
  w.rows = w.segs + align_up(sizeof(Segment) * ((size_t)n_groups + c->batch));
  w.total = w.rows + align_up(sizeof(float) * 2 * (size_t)rows * c->H_q * chunk_part_row(c->D));
  return w;
}

kvq_status prefix_config(const kvq_config* cfg, int32_t n_groups, int64_t rows) {
  const kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (cfg->page_tokens < 1) return fail(KVQ_ERR_ARG, "the cache is not paged");
  if (n_groups < 1 || n_groups > cfg->batch) return fail(KVQ_ERR_ARG, "n_groups=%d not in [1, batch=%d]", n_groups, cfg->batch);
  if (rows < 0 || rows > 0x7fffffff) return fail(KVQ_ERR_ARG, "rows=%lld", (long long)rows);
  return KVQ_OK;
}

kvq_status check_prefix_ws(const kvq_config* cfg, int32_t n_groups, int64_t rows, void* ws, size_t bytes) {
  if (!ws) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = prefix_ws(cfg, n_groups, rows).total;
  if (bytes < need) return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", bytes, need);
  if (((uintptr_t)ws) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return KVQ_OK;
}

kvq_status check_rows(const kvq_config* cfg, int32_t total_q, int32_t max_q, int32_t max_group_q) {
  if (total_q < 0 || max_q < 0 || max_group_q < max_q || max_group_q > total_q)
    return fail(KVQ_ERR_ARG, "total_q=%d, max_q=%d, max_group_q=%d", total_q, max_q, max_group_q);
  if (max_q > cfg->max_T) return fail(KVQ_ERR_CAPACITY, "max_q=%d > max_T=%d", max_q, cfg->max_T);
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_prefix_workspace_bytes(const kvq_config* cfg, int32_t n_groups, int64_t rows, size_t* bytes) {
  const kvq_status st = prefix_config(cfg, n_groups, rows);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  *bytes = prefix_ws(cfg, n_groups, rows).total;
  return ok();
}

kvq_status kvq_prefix_workspace_init(const kvq_config* cfg, int32_t n_groups, int64_t rows, void* workspace, size_t ws_bytes,
                                     void* stream) {
  kvq_status st = prefix_config(cfg, n_groups, rows);
  if (st != KVQ_OK) return st;
  if ((st = check_prefix_ws(cfg, n_groups, rows, workspace, ws_bytes)) != KVQ_OK) return st;
  const PrefixWs w = prefix_ws(cfg, n_groups, rows);
  cudaError_t e = cudaMemsetAsync(workspace, 0, w.zeroed, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemsetAsync((char*)workspace + w.segs, 0, w.rows - w.segs, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return ok();
}

kvq_status kvq_prefix_plan(const kvq_config* cfg, const int32_t* block_table, const int32_t* cu_groups, int32_t n_groups,
                           const int32_t* cu_q, int32_t total_q, int32_t max_q, int32_t max_group_q, const int32_t* seq_lens,
                           void* workspace, size_t ws_bytes, void* stream) {
  kvq_status st = prefix_config(cfg, n_groups, 0);
  if (st != KVQ_OK) return st;
  if ((st = check_rows(cfg, total_q, max_q, max_group_q)) != KVQ_OK) return st;
  if (!block_table || !cu_groups || !cu_q || !seq_lens) return fail(KVQ_ERR_ARG, "block_table / cu_groups / cu_q / seq_lens is NULL");
  if (((uintptr_t)block_table | (uintptr_t)cu_groups | (uintptr_t)cu_q | (uintptr_t)seq_lens) & 3u)
    return fail(KVQ_ERR_ARG, "block_table / cu_groups / cu_q / seq_lens must be 4-byte aligned");
  if ((st = check_prefix_ws(cfg, n_groups, 0, workspace, ws_bytes)) != KVQ_OK) return st;
  PlanArgs a{};
  a.lo = make_layout(cfg);
  a.table = block_table;
  a.cu_groups = cu_groups;
  a.cu_q = cu_q;
  a.seq_lens = seq_lens;
  a.n_groups = n_groups;
  a.total_q = total_q;
  a.max_q = max_q;
  a.max_group_q = max_group_q;
  a.tile = chunk_tile(cfg->D);
  a.status = (uint32_t*)workspace;
  a.segs = (Segment*)((char*)workspace + prefix_ws(cfg, n_groups, 0).segs);
  const cudaError_t e = launch_dependent(prefix_plan_kernel, dim3(n_groups), dim3(kPlanThreads), 0, (cudaStream_t)stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "prefix plan kernel");
  return ok();
}

kvq_status kvq_prefix_attention(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0, int32_t n_layers, int32_t n_groups,
                                const void* q, int32_t total_q, int32_t max_q, int32_t max_group_q, void* out, void* workspace,
                                size_t ws_bytes, void* stream) {
  kvq_status st = prefix_config(cfg, n_groups, 0);
  if (st != KVQ_OK) return st;
  if (layer0 < 0 || n_layers < 1 || n_layers > cfg->L - layer0)
    return fail(KVQ_ERR_ARG, "layers [%d, +%d) outside [0, %d)", layer0, n_layers, cfg->L);
  if ((st = check_rows(cfg, total_q, max_q, max_group_q)) != KVQ_OK) return st;
  if (total_q > 0 && (!q || !out)) return fail(KVQ_ERR_ARG, "q / out is NULL");
  if (((uintptr_t)q | (uintptr_t)out) & 15u) return fail(KVQ_ERR_ARG, "q / out must be 16-byte aligned");
  {
    const uintptr_t bytes = (uintptr_t)2 * n_layers * total_q * cfg->H_q * cfg->D, x = (uintptr_t)q, y = (uintptr_t)out;
    if (total_q > 0 && x < y + bytes && y < x + bytes) return fail(KVQ_ERR_ARG, "q and out overlap");
  }
  ChunkArgs a{};
  if ((st = cache_ptrs(cfg, cache, &a.cp)) != KVQ_OK) return st;
  const int64_t rows = (int64_t)n_layers * total_q;
  if (rows > 0x7fffffff) return fail(KVQ_ERR_UNSUPPORTED, "%d layers of %d rows", n_layers, total_q);
  if ((st = check_prefix_ws(cfg, n_groups, rows, workspace, ws_bytes)) != KVQ_OK) return st;
  if (total_q == 0 || max_q == 0) return ok();
  a.lo = make_layout(cfg);
  a.layer0 = layer0;
  a.n_layers = n_layers;
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.total_q = total_q;
  a.max_q = max_q;
  const int grid = chunk_workspace(cfg, workspace, &a);
  const PrefixWs w = prefix_ws(cfg, n_groups, rows);
  a.segs = (const Segment*)((char*)workspace + w.segs);
  a.rows = (float*)((char*)workspace + w.rows);
  a.n_groups = n_groups;
  a.max_group_q = max_group_q;
  int mode;
  // owners: sequences and prefixes, and the rows of the prefixes' row tiles once more
  const int64_t owners = (int64_t)cfg->batch + n_groups + (int64_t)total_q * a.lo.g / 128;
  if ((st = chunk_common(cfg, &a, max_group_q, owners, &mode)) != KVQ_OK) return st;
  cudaError_t e = mode == kChunkFew ? launch_prefix_few(a, grid, (cudaStream_t)stream)
                  : cfg->D == 128   ? launch_prefix_d128(a, mode, grid, (cudaStream_t)stream)
                                    : launch_prefix_d256(a, grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefix attention kernels");
  return ok();
}

}  // extern "C"
