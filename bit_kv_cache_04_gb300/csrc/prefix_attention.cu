// kvq_prefix_attention: attention of the newest tokens of every sequence where groups of sequences hold the same
// pages for a common prefix.
//
// A group's rows are the new tokens of all its sequences times the query heads of a kv head.  A unit of work is a row tile of
// them over the tokens [0, P) that the group shares, which all of the rows see, and then over the tiles that each of its
// sequences has behind P, which only that sequence's rows see (the others' scores are -inf there).  So the shared packed tokens are read,
// dequantized and multiplied once for all rows of the tile instead of once a sequence, and a row's softmax runs over both parts
// like over any other tiles: no second pass joins them.  The chunk attention kernel (chunk_kernel.cuh, SEG) takes
// the units in place of its own.
// (First built as two units a row, prefix and own tokens, joined by a pass of its own: a unit of one tile of own tokens took
// 13 us of latency, and 8 x 8 beams over prompts of up to 8192 tokens with 16-bit windows 467 us.)
//
// On one GB300, plan and attention of one layer: 4 beams over 4096 tokens 28.8 us, 8 x 8 beams over prompts of up to 8192 tokens with 16-bit windows 185 us
// (the chunk attention of each sequence 532 us), drafts of up to 4 tokens of 32 chats over 32768 tokens 212 us (767 us), 16 questions
// of up to 200 tokens over 12007 tokens of 256-channel heads 1219 us (1271 us).  The plan takes 6 to 13 us of that (8 to 17 us by itself), a chain of
// dependent steps in one block.  Single tokens can also go through the single-token decode, every sequence by itself, its shared pages from the L2: layer by
// layer that is faster for few sequences behind short prompts (4 beams over 4096 tokens 17 us against 21.5 us and a plan for all layers, 16
// beams 45 against 60 us) and slower for many (4 x 16 beams over 16384 tokens 344 against 106 us).
// What bounds the attention is latency between dependent steps, as in the chunk attention: a CTA's tile takes 2 us, whether all its rows see it or one
// sequence's do; with few tiles, the 20 to 30 us that a run's start and its join cost.
//
// The prefix is what the block table says: the pages that the group's sequences hold in the same places, as far as
// they are quantized in all of them and before every new token, in whole tiles.  kvq_prefix_plan finds it and writes the units
// and the list of own tiles, on the device.
#include <algorithm>
#include <climits>

#include "chunk_attention.cuh"
#include "kvq_host.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
// A unit's start (queries, first scores, outputs) against a tile's time, as places on the line.  With 4 and 8 of them 64 units over 8 prompts of 8192 tokens took
// 84 and 98 us (128 tokens of their own) or 129 and 117 us (512), drafts of 32 chats 212 and 210 us; with 2 the drafts 221 us.
constexpr int kUnitCost = 4;
constexpr int kPlanSmall = 1024;  // sequences whose state fits shared memory; more have it in the workspace

// What the plan keeps of every sequence.
struct SeqState {
  int32_t *cu, *lens, *n;  // first row; length and new tokens of those that take part, else 0
  int32_t *owner_n;        // tokens of the rows that begin with this sequence: its own, its group's, or 0
  int32_t *owner_p;        // the prefix that its group shares
  int32_t *owner_end;      // the sequence behind the last one of the rows
  int32_t *unit_at;        // its first unit
};
constexpr int kSeqWords = 7;

struct PlanArgs {
  Layout lo;
  const int32_t* table;
  const int32_t* cu_groups;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int n_groups, total_q, max_q, max_group_q, tile_log, row_log, n_units, own_tiles, columns;  // (logarithms of tokens a tile, rows a row tile)
  uint32_t g_magic;  // floor(2^32 / g) + 1
  uint32_t* status;
  int32_t* plan;     // total_q, max_q, max_group_q, n_groups
  uint32_t* ticket;  // blocks that are done; zero between calls
  int32_t* parts;    // [n_groups] INT_MAX less the first column where the group's sequences part, 0: none; zero between calls
  int32_t* lens;     // [batch] as SeqState's, for the attention
  int32_t* seqs;     // [kSeqWords][batch], large batches
  int2* where;
  SharedUnit* units;
  OwnTile* own;
};

__device__ __forceinline__ int ceil_shift(int a, int log) { return (a + (1 << log) - 1) >> log; }
// r / g (r < 2^28)
__device__ __forceinline__ int token_of(const PlanArgs& a, int r) { return a.lo.g == 1 ? r : (int)__umulhi((uint32_t)r, a.g_magic); }
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }

// New tokens of sequence b (0: none, or its rows or length are out of order, which sets *bad), its first row and length.
__device__ __forceinline__ int new_tokens(const PlanArgs& a, int b, int* cu, int* T, bool* bad) {
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], t = a.seq_lens[b], n = (int)((uint32_t)c1 - (uint32_t)c0);
  *cu = c0;
  *T = t;
  if (c0 < 0 || c1 < c0 || c1 > a.total_q || n > a.max_q || t < n || t > a.lo.max_T) {
    *bad = true;
    return 0;
  }
  return n;
}

// Group g's part of the table, columns [j0, j1): the first one where its sequences with new tokens do not hold the same page.
__device__ __forceinline__ void find_parting(const PlanArgs& a, int g, int j0, int j1) {
  __shared__ int limit, first, live, found;
  const int tid = threadIdx.x, mp = a.lo.max_pages, b0 = a.cu_groups[g], b1 = a.cu_groups[g + 1];
  if (tid == 0) {
    limit = first = found = INT_MAX;
    live = 0;
  }
  if (b0 < 0 || b1 < b0 || b1 > a.lo.B) return;  // (uniform; the last block says so)
  __syncthreads();
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    int cu, T;
    bool bad = false;
    const int n = new_tokens(a, b, &cu, &T, &bad);
    if (n == 0) continue;
    atomicMin(&limit, min(q_end_of(a.lo, T), T - n));
    atomicMin(&first, b);
    atomicAdd(&live, 1);
  }
  __syncthreads();
  j1 = min(j1, limit / a.lo.pt);
  const int columns = j1 - j0;
  if (live < 2 || columns <= 0) return;
  // threads side by side take columns; few columns: threads share a column's sequences
  const int32_t* ref = a.table + (int64_t)first * mp;
  const int wide = min((columns + 31) & ~31, kPlanThreads), subs = kPlanThreads / wide, sub = tid / wide;
  int mine = INT_MAX;
  if (sub < subs)
    for (int j = j0 + tid % wide; j < j1; j += wide) {
      const int p = ref[j];
      bool same = p >= 0 && p < a.lo.n_pages;
      const int32_t* at = a.table + j;
#pragma unroll 1
      for (int b = first + 1 + sub; b < b1 && same; b += 8 * subs) {
        int v[8];
        bool differ = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = b + i * subs < b1 ? at[(int64_t)(b + i * subs) * mp] : p;
#pragma unroll
        for (int i = 0; i < 8; ++i) differ |= v[i] != p;
        if (differ) {  // (a slot without new tokens has no say)
#pragma unroll 1
          for (int i = b; i < min(b + 8 * subs, b1); i += subs) same &= at[(int64_t)i * mp] == p || a.cu_q[i + 1] == a.cu_q[i];
        }
      }
      if (!same) {
        mine = j;
        break;
      }
    }
  if (mine != INT_MAX) atomicMin(&found, mine);
  __syncthreads();
  if (tid == 0 && found != INT_MAX) atomicMax(a.parts + g, INT_MAX - found);
}

// What group g, sequences [b0, b1), shares: the prefix, and whether taking it in common saves tiles.  A warp.
__device__ __forceinline__ void plan_group(const PlanArgs& a, const SeqState& q, int g, int b0, int b1) {
  const int lane = threadIdx.x & 31, gq = a.lo.g;
  int live = 0, limit = INT_MAX, first = INT_MAX, rows = 0;
  bool bad = false;
  const int parting = __ldcg(a.parts + g);
  for (int b = b0 + lane; b < b1; b += 32) {
    int cu, T;
    const int n = new_tokens(a, b, &cu, &T, &bad);
    q.cu[b] = cu;
    q.n[b] = n;
    q.lens[b] = a.lens[b] = n ? T : 0;
    q.owner_n[b] = n;
    q.owner_p[b] = 0;
    q.owner_end[b] = b + 1;
    if (n) {
      ++live;
      rows += n;
      limit = min(limit, min(q_end_of(a.lo, T), T - n));
      first = min(first, b);
    }
  }
  live = warp_sum(live);
  rows = warp_sum(rows);
  limit = __reduce_min_sync(0xffffffffu, limit);
  first = __reduce_min_sync(0xffffffffu, first);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) a.parts[g] = 0;
  if (!bad && live > 1 && rows > a.max_group_q) bad = true;
  if (bad && lane == 0) atomicOr(a.status, KVQ_DEV_LENGTH);
  // (with a sequence out of order the others' rows need not be one run: they go without a common prefix)
  if (bad || live < 2) return;
  const int pages = min(parting ? INT_MAX - parting : INT_MAX, limit / a.lo.pt);
  const int tiles_p = (int)((int64_t)pages * a.lo.pt >> a.tile_log), P = tiles_p << a.tile_log;
  if (P == 0) return;
  // tiles taken apart (row tiles of each sequence over all it has cached), and together
  __syncwarp();
  const int cu0 = q.cu[first];
  int64_t apart = 0, together = 0;
  for (int b = b0 + lane; b < b1; b += 32) {
    const int n = q.n[b];
    if (!n) continue;
    const int tiles = ceil_shift(q.lens[b], a.tile_log), r0 = (q.cu[b] - cu0) * gq, r1 = r0 + n * gq;
    apart += (int64_t)ceil_shift(n * gq, a.row_log) * tiles;
    together += (int64_t)(((r1 - 1) >> a.row_log) - (r0 >> a.row_log) + 1) * (tiles - tiles_p);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    apart += __shfl_xor_sync(0xffffffffu, apart, o);
    together += __shfl_xor_sync(0xffffffffu, together, o);
  }
  together += (int64_t)ceil_shift(rows * gq, a.row_log) * tiles_p;
  if (together >= apart) return;
  for (int b = b0 + lane; b < b1; b += 32) {
    q.owner_n[b] = b == first ? rows : 0;
    q.owner_p[b] = b == first ? P : 0;
    q.owner_end[b] = b1;
  }
}

// Row tile k of the rows that begin with sequence b0, unit i: its rows, prefix and own tiles.  A warp.
__device__ __forceinline__ void plan_unit(const PlanArgs& a, const SeqState& q, int i, int b0, int k, int* own_count) {
  const int lane = threadIdx.x & 31, gq = a.lo.g, shared = q.owner_p[b0], end = q.owner_end[b0];
  SharedUnit u;
  u.cu = q.cu[b0];
  u.first = b0;
  u.r0 = k << a.row_log;
  u.rows = min(1 << a.row_log, q.owner_n[b0] * gq - u.r0);
  const int tok0 = token_of(a, u.r0), tok1 = token_of(a, u.r0 + u.rows - 1);  // of the owner's
  if (shared)
    u.prefix = shared;
  else  // one sequence: what all of the rows see of it in the packed tiers
    u.prefix = min(q_end_of(a.lo, q.lens[b0]), q.lens[b0] - q.n[b0] + tok0 + 1) >> a.tile_log << a.tile_log;
  auto tiles_of = [&](int b, int* p_lo, int* rows) {
    if (b >= end || !q.n[b]) return 0;
    const int off = q.cu[b] - u.cu, n = q.n[b], T = q.lens[b], t0 = max(tok0, off), t1 = min(tok1, off + n - 1);
    if (t0 > t1) return 0;
    *rows = max(0, off * gq - u.r0) | min(u.rows, (off + n) * gq - u.r0) << 16;
    *p_lo = T - n + t0 - off;
    return ((T - n + t1 - off) >> a.tile_log) - (u.prefix >> a.tile_log) + 1;
  };
  int total = 0, low = INT_MAX, tiles = 0, rows = 0;  // (the last turn's are kept: mostly it is the only one)
#pragma unroll 1
  for (int b = b0 + lane; b - lane < end; b += 32) {
    int p = INT_MAX;
    tiles = tiles_of(b, &p, &rows);
    total += tiles;
    low = min(low, p);
  }
  u.n_own = total = warp_sum(total);
  u.p_lo = __reduce_min_sync(0xffffffffu, low);
  int at = 0;
  if (lane == 0) at = atomicAdd(own_count, total);  // (which places a unit gets changes no result)
  u.own = at = __shfl_sync(0xffffffffu, at, 0);
  if (at > a.own_tiles - total) u.rows = 0;  // (the list holds all that lengths up to max_T need)
  if (lane == 0) a.units[i] = u;
  if (u.rows == 0) return;
#pragma unroll 1
  for (int b = b0 + lane; b - lane < end; b += 32) {
    int p;
    if (end - b0 > 32) tiles = tiles_of(b, &p, &rows);
    // lanes' tiles one behind the other, each written by its lane
    int before = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    const int T = b < end ? q.lens[b] : 0;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) a.own[at + before - tiles + t] = OwnTile{b, u.prefix + (t << a.tile_log), T, rows};
    at += __shfl_sync(0xffffffffu, before, 31);
  }
}

// Grid (groups, runs of table columns); the last block to finish writes the plan.  The attention is let go at this grid's end: begun while the attention before
// still ran, an SM could have that one's table entries in its first-level cache.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ bool last;
  __shared__ int scan[kPlanWarps], own_count;
  __shared__ int32_t small[kSeqWords][kPlanSmall];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.lo.B;
  grid_dependency_wait();
  find_parting(a, blockIdx.x, blockIdx.y * a.columns, (blockIdx.y + 1) * a.columns);
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
    own_count = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // the groups cover the batch, in order
  bool wrong = false;
  for (int i = tid; i <= a.n_groups; i += kPlanThreads) {
    const int at = a.cu_groups[i];
    wrong |= i == 0 ? at != 0 : at < a.cu_groups[i - 1];
    if (i == a.n_groups) wrong |= at != B;
  }
  const bool in_order = !__syncthreads_or(wrong);
  if (tid == 0) {
    *a.ticket = 0;
    a.plan[0] = a.total_q;
    a.plan[1] = a.max_q;
    a.plan[2] = a.max_group_q;
    a.plan[3] = a.n_groups;
    const uint32_t bad = !in_order ? KVQ_DEV_SEQ : a.cu_q[0] != 0 ? KVQ_DEV_LENGTH : 0;
    if (bad) atomicOr(a.status, bad);
  }
  int units = 0;
  if (in_order) {
    SeqState q;
    int32_t** const field[kSeqWords] = {&q.cu, &q.lens, &q.n, &q.owner_n, &q.owner_p, &q.owner_end, &q.unit_at};
#pragma unroll
    for (int i = 0; i < kSeqWords; ++i) *field[i] = B <= kPlanSmall ? small[i] : a.seqs + (int64_t)i * B;
    for (int g = warp; g < a.n_groups; g += kPlanWarps) plan_group(a, q, g, a.cu_groups[g], a.cu_groups[g + 1]);
    __syncthreads();
    // every owner's row tiles
    for (int base = 0; base < B; base += kPlanThreads) {
      const int b = base + tid, mine = b < B ? ceil_shift(q.owner_n[b] * a.lo.g, a.row_log) : 0;
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      const int s = scan[lane], before = warp_sum(lane < warp ? s : 0);
      if (b < B) q.unit_at[b] = units + before + x - mine;
      units += warp_sum(s);
    }
    units = min(units, a.n_units);
    __syncthreads();
    for (int i = warp; i < units; i += kPlanWarps) {
      int lo = 0, hi = B;  // the last sequence whose units begin at or before i: it has some
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (q.unit_at[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      plan_unit(a, q, i, lo, i - q.unit_at[lo], &own_count);
    }
    // positions and sequences of the rows
    for (int b = warp; b < B; b += kPlanWarps) {
      const int n = q.n[b], cu = q.cu[b], p = q.lens[b] - n;
      for (int i = lane; i < n; i += 32) a.where[cu + i] = make_int2(p + i, b);
    }
  } else {
    for (int g = tid; g < a.n_groups; g += kPlanThreads) a.parts[g] = 0;
  }
  for (int i = units + tid; i < a.n_units; i += kPlanThreads) a.units[i] = SharedUnit{};
}

// Workspace: that of the chunk attention, then the plan.
struct PrefixWs {
  size_t plan, parts, lens, seqs, where, units, own, total, zeroed;
  int n_units, own_tiles;
};
kvq_status prefix_ws(const kvq_config* c, int n_groups, int64_t rows, PrefixWs* out) {
  PrefixWs w{};
  const int64_t g = c->H_q / c->H_kv, tiles = c->max_T / chunk_tile(c->D) + 2;
  const int64_t units = rows * g / 128 + c->batch, own = (units + c->batch) * tiles;
  if (units > 1 << 24 || own > 1 << 28) return fail(KVQ_ERR_UNSUPPORTED, "a plan of %lld row tiles over %lld tiles", (long long)units, (long long)own);
  w.n_units = (int)units;
  w.own_tiles = (int)own;
  w.plan = align_up(chunk_workspace_bytes(c, &w.zeroed));
  w.parts = w.plan + kWsAlign;
  w.lens = w.parts + align_up(sizeof(int32_t) * (size_t)n_groups);
  w.seqs = w.lens + align_up(sizeof(int32_t) * (size_t)c->batch);
  w.where = w.seqs + (c->batch > kPlanSmall ? align_up(sizeof(int32_t) * kSeqWords * (size_t)c->batch) : 0);
  w.units = w.where + align_up(sizeof(int2) * (size_t)rows);
  w.own = w.units + align_up(sizeof(SharedUnit) * (size_t)units);
  w.total = w.own + align_up(sizeof(OwnTile) * (size_t)own);
  *out = w;
  return KVQ_OK;
}

kvq_status prefix_config(const kvq_config* cfg, int32_t n_groups, int64_t rows) {
  const kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (cfg->page_tokens < 1) return fail(KVQ_ERR_ARG, "the cache is not paged");
  if (n_groups < 1 || n_groups > cfg->batch) return fail(KVQ_ERR_ARG, "n_groups=%d not in [1, batch=%d]", n_groups, cfg->batch);
  if (rows < 0 || rows > 0x7fffffff) return fail(KVQ_ERR_ARG, "rows=%lld", (long long)rows);
  return KVQ_OK;
}

kvq_status check_prefix_ws(const kvq_config* cfg, int32_t n_groups, int64_t rows, void* ws, size_t bytes, PrefixWs* w) {
  if (!ws) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  const kvq_status st = prefix_ws(cfg, n_groups, rows, w);
  if (st != KVQ_OK) return st;
  if (bytes < w->total) return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", bytes, w->total);
  if (((uintptr_t)ws) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return KVQ_OK;
}

kvq_status check_rows(const kvq_config* cfg, int32_t total_q, int32_t max_q, int32_t max_group_q) {
  if (total_q < 0 || max_q < 0 || max_group_q < max_q || max_group_q > total_q)
    return fail(KVQ_ERR_ARG, "total_q=%d, max_q=%d, max_group_q=%d", total_q, max_q, max_group_q);
  if (max_q > cfg->max_T) return fail(KVQ_ERR_CAPACITY, "max_q=%d > max_T=%d", max_q, cfg->max_T);
  if ((int64_t)max_group_q * (cfg->H_q / cfg->H_kv) > 1 << 28) return fail(KVQ_ERR_UNSUPPORTED, "max_group_q=%d", max_group_q);
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_prefix_workspace_bytes(const kvq_config* cfg, int32_t n_groups, int32_t rows, size_t* bytes) {
  kvq_status st = prefix_config(cfg, n_groups, rows);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  PrefixWs w;
  if ((st = prefix_ws(cfg, n_groups, rows, &w)) != KVQ_OK) return st;
  *bytes = w.total;
  return ok();
}

kvq_status kvq_prefix_workspace_init(const kvq_config* cfg, int32_t n_groups, int32_t rows, void* workspace, size_t ws_bytes,
                                     void* stream) {
  kvq_status st = prefix_config(cfg, n_groups, rows);
  if (st != KVQ_OK) return st;
  PrefixWs w;
  if ((st = check_prefix_ws(cfg, n_groups, rows, workspace, ws_bytes, &w)) != KVQ_OK) return st;
  cudaError_t e = cudaMemsetAsync(workspace, 0, w.zeroed, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemsetAsync((char*)workspace + w.plan, 0, w.own - w.plan, (cudaStream_t)stream);
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
  PrefixWs w;
  if ((st = check_prefix_ws(cfg, n_groups, total_q, workspace, ws_bytes, &w)) != KVQ_OK) return st;
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
  a.tile_log = chunk_tile(cfg->D) == 128 ? 7 : 6;
  a.row_log = chunk_form(cfg, (int64_t)max_group_q * a.lo.g) == kChunkPaired ? 8 : 7;
  a.g_magic = (uint32_t)((1ull << 32) / a.lo.g + 1);
  a.n_units = w.n_units;
  a.own_tiles = w.own_tiles;
  char* base = (char*)workspace;
  a.status = (uint32_t*)workspace;
  a.plan = (int32_t*)(base + w.plan);
  a.ticket = (uint32_t*)(base + w.plan) + 4;
  a.parts = (int32_t*)(base + w.parts);
  a.lens = (int32_t*)(base + w.lens);
  a.seqs = (int32_t*)(base + w.seqs);
  a.where = (int2*)(base + w.where);
  a.units = (SharedUnit*)(base + w.units);
  a.own = (OwnTile*)(base + w.own);
  // columns of a block: 256, more where that would be more than two blocks an SM
  const int64_t all = (int64_t)cfg->max_T / cfg->page_tokens + 1, most = std::max<int64_t>(1, 2 * (int64_t)sm_count() / n_groups);
  a.columns = (int)std::max<int64_t>(256, (all + most - 1) / most);
  const unsigned runs = (unsigned)((all + a.columns - 1) / a.columns);
  const cudaError_t e = launch_dependent(prefix_plan_kernel, dim3(n_groups, runs), dim3(kPlanThreads), 0, (cudaStream_t)stream, a);
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
  PrefixWs w;
  if ((st = check_prefix_ws(cfg, n_groups, total_q, workspace, ws_bytes, &w)) != KVQ_OK) return st;
  if (total_q == 0 || max_q == 0) return ok();
  a.lo = make_layout(cfg);
  a.layer0 = layer0;
  a.n_layers = n_layers;
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.total_q = total_q;
  a.max_q = max_q;
  const int grid = chunk_workspace(cfg, workspace, &a);
  a.unit_cost = kUnitCost;
  // the kernel counts its tiles in 32 bits: prefixes of all units, the own tiles, and what a unit costs besides
  const int64_t line = (int64_t)w.n_units * (cfg->max_T / chunk_tile(cfg->D) + a.unit_cost) + w.own_tiles;
  if (line * n_layers * cfg->H_kv > 0x7fffffff - 2 * grid)
    return fail(KVQ_ERR_UNSUPPORTED, "too many tiles for one call: pass fewer layers or rows");
  int mode;
  if ((st = chunk_common(cfg, &a, max_group_q, cfg->batch, &mode)) != KVQ_OK) return st;
  a.by_warp = 0;
  const char* base = (const char*)workspace;
  a.plan = (const int32_t*)(base + w.plan);
  a.lens = (const int32_t*)(base + w.lens);
  a.where = (const int2*)(base + w.where);
  a.units = (const SharedUnit*)(base + w.units);
  a.own = (const OwnTile*)(base + w.own);
  a.n_units = w.n_units;
  a.own_tiles = w.own_tiles;
  a.n_groups = n_groups;
  a.max_group_q = max_group_q;
  a.most_rows = mode == kChunkFew ? a.cols : mode == kChunkPaired ? 256 : 128;
  cudaError_t e = mode == kChunkFew ? launch_prefix_few(a, grid, (cudaStream_t)stream)
                  : cfg->D == 128   ? launch_prefix_d128(a, mode, grid, (cudaStream_t)stream)
                                    : launch_prefix_d256(a, grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefix attention kernels");
  return ok();
}

}  // extern "C"
