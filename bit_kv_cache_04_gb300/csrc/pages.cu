// Pages of a paged cache: counts, release, fork, reserve (with a private copy
// of a shared, partly filled page), reorder and compaction.
//
// The bookkeeping is integers: a few thousand table entries and counts, so
// one block decides (its passes over refs are the only ones longer than the
// lists), and launch latency is what these calls cost: a reservation for 64
// sequences 9 us, for 256 of them 23 us (32 us with a copy for every second one), compaction of 6000 pages' counts 6 us.
// Beyond that the one block shows: 1024 sequences 76 us (108 us), 4096 298 us (524 us), 32768 2.6 ms (13 ms: the ranks
// among sequences that share a page are quadratic); 65536 pages 42 us, 2^20 614 us.  The bytes that have to move (shared
// pages that get written, windows of forked sequences, compacted pages) are
// copied by a second, grid-wide kernel that reads the decision from the
// workspace: 2 bytes of traffic per byte moved, HBM-bound (6000 pages half used compacted in 288 us, 83 % of the copy
// rate; two prompts forked twice, 14 us of dependent launches).  A reordering needs no plan: every group's columns are its own, a block for 128 of
// them (4 beams of 4099 tokens 6.2 us); the windows, one read and one write for each slot that changes, go at 93 to 97 % of the copy rate (16 x 8 beams
// with 128 tokens in 16 layers, 225 to 235 us).
#include <algorithm>

#include "kvq_host.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxPageBatch = 32768;
constexpr int kMaxReorder = 32;  // slots of a group
constexpr int kReorderThreads = 128;

// Workspace (int32 words after the status block): header, then arrays.
struct PagesWs {
  uint32_t* status;
  int32_t* n_moves;  // pages to copy
  int32_t* mark;     // [batch] 1 while a sequence is in the current list; reorder: a group's blocks that have begun; zero between calls
  int32_t* src;      // [n] moves: page copied from
  int32_t* dst;      // [n] and to
  int32_t* map;      // [n_pages] compact: new id, or -1 of a free page
  int32_t* fork_ok;  // [batch] fork: pair accepted
  int32_t* shared;   // [batch] reserve: the page a listed sequence has to copy, or -1
  int32_t* first;    // [batch] reserve: needed pages, then their offset in `free_list`
  int32_t* free_list;  // [n_pages]
};

struct PagesArgs {
  Layout lo;
  CachePtrs cp;
  PagesWs ws;
  int32_t* table;
  int32_t* refs;
  int32_t* seq_lens;
  const int32_t* seqs;   // release, reserve; fork: sources
  const int32_t* other;  // reserve: n_new; fork: targets
  int n;
  int32_t* table_out;
  int32_t* refs_out;
};

size_t pages_ws_layout(const kvq_config* c, void* base, PagesWs* w) {
  const size_t moves = (size_t)std::max(c->n_pages, c->batch);
  size_t off = kWsAlign;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = align_up(off + sizeof(int32_t) * n);
    return base ? (int32_t*)((char*)base + at) : nullptr;
  };
  PagesWs r{};
  r.status = (uint32_t*)base;
  r.n_moves = take(1);
  r.mark = take(c->batch);
  r.src = take(moves);
  r.dst = take(moves);
  r.map = take(c->n_pages);
  r.fork_ok = take(c->batch);
  r.shared = take(c->batch);
  r.first = take(c->batch);
  r.free_list = take(c->n_pages);
  if (w) *w = r;
  return off;
}

// Kernels here that change the table or the lengths let the stream's next kernel go at their ends only.  The chunk attention reads both with
// non-coherent loads: begun while an attention before these calls still ran, it could find in an SM's first-level cache what that one had read there
// since.  (A kernel behind such an end begins after it, and may let the next one go at its start.)

// ---- counts -----------------------------------------------------------------

__global__ void count_refs_kernel(PagesArgs a) {
  const int64_t total = (int64_t)a.lo.B * a.lo.max_pages;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total; e += (int64_t)gridDim.x * blockDim.x) {
    const int p = a.table[e];
    if (p == -1) continue;
    if (p < 0 || p >= a.lo.n_pages)
      atomicOr(a.ws.status, KVQ_DEV_PAGE);
    else
      atomicAdd(a.refs + p, 1);
  }
}

// ---- release -------------------------------------------------------------------

// One block per listed sequence.  The exchange makes a second listing of the
// same sequence find -1 everywhere, whichever block is first.
__global__ void release_kernel(PagesArgs a) {
  grid_dependency_wait();
  const int s = a.seqs[blockIdx.x];
  if (s < 0 || s >= a.lo.B) {
    if (threadIdx.x == 0) atomicOr(a.ws.status, KVQ_DEV_SEQ);
    return;
  }
  int32_t* row = a.table + (int64_t)s * a.lo.max_pages;
  for (int j = threadIdx.x; j < a.lo.max_pages; j += blockDim.x) {
    if (row[j] == -1) continue;
    const int p = atomicExch(row + j, -1);
    if (p == -1) continue;
    if (p < 0 || p >= a.lo.n_pages) {
      atomicOr(a.ws.status, KVQ_DEV_PAGE);
    } else if (atomicSub(a.refs + p, 1) <= 0) {
      atomicAdd(a.refs + p, 1);
      atomicOr(a.ws.status, KVQ_DEV_PAGE);
    }
  }
  if (threadIdx.x == 0) a.seq_lens[s] = 0;
}

// ---- fork ----------------------------------------------------------------------

// One block per pair.  Every accepted target is empty, listed by no earlier
// pair and no pair's source, so no block writes what another one reads.
__global__ void fork_kernel(PagesArgs a) {
  grid_dependency_wait();
  const int i = blockIdx.x, mp = a.lo.max_pages;
  const int s = a.seqs[i], d = a.other[i];
  bool bad = s < 0 || s >= a.lo.B || d < 0 || d >= a.lo.B || s == d;
  for (int j = threadIdx.x; j < a.n; j += blockDim.x)
    bad |= (j < i && a.other[j] == d) || a.other[j] == s || a.seqs[j] == d;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      atomicOr(a.ws.status, KVQ_DEV_SEQ);
      a.ws.fork_ok[i] = 0;
    }
    return;
  }
  const int32_t* from = a.table + (int64_t)s * mp;
  int32_t* to = a.table + (int64_t)d * mp;
  const int T = a.seq_lens[s];
  bool full = threadIdx.x == 0 && a.seq_lens[d] != 0;
  for (int j = threadIdx.x; j < mp; j += blockDim.x) full |= to[j] != -1;
  const bool bad_len = T < 0 || T > a.lo.max_T;
  const int qe = bad_len ? 0 : q_end_of(a.lo, T);
  const int share = (int)(((int64_t)qe + a.lo.pt - 1) / a.lo.pt);
  bool bad_page = false;
  for (int j = threadIdx.x; j < share; j += blockDim.x) bad_page |= from[j] < 0 || from[j] >= a.lo.n_pages;
  const int any_full = __syncthreads_or(full), any_page = __syncthreads_or(bad_page);
  if (any_full || any_page || bad_len) {
    if (threadIdx.x == 0) {
      atomicOr(a.ws.status, any_full ? KVQ_DEV_SEQ : bad_len ? KVQ_DEV_LENGTH : KVQ_DEV_PAGE);
      a.ws.fork_ok[i] = 0;
    }
    return;
  }
  for (int j = threadIdx.x; j < share; j += blockDim.x) {
    const int p = from[j];
    to[j] = p;
    atomicAdd(a.refs + p, 1);
  }
  if (threadIdx.x == 0) {
    a.seq_lens[d] = T;
    a.ws.fork_ok[i] = 1;
  }
}

// The 16-bit windows of accepted pairs: block (pair, layer, K or V and part).
__global__ void fork_window_kernel(PagesArgs a, int parts) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int i = blockIdx.x;
  if (!a.ws.fork_ok[i]) return;
  const int which = blockIdx.z / parts, part = blockIdx.z % parts;
  const int64_t unit = (int64_t)a.lo.H * a.lo.ring * a.lo.D / 8;  // 16-byte words of one (layer, sequence)
  uint4* base = reinterpret_cast<uint4*>(which ? a.cp.v_resid : a.cp.k_resid);
  [[maybe_unused]] const CachePtrs& cp = a.cp;
  if (!KVQ_CHECK((int)blockIdx.y < a.lo.L && (uint32_t)a.seqs[i] < (uint32_t)a.lo.B && (uint32_t)a.other[i] < (uint32_t)a.lo.B))
    return;
  const uint4* from = base + ((int64_t)blockIdx.y * a.lo.B + a.seqs[i]) * unit;
  uint4* to = base + ((int64_t)blockIdx.y * a.lo.B + a.other[i]) * unit;
  const int64_t per = (unit + parts - 1) / parts, e1 = min(unit, (part + 1) * per);
  int64_t e = part * per + threadIdx.x;
  for (; e + 3 * (int64_t)blockDim.x < e1; e += 4 * (int64_t)blockDim.x) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = from[e + k * (int64_t)blockDim.x];
#pragma unroll
    for (int k = 0; k < 4; ++k) to[e + k * (int64_t)blockDim.x] = v[k];
  }
  for (; e < e1; e += blockDim.x) to[e] = from[e];
}

// ---- reserve -----------------------------------------------------------------

// Exclusive prefix sum of v over the block's threads; *total gets the sum.
__device__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums may still be read from the last call
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return (warp ? warp_sums[warp - 1] : 0) + x - v;
}

// What sequence s needs for nn more tokens: the slot of the partly filled page its next
// quantized token goes to (or -1), and the slots [s0, s1) that must hold pages.
struct Need {
  int partial, s0, s1;
};
__device__ __forceinline__ Need need_of(const Layout& lo, int T, int nn) {
  const int qe = q_end_of(lo, T);
  Need r;
  r.partial = qe % lo.pt && nn > 0 ? qe / lo.pt : -1;
  r.s0 = (int)(((int64_t)qe + lo.pt - 1) / lo.pt);
  r.s1 = nn > 0 ? (int)(((int64_t)T + nn + lo.pt - 1) / lo.pt) : r.s0;
  return r;
}

// One block; a warp per listed sequence.
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(PagesArgs a) {
  extern __shared__ int32_t shared_page[];  // [n] page to copy, or -1
  __shared__ int warp_sums[32];
  __shared__ uint32_t err;
  __shared__ int found;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = kPlanThreads / 32;
  const int n = a.n, mp = a.lo.max_pages;
  if (threadIdx.x == 0) {
    err = 0;
    found = 0;
    *a.ws.n_moves = 0;
  }
  __syncthreads();
  // every sequence's checks, its partly filled shared page, and the pages it lacks
  for (int i = warp; i < n; i += nw) {
    const int s = a.seqs[i], nn = a.other[i];
    uint32_t bad = 0;
    int page = -1, missing = 0;
    if (s < 0 || s >= a.lo.B) {
      bad = KVQ_DEV_SEQ;
    } else {
      int before = 0;
      if (lane == 0) before = atomicExch(a.ws.mark + s, 1);
      if (__shfl_sync(0xffffffffu, before, 0)) bad = KVQ_DEV_SEQ;
      const int T = a.seq_lens[s];
      if (T < 0 || T > a.lo.max_T || nn < 0)
        bad |= KVQ_DEV_LENGTH;
      else if (nn > a.lo.max_T - T)
        bad |= KVQ_DEV_CAPACITY;
      if (!bad) {
        const int32_t* row = a.table + (int64_t)s * mp;
        const Need w = need_of(a.lo, T, nn);
        if (w.partial >= 0) {
          const int p = row[w.partial];
          if (p < 0 || p >= a.lo.n_pages || a.refs[p] < 1)
            bad |= KVQ_DEV_PAGE;
          else if (a.refs[p] > 1)
            page = p;
        }
        for (int j = w.s0 + lane; j < w.s1; j += 32) {
          const int p = row[j];
          if (p == -1)
            ++missing;
          else if (p < 0 || p >= a.lo.n_pages || a.refs[p] != 1)  // the next pages are the sequence's own
            bad |= KVQ_DEV_PAGE;
        }
        missing = __reduce_add_sync(0xffffffffu, missing);
        bad = __reduce_or_sync(0xffffffffu, bad);
      }
    }
    if (lane == 0) {
      if (bad) atomicOr(&err, bad);
      shared_page[i] = page;
      a.ws.first[i] = missing;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = a.seqs[i];
    if (s >= 0 && s < a.lo.B) a.ws.mark[s] = 0;
  }
  if (err) {  // uniform: nothing is changed
    if (threadIdx.x == 0) atomicOr(a.ws.status, err);
    return;
  }
  // in list order, all readers but the last one left copy: the rank among
  // the earlier sequences that have the same page decides
  for (int i = warp; i < n; i += nw) {
    const int p = shared_page[i];
    int copy = 0;
    if (p >= 0) {
      int rank = 0;
      for (int j = lane; j < i; j += 32) rank += shared_page[j] == p;
      rank = __reduce_add_sync(0xffffffffu, rank);
      copy = rank < a.refs[p] - 1;
    }
    if (lane == 0) a.ws.shared[i] = copy ? p : -1;
  }
  __syncthreads();
  // offsets of every sequence's new pages and of its copy
  int pages = 0, copies = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int copy = i < n && a.ws.shared[i] >= 0, need = i < n ? a.ws.first[i] + copy : 0;
    int sum;
    const int at = block_scan(need, warp_sums, &sum);
    int csum;
    const int cat = block_scan(copy, warp_sums, &csum);
    if (i < n) {
      a.ws.first[i] = pages + at;
      if (copy) {
        a.ws.src[copies + cat] = a.ws.shared[i];
        a.ws.dst[copies + cat] = pages + at;  // place in the free list, replaced below
      }
    }
    pages += sum;
    copies += csum;
  }
  // the lowest free pages, until there are enough
  for (int p0 = 0; p0 < a.lo.n_pages && found < pages; p0 += kPlanThreads) {
    const int p = p0 + threadIdx.x;
    const int is_free = p < a.lo.n_pages && a.refs[p] == 0;
    int sum;
    const int at = found + block_scan(is_free, warp_sums, &sum);
    if (is_free && at < pages) a.ws.free_list[at] = p;
    __syncthreads();
    if (threadIdx.x == 0) found += sum;
    __syncthreads();
  }
  if (found < pages) {
    if (threadIdx.x == 0) atomicOr(a.ws.status, KVQ_DEV_CAPACITY);
    return;
  }
  for (int i = warp; i < n; i += nw) {
    const int s = a.seqs[i];
    int32_t* row = a.table + (int64_t)s * mp;
    const Need w = need_of(a.lo, a.seq_lens[s], a.other[i]);
    int at = a.ws.first[i];
    if (a.ws.shared[i] >= 0) {
      if (lane == 0) {
        const int p = a.ws.free_list[at];
        row[w.partial] = p;
        a.refs[p] = 1;
        atomicSub(a.refs + a.ws.shared[i], 1);
      }
      ++at;
    }
    for (int j0 = w.s0; j0 < w.s1; j0 += 32) {
      const int j = j0 + lane;
      const bool lacks = j < w.s1 && row[j] == -1;
      const uint32_t m = __ballot_sync(0xffffffffu, lacks);
      if (lacks) {
        const int p = a.ws.free_list[at + __popc(m & ((1u << lane) - 1u))];
        row[j] = p;
        a.refs[p] = 1;
      }
      at += __popc(m);
    }
  }
  for (int m = threadIdx.x; m < copies; m += kPlanThreads) a.ws.dst[m] = a.ws.free_list[a.ws.dst[m]];
  if (threadIdx.x == 0) *a.ws.n_moves = copies;
}

// ---- compaction --------------------------------------------------------------------

// One block: counts the used pages, then pairs the k-th used page at or
// beyond the count with the k-th free one below it.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesArgs a) {
  __shared__ int warp_sums[32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int n = a.lo.n_pages;
  int mine = 0, used;
  for (int p = threadIdx.x; p < n; p += kPlanThreads) mine += a.refs[p] > 0;
  block_scan(mine, warp_sums, &used);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < n; p0 += kPlanThreads) {
    const int p = p0 + threadIdx.x;
    const int r = p < n ? a.refs[p] : 0;
    const int hole = p < used && r <= 0, mover = p >= used && p < n && r > 0;
    // one scan for both: a chunk holds at most 1024 of each
    int sum;
    const int at = block_scan(hole + (mover << 16), warp_sums, &sum);
    if (hole) a.ws.dst[holes + (at & 0xffff)] = p;
    if (mover) a.ws.src[movers + (at >> 16)] = p;
    if (p < n) a.ws.map[p] = r > 0 ? p : -1;  // a mover's entry is replaced below
    holes += sum & 0xffff;
    movers += sum >> 16;
  }
  __syncthreads();
  // counts: the moved ones first (their sources may be overwritten when
  // refs_out is refs), then the rest
  for (int m = threadIdx.x; m < movers; m += kPlanThreads) {
    const int s = a.ws.src[m], d = a.ws.dst[m];
    a.ws.map[s] = d;
    a.refs_out[d] = a.refs[s];
    if (a.refs_out == a.refs) a.refs_out[s] = 0;
  }
  if (a.refs_out != a.refs)
    for (int p = threadIdx.x; p < n; p += kPlanThreads) {
      const int r = a.refs[p];
      if (p >= used)
        a.refs_out[p] = 0;
      else if (r > 0)
        a.refs_out[p] = r;
    }
  if (threadIdx.x == 0) *a.ws.n_moves = movers;
}

// ---- reorder -------------------------------------------------------------------------

// A group's slots after a selection: slot b becomes what slot parents[b] was.  Every column of the table (and every
// 16-byte word of the windows) belongs to one thread, which reads all it needs of the group before it writes: no copy
// of the old state is kept.

// The group's parents and lengths into shared memory; 0, or the status bit of what is wrong with them.
__device__ __forceinline__ uint32_t group_state(const PagesArgs& a, int group, int* parent, int* len) {
  bool bad = false, bad_len = false;
  if ((int)threadIdx.x < a.n) {
    const int p = a.other[(int64_t)group * a.n + threadIdx.x], T = a.seq_lens[(int64_t)group * a.n + threadIdx.x];
    parent[threadIdx.x] = p;
    len[threadIdx.x] = T;
    bad = p < 0 || p >= a.n;
    bad_len = T < 0 || T > a.lo.max_T;
  }
  const int any = __syncthreads_or(bad), any_len = __syncthreads_or(bad_len);
  return any ? KVQ_DEV_SEQ : any_len ? KVQ_DEV_LENGTH : 0;
}

// Block (group, run of table columns).  Pages that hold quantized tokens go to all children; pages behind them, taken by a
// reservation, must stay one sequence's own: the heir's, which is the slot itself or else its lowest child.
// A page's count changes by what its entries become, summed over the group's slots that hold it in this column: pages that all of
// them share, the prompt's, take no atomics.
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(PagesArgs a) {
  __shared__ int parent[kMaxReorder], children[kMaxReorder], heir[kMaxReorder], len[kMaxReorder], share[kMaxReorder];
  __shared__ int column[kMaxReorder][kReorderThreads];
  __shared__ bool last;
  grid_dependency_wait();
  const int group = blockIdx.x, K = a.n, mp = a.lo.max_pages;
  if (const uint32_t wrong = group_state(a, group, parent, len)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.ws.status, wrong);
    return;
  }
  if ((int)threadIdx.x < K) {
    int n = 0, low = -1;
    for (int b = K - 1; b >= 0; --b)
      if (parent[b] == (int)threadIdx.x) {
        ++n;
        low = b;
      }
    children[threadIdx.x] = n;
    heir[threadIdx.x] = parent[threadIdx.x] == (int)threadIdx.x ? (int)threadIdx.x : low;
    share[threadIdx.x] = (int)(((int64_t)q_end_of(a.lo, len[threadIdx.x]) + a.lo.pt - 1) / a.lo.pt);
  }
  // the lengths are written by the group's last block: the others have read them
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ws.mark + (int64_t)group * K, 1) == (int)gridDim.y - 1;
  }
  __syncthreads();
  if (last) {
    if (threadIdx.x == 0) a.ws.mark[(int64_t)group * K] = 0;
    if ((int)threadIdx.x < K) a.seq_lens[(int64_t)group * K + threadIdx.x] = len[parent[threadIdx.x]];
  }
  const int j = blockIdx.y * kReorderThreads + threadIdx.x;
  if (j >= mp) return;
  int32_t* at = a.table + (int64_t)group * K * mp + j;
  int* mine = &column[0][threadIdx.x];
  bool same = true;
#pragma unroll 8
  for (int b = 0; b < K; ++b) mine[b * kReorderThreads] = at[(int64_t)b * mp];
  const int p0 = mine[0];
  for (int b = 0; b < K; ++b) same &= mine[b * kReorderThreads] == p0 && (p0 == -1 || j < share[b]);
  if (same && p0 >= -1 && p0 < a.lo.n_pages) return;
  for (int b = 0; b < K; ++b) {
    const int p = mine[b * kReorderThreads];
    if (p == -1) continue;
    if (p < 0 || p >= a.lo.n_pages) {
      atomicOr(a.ws.status, KVQ_DEV_PAGE);
      continue;
    }
    bool again = false;
    int change = 0;
    for (int c = 0; c < K; ++c)
      if (mine[c * kReorderThreads] == p) {
        again |= c < b;
        change += (j < share[c] ? children[c] : children[c] > 0) - 1;
      }
    if (!again && change) atomicAdd(a.refs + p, change);
  }
  for (int b = 0; b < K; ++b) {
    const int s = parent[b];
    if (s != b) at[(int64_t)b * mp] = j < share[s] || heir[s] == b ? mine[s * kReorderThreads] : -1;
  }
}

// The 16-bit windows of one (group, layer, K or V): a thread a word.  Only slots that change are written, and
// only those that they come from are read, each once.  N: sources that fit a thread's registers.
template <int N>
__global__ void __launch_bounds__(kReorderThreads) reorder_window_kernel(PagesArgs a) {
  __shared__ int parent[kMaxReorder], len[kMaxReorder], source[kMaxReorder], first[kMaxReorder + 1], to[kMaxReorder];
  __shared__ int n_sources;
  grid_dependency_wait();
  const int group = blockIdx.z, K = a.n, layer = blockIdx.y >> 1;
  if (group_state(a, group, parent, len)) return;  // (the other kernel has said so; lengths that it has moved are good ones)
  if (threadIdx.x == 0) {  // the moves, by source
    int n = 0, m = 0;
    for (int s = 0; s < K; ++s) {
      const int m0 = m;
      for (int b = 0; b < K; ++b)
        if (parent[b] == s && b != s) to[m++] = b;
      if (m > m0) {
        source[n] = s;
        first[n++] = m0;
      }
    }
    first[n] = m;
    n_sources = n;
  }
  __syncthreads();
  const int64_t unit = (int64_t)a.lo.H * a.lo.ring * a.lo.D / 8;  // 16-byte words of one (layer, sequence)
  [[maybe_unused]] const CachePtrs& cp = a.cp;
  if (!KVQ_CHECK(layer < a.lo.L && (group + 1) * K <= a.lo.B)) return;
  uint4* base = reinterpret_cast<uint4*>(blockIdx.y & 1 ? a.cp.v_resid : a.cp.k_resid) + ((int64_t)layer * a.lo.B + (int64_t)group * K) * unit;
  const int sources = n_sources;
  for (int64_t e = blockIdx.x * (int64_t)kReorderThreads + threadIdx.x; e < unit; e += (int64_t)gridDim.x * kReorderThreads) {
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < sources) v[i] = base[source[i] * unit + e];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < sources)
        for (int m = first[i]; m < first[i + 1]; ++m) base[to[m] * unit + e] = v[i];
  }
}

// ---- copies --------------------------------------------------------------------

// Copies page src[m] to dst[m] for every move, all layers, K and V.  The rows
// of one (layer, page) are one run of bytes; blocks take runs in turn.  V is the widest
// word that divides both runs' bytes.  TABLE: the block table's entries through `map` too.
template <class V, bool TABLE>
__global__ void __launch_bounds__(256) copy_pages_kernel(PagesArgs a, int k_words, int v_words) {
  if constexpr (!TABLE) grid_launch_dependents();
  grid_dependency_wait();
  if constexpr (TABLE) {
    const int64_t total = (int64_t)a.lo.B * a.lo.max_pages;
    bool bad = false;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * blockDim.x) {
      const int p = a.table[e];
      int to = -1;
      if (p != -1) {
        if (p >= 0 && p < a.lo.n_pages) to = a.ws.map[p];
        bad |= to == -1;
      }
      a.table_out[e] = to;
    }
    if (bad) atomicOr(a.ws.status, KVQ_DEV_PAGE);
  }
  const int64_t runs = (int64_t)*a.ws.n_moves * a.lo.L * 2;
  for (int64_t r = blockIdx.x; r < runs; r += gridDim.x) {
    const int which = (int)(r & 1);
    const int64_t q = r >> 1;
    const int layer = (int)(q % a.lo.L);
    const int64_t m = q / a.lo.L;
    const int words = which ? v_words : k_words;
    V* base = reinterpret_cast<V*>(which ? a.cp.v_main : a.cp.k_main);
    [[maybe_unused]] const CachePtrs& cp = a.cp;
    if (!KVQ_CHECK((uint32_t)a.ws.src[m] < (uint32_t)(a.lo.n_pages - a.lo.bounds_shrink) &&
                   (uint32_t)a.ws.dst[m] < (uint32_t)(a.lo.n_pages - a.lo.bounds_shrink)))
      continue;
    const V* from = base + ((int64_t)layer * a.lo.n_pages + a.ws.src[m]) * words;
    V* to = base + ((int64_t)layer * a.lo.n_pages + a.ws.dst[m]) * words;
    int e = threadIdx.x;
    for (; e + 2 * blockDim.x < words; e += 3 * blockDim.x) {
      V v[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] = from[e + k * blockDim.x];
#pragma unroll
      for (int k = 0; k < 3; ++k) to[e + k * blockDim.x] = v[k];
    }
    for (; e < words; e += blockDim.x) to[e] = from[e];
  }
}

template <class V, bool TABLE>
cudaError_t launch_copy_as(const PagesArgs& a, int64_t k_bytes, int64_t v_bytes, int64_t max_moves, cudaStream_t s) {
  const int64_t runs = max_moves * a.lo.L * 2;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(runs, (int64_t)sm_count() * 8));
  return launch_dependent(copy_pages_kernel<V, TABLE>, dim3((unsigned)want), dim3(256), 0, s, a,
                          (int)(k_bytes / sizeof(V)), (int)(v_bytes / sizeof(V)));
}

template <bool TABLE>
cudaError_t launch_copy(const PagesArgs& a, int64_t max_moves, cudaStream_t s) {
  const int64_t per = (int64_t)a.lo.H * a.lo.pt;
  const int64_t kb = per * a.lo.kf.row, vb = per * a.lo.vf.row;
  const int64_t both = kb | vb;
  if (both % 16 == 0) return launch_copy_as<uint4, TABLE>(a, kb, vb, max_moves, s);
  if (both % 4 == 0) return launch_copy_as<uint32_t, TABLE>(a, kb, vb, max_moves, s);
  return launch_copy_as<uint16_t, TABLE>(a, kb, vb, max_moves, s);
}

// ---- host checks shared by the entries ------------------------------------------------

// What the bookkeeping holds: pages needed by one call, a copy for each sequence among them, are counted in 32 bits.
kvq_status pages_config(const kvq_config* cfg) {
  const kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (cfg->page_tokens < 1) return fail(KVQ_ERR_ARG, "the cache is not paged");
  if (cfg->batch > kMaxPageBatch) return fail(KVQ_ERR_UNSUPPORTED, "batch=%d > %d", cfg->batch, kMaxPageBatch);
  if ((int64_t)cfg->batch * ((int64_t)cfg->max_pages_per_seq + 1) > 0x7fffffff)
    return fail(KVQ_ERR_UNSUPPORTED, "a block table of %d x %d entries", cfg->batch, cfg->max_pages_per_seq);
  return KVQ_OK;
}

kvq_status pages_args(const kvq_config* cfg, const kvq_cache* cache, bool need_cache, const int32_t* table,
                      const int32_t* refs, void* workspace, size_t ws_bytes, PagesArgs* a) {
  kvq_status st = pages_config(cfg);
  if (st != KVQ_OK) return st;
  if (!table || !refs) return fail(KVQ_ERR_ARG, "block_table / refs is NULL");
  if (((uintptr_t)table | (uintptr_t)refs) & 3u) return fail(KVQ_ERR_ARG, "block_table / refs must be 4-byte aligned");
  if (!workspace) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = pages_ws_layout(cfg, nullptr, nullptr);
  if (ws_bytes < need) return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", ws_bytes, need);
  if (((uintptr_t)workspace) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (need_cache) {
    // the table argument is the one these calls change; the cache's own is not read
    kvq_cache c = {};
    if (cache) {
      c = *cache;
      if (!c.block_table) c.block_table = table;
    }
    if ((st = cache_ptrs(cfg, cache ? &c : nullptr, &a->cp)) != KVQ_OK) return st;
  }
  a->lo = make_layout(cfg);
  if ((int64_t)a->lo.H * a->lo.pt * std::max(a->lo.kf.row, a->lo.vf.row) > (int64_t)1 << 30)
    return fail(KVQ_ERR_UNSUPPORTED, "pages of more than 1 GiB");
  pages_ws_layout(cfg, workspace, &a->ws);
  a->cp.status = a->ws.status;
  a->table = const_cast<int32_t*>(table);
  a->refs = const_cast<int32_t*>(refs);
  return KVQ_OK;
}

kvq_status list_args(const kvq_config* cfg, const int32_t* seq_lens, const int32_t* l1, const int32_t* l2, int32_t n,
                     PagesArgs* a) {
  if (n < 0 || n > cfg->batch) return fail(KVQ_ERR_ARG, "n=%d not in [0, batch=%d]", n, cfg->batch);
  if (!seq_lens || (n > 0 && (!l1 || !l2))) return fail(KVQ_ERR_ARG, "seq_lens / a list is NULL");
  if (((uintptr_t)seq_lens | (uintptr_t)l1 | (uintptr_t)l2) & 3u)
    return fail(KVQ_ERR_ARG, "lists must be 4-byte aligned");
  a->seq_lens = const_cast<int32_t*>(seq_lens);
  a->seqs = l1;
  a->other = l2;
  a->n = n;
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_pages_workspace_bytes(const kvq_config* cfg, size_t* bytes) {
  const kvq_status st = pages_config(cfg);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  *bytes = pages_ws_layout(cfg, nullptr, nullptr);
  return ok();
}

kvq_status kvq_pages_init(const kvq_config* cfg, const int32_t* block_table, int32_t* refs, void* workspace,
                          size_t ws_bytes, void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, nullptr, false, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(workspace, 0, (size_t)((char*)a.ws.src - (char*)workspace), s);
  if (e == cudaSuccess) e = cudaMemsetAsync(refs, 0, sizeof(int32_t) * (size_t)cfg->n_pages, s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  const int64_t total = (int64_t)cfg->batch * cfg->max_pages_per_seq;
  count_refs_kernel<<<(unsigned)std::min<int64_t>((total + 255) / 256, (int64_t)sm_count() * 8), 256, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "page count kernel");
  return ok();
}

kvq_status kvq_pages_release(const kvq_config* cfg, int32_t* block_table, int32_t* refs, int32_t* seq_lens,
                             const int32_t* seqs, int32_t n, void* workspace, size_t ws_bytes, void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, nullptr, false, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  if ((st = list_args(cfg, seq_lens, seqs, seqs, n, &a)) != KVQ_OK) return st;
  if (n == 0) return ok();
  cudaError_t e = launch_dependent(release_kernel, dim3(n), dim3(256), 0, (cudaStream_t)stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "page release kernel");
  return ok();
}

kvq_status kvq_pages_fork(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table, int32_t* refs,
                          int32_t* seq_lens, const int32_t* src, const int32_t* dst, int32_t n, void* workspace,
                          size_t ws_bytes, void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, cache, true, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  if ((st = list_args(cfg, seq_lens, src, dst, n, &a)) != KVQ_OK) return st;
  if (a.lo.ring && a.lo.L > 65535) return fail(KVQ_ERR_UNSUPPORTED, "L=%d", a.lo.L);  // a row of the windows' grid each
  if (n == 0) return ok();
  cudaError_t e = launch_dependent(fork_kernel, dim3(n), dim3(256), 0, (cudaStream_t)stream, a);
  if (e == cudaSuccess && a.lo.ring) {
    // parts of a window of about 64 KiB, more while the grid is small
    const int64_t bytes = (int64_t)a.lo.H * a.lo.ring * a.lo.D * 2;
    const int64_t blocks = (int64_t)n * a.lo.L * 2;
    int64_t parts = std::max<int64_t>((bytes + 65535) / 65536, (int64_t)sm_count() * 4 / blocks);
    parts = std::max<int64_t>(1, std::min<int64_t>(parts, std::min<int64_t>((bytes + 4095) / 4096, 1024)));
    e = launch_dependent(fork_window_kernel, dim3(n, a.lo.L, (unsigned)(2 * parts)), dim3(256), 0,
                         (cudaStream_t)stream, a, (int)parts);
  }
  if (e != cudaSuccess) return cuda_fail(e, "page fork kernels");
  return ok();
}

kvq_status kvq_pages_reserve(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table, int32_t* refs,
                             const int32_t* seq_lens, const int32_t* seqs, const int32_t* n_new, int32_t n,
                             void* workspace, size_t ws_bytes, void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, cache, true, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  if ((st = list_args(cfg, seq_lens, seqs, n_new, n, &a)) != KVQ_OK) return st;
  if (n == 0) return ok();
  const size_t smem = sizeof(int32_t) * (size_t)n;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)  // always to the same value: another thread may call between this and the launch
    e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(sizeof(int32_t) * kMaxPageBatch));
  if (e == cudaSuccess) e = launch_dependent(reserve_kernel, dim3(1), dim3(kPlanThreads), smem, (cudaStream_t)stream, a);
  if (e == cudaSuccess) e = launch_copy<false>(a, n, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "page reserve kernels");
  return ok();
}

kvq_status kvq_pages_reorder(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table, int32_t* refs,
                             int32_t* seq_lens, const int32_t* parents, int32_t group, void* workspace, size_t ws_bytes,
                             void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, cache, true, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  if (group < 1 || cfg->batch % group) return fail(KVQ_ERR_ARG, "group=%d does not divide batch=%d", group, cfg->batch);
  if (group > kMaxReorder) return fail(KVQ_ERR_UNSUPPORTED, "group=%d > %d", group, kMaxReorder);
  if (!seq_lens || !parents) return fail(KVQ_ERR_ARG, "seq_lens / parents is NULL");
  if (((uintptr_t)seq_lens | (uintptr_t)parents) & 3u) return fail(KVQ_ERR_ARG, "lists must be 4-byte aligned");
  if (a.lo.ring && a.lo.L > 32767) return fail(KVQ_ERR_UNSUPPORTED, "L=%d", a.lo.L);  // two rows of the windows' grid each
  const int64_t columns = ((int64_t)cfg->max_pages_per_seq + kReorderThreads - 1) / kReorderThreads;
  if (columns > 65535) return fail(KVQ_ERR_UNSUPPORTED, "max_pages_per_seq=%d", cfg->max_pages_per_seq);
  a.seq_lens = seq_lens;
  a.other = parents;
  a.n = group;
  const int groups = cfg->batch / group;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_dependent(reorder_kernel, dim3(groups, (unsigned)columns), dim3(kReorderThreads), 0, s, a);
  if (e == cudaSuccess && a.lo.ring && group > 1) {
    // words in turn once the grid fills the card several times
    const int64_t unit = (int64_t)a.lo.H * a.lo.ring * a.lo.D / 8, blocks = (int64_t)groups * a.lo.L * 2;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((unit + kReorderThreads - 1) / kReorderThreads,
                                                                 std::max<int64_t>(1, (int64_t)sm_count() * 64 / blocks)));
    const dim3 grid((unsigned)parts, (unsigned)(2 * a.lo.L), (unsigned)groups);
    e = group <= 8    ? launch_dependent(reorder_window_kernel<8>, grid, dim3(kReorderThreads), 0, s, a)
        : group <= 16 ? launch_dependent(reorder_window_kernel<16>, grid, dim3(kReorderThreads), 0, s, a)
                      : launch_dependent(reorder_window_kernel<32>, grid, dim3(kReorderThreads), 0, s, a);
  }
  if (e != cudaSuccess) return cuda_fail(e, "page reorder kernels");
  return ok();
}

kvq_status kvq_pages_compact(const kvq_config* cfg, const kvq_cache* cache, const int32_t* block_table,
                             const int32_t* refs, int32_t* table_out, int32_t* refs_out, void* workspace,
                             size_t ws_bytes, void* stream) {
  PagesArgs a{};
  kvq_status st = pages_args(cfg, cache, true, block_table, refs, workspace, ws_bytes, &a);
  if (st != KVQ_OK) return st;
  if (!table_out || !refs_out) return fail(KVQ_ERR_ARG, "table_out / refs_out is NULL");
  if (((uintptr_t)table_out | (uintptr_t)refs_out) & 3u) return fail(KVQ_ERR_ARG, "outputs must be 4-byte aligned");
  a.table_out = table_out;
  a.refs_out = refs_out;
  cudaError_t e = launch_dependent(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, a);
  if (e == cudaSuccess) e = launch_copy<true>(a, std::max(1, cfg->n_pages / 2), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "page compaction kernels");
  return ok();
}

}  // extern "C"
