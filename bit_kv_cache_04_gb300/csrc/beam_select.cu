// kvq_beam_select: the best continuations of every group's beams over the
// whole vocabulary.
//
// With x the logits of beam b, s its score and l = log sum_v e^x_v, candidate (b, v) scores s + x_v - l.  Per
// beam only the K largest logits can be among the group's K best, so a row is read once for three things:
// its maximum, its sum of exponentials (fp32 a thread, joined in 64 bits) and its K largest values with their places.
//
// Bound by HBM where the batch is large (2 or 4 bytes a logit, read once), by launch and dependent steps where it is small.
// A row is cut into `splits` blocks so that small batches fill the card too; the group's last block
// (a ticket; no block waits) joins the pieces and picks the K best in 64 bits.
//
// The K largest: a warp keeps its list sorted over its lanes and looks closer at a batch of values only where one passes
// the list's last or the block's bound (the best of its warps' last ones).  Of n values in random order
// about K ln(n / K) ever enter a list, so the stream's cost is that of the maximum and the exponentials.
#include <algorithm>
#include <climits>
#include <cfloat>

#include "block_codec.cuh"
#include "kvq_host.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kMaxBeams = 32;       // a list is one warp wide
constexpr int kMaxVocab = (1 << 26) - 1;  // beam * vocab + token stays below INT_MAX

struct SelectWs {
  uint32_t* tickets;  // [groups], zero between calls
  float2* sums;       // [rows][splits]: maximum, sum of e^(x - maximum)
  int2* best;         // [rows][splits][beams]: fp32 bits of a logit and its token, descending
};

struct SelectArgs {
  const char* logits;
  int64_t group_stride, beam_stride;  // in elements
  const float* scores;
  const int32_t* done;
  float* scores_out;
  int32_t *tokens, *parents, *done_out;
  SelectWs ws;
  int beams, vocab, eos, splits;
};

// a before b in a list: larger value, then lower place
template <class V>
__device__ __forceinline__ bool before(V av, int ai, V bv, int bi) {
  return av > bv || (av == bv && ai < bi);
}

// A warp's sorted list, entry i in lane i, and its K-th entry.
template <class V>
struct BestList {
  V v, last_v;
  int i, last_i;
  __device__ __forceinline__ void clear(V lowest) {
    v = last_v = lowest;
    i = last_i = INT_MAX;
  }
  __device__ __forceinline__ bool takes(V x, int at) const { return before(x, at, last_v, last_i); }
  // x, at: equal in all lanes
  __device__ __forceinline__ void insert(V x, int at, int beams) {
    const int lane = threadIdx.x & 31;
    const int pos = __popc(__ballot_sync(0xffffffffu, before(v, i, x, at)));
    const V up = __shfl_up_sync(0xffffffffu, v, 1);
    const int upi = __shfl_up_sync(0xffffffffu, i, 1);
    if (lane >= pos) {
      v = lane == pos ? x : up;
      i = lane == pos ? at : upi;
    }
    last_v = __shfl_sync(0xffffffffu, v, beams - 1);
    last_i = __shfl_sync(0xffffffffu, i, beams - 1);
  }
  // the lanes' x where `in`, each if it belongs into the list
  __device__ __forceinline__ void offer(V x, int at, bool in, int beams) {
    uint32_t hits = __ballot_sync(0xffffffffu, in && takes(x, at));
    while (hits) {
      const int src = __ffs(hits) - 1;
      hits &= hits - 1;
      const V xv = __shfl_sync(0xffffffffu, x, src);
      const int xi = __shfl_sync(0xffffffffu, at, src);
      if (takes(xv, xi)) insert(xv, xi, beams);
    }
  }
};

// fp32 as an int of the same order
__device__ __forceinline__ int ordered(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

template <int DT>
struct LogitType {
  static constexpr int BYTES = DT == KVQ_DT_F32 ? 4 : 2, PER = 16 / BYTES;
  static constexpr uint32_t LOWEST = DT == KVQ_DT_F32 ? 0xff800000u : DT == KVQ_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;  // -inf
  __device__ __forceinline__ static void widen(uint4 w, float (&x)[PER]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == KVQ_DT_F32) {
        x[k] = __uint_as_float(u[k]);
      } else if constexpr (DT == KVQ_DT_BF16) {
        x[2 * k] = __uint_as_float(u[k] << 16);
        x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
};

// NaN counts as -inf, +inf as the largest finite number
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

// 16-byte word w, counted from the boundary at or before the row, `skew` elements before its start.  Elements outside
// the row are -inf.
template <int DT>
__device__ __forceinline__ uint4 row_word(const char* row, int skew, int vocab, int w) {
  using T = LogitType<DT>;
  const int first = w * T::PER - skew;  // token of the word's first element
  const char* at = row + (int64_t)first * T::BYTES;
  if (first >= 0 && first + T::PER <= vocab) return __ldcs(reinterpret_cast<const uint4*>(at));
  uint32_t u[4] = {T::LOWEST, T::LOWEST, T::LOWEST, T::LOWEST};
#pragma unroll
  for (int e = 0; e < T::PER; ++e) {
    if (first + e < 0 || first + e >= vocab) continue;
    if constexpr (T::BYTES == 4) {
      u[e] = reinterpret_cast<const uint32_t*>(at)[e];
    } else {
      const uint32_t v = reinterpret_cast<const uint16_t*>(at)[e];
      u[e / 2] = e & 1 ? (u[e / 2] & 0xffffu) | v << 16 : (u[e / 2] & 0xffff0000u) | v;
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// 16 bytes from byte `shift` of (a, b) on; shift is the same in all lanes.
__device__ __forceinline__ uint4 straddle(uint4 a, uint4 b, int shift) {
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
  }
  const int bits = (shift & 3) * 8;
  return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits), __funnelshift_r(x[2], x[3], bits),
                    __funnelshift_r(x[3], x[4], bits));
}

struct SelectShared {
  int bound;  // ordered(): no value below it is among the block's K largest
  float m[kSelWarps], s[kSelWarps];
  float v[kSelWarps][kMaxBeams];
  double dv[kSelWarps][kMaxBeams];
  int i[kSelWarps][kMaxBeams];
  double max[kMaxBeams], log_sum[kMaxBeams], score[kMaxBeams];
  int done[kMaxBeams];
  bool last;
};

// Words [w0, w1) of a row, counted from its start: the block's maximum, sum and K largest into the workspace.  A warp takes
// `up` times 32 words side by side, so that a row that starts off a 16-byte boundary has its words put together from the
// aligned ones of this lane and the next: which thread sums what, and with it every bit of the
// result, does not depend on where the row lies.
template <int DT>
__device__ __forceinline__ void scan_row(const SelectArgs& a, SelectShared& sh, const char* row, int skew, int w0, int w1,
                                         int64_t piece) {
  using T = LogitType<DT>;
  constexpr int U = 4;  // words in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // finite, so that rows of -inf alone sum up to nothing instead of NaN
  float m = -FLT_MAX, s = 0.f;
  BestList<float> list;
  list.clear(-INFINITY);
  const int up = min(U, (w1 - w0 + kSelThreads - 1) / kSelThreads), stride = up * kSelThreads;
  uint4 next[U], tail;
  auto load = [&](int w) {
    tail = make_uint4(T::LOWEST, T::LOWEST, T::LOWEST, T::LOWEST);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      next[u] = tail;
      if (u < up && w + u * 32 < w1 + (skew ? 1 : 0)) next[u] = row_word<DT>(row, skew, a.vocab, w + u * 32);
    }
    if (skew && lane == 0 && w + up * 32 <= w1) tail = row_word<DT>(row, skew, a.vocab, w + up * 32);
  };
  int w = w0 + warp * up * 32 + lane;
  load(w);
#pragma unroll 1
  for (; w - lane < w1; w += stride) {  // whole warps
    uint4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = next[u];
    if (skew) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool end = u + 1 == U || u + 1 == up;
        uint4 n = next[u];
        if (lane == 0) n = end ? tail : next[u + 1 < U ? u + 1 : u];
        const int from = (lane + 1) & 31;
        n.x = __shfl_sync(0xffffffffu, n.x, from);
        n.y = __shfl_sync(0xffffffffu, n.y, from);
        n.z = __shfl_sync(0xffffffffu, n.z, from);
        n.w = __shfl_sync(0xffffffffu, n.w, from);
        now[u] = straddle(now[u], n, skew * T::BYTES);
      }
    }
    load(w + stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= up) break;
      if (w + u * 32 >= w1) now[u] = make_uint4(T::LOWEST, T::LOWEST, T::LOWEST, T::LOWEST);  // the next block's
      float x[T::PER];
      T::widen(now[u], x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < T::PER; ++e) top = fmaxf(top, x[e]);  // of a NaN and a number the number
      if (top == INFINITY) {
#pragma unroll
        for (int e = 0; e < T::PER; ++e) x[e] = tame(x[e]);
        top = FLT_MAX;
      }
      if (top > m) {
        s *= exp2_approx((m - top) * kLog2e);
        m = top;
      }
      auto sum = [&] {  // x - m is exact where it matters, near the maximum
        const uint64_t mm = pk2(m, m), c = pk2(kLog2e, kLog2e);
        uint64_t t = 0;
#pragma unroll
        for (int e = 0; e < T::PER; e += 2) {
          float e0, e1;
          upk2(mul2(sub2(pk2(x[e], x[e + 1]), mm), c), e0, e1);
          t = add2(t, pk2(exp2_approx(e0), exp2_approx(e1)));
        }
        float t0, t1;
        upk2(t, t0, t1);
        return t0 + t1;
      };
      float t = sum();
      if (t != t) {
#pragma unroll
        for (int e = 0; e < T::PER; ++e) x[e] = tame(x[e]);
        top = fmaxf(top, -INFINITY);
        t = sum();
      }
      s += t;
      const float bound = unordered(*(volatile int*)&sh.bound);
      if (__any_sync(0xffffffffu, top >= list.last_v && top >= bound)) {
        const int first = (w + u * 32) * T::PER, end = min(a.vocab, w1 * T::PER);
#pragma unroll
        for (int e = 0; e < T::PER; ++e) list.offer(x[e], first + e, x[e] >= bound && first + e < end, a.beams);
        if (lane == 0) atomicMax(&sh.bound, ordered(list.last_v));
      }
    }
  }
  // the block's
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  s *= exp2_approx((m - wm) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    sh.m[warp] = wm;
    sh.s[warp] = s;
  }
  sh.v[warp][lane] = list.v;
  sh.i[warp][lane] = list.i;
  __syncthreads();
  if (warp) return;
#pragma unroll 1
  for (int k = 1; k < kSelWarps; ++k) {
    const float v = sh.v[k][lane];
    const int i = sh.i[k][lane];
    list.offer(v, i, lane < a.beams && i != INT_MAX, a.beams);
  }
  const float pm = lane < kSelWarps ? sh.m[lane] : -FLT_MAX, ps = lane < kSelWarps ? sh.s[lane] : 0.f;
  float bm = pm;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
  float bs = ps * exp2_approx((pm - bm) * kLog2e);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) bs += __shfl_xor_sync(0xffffffffu, bs, o);
  if (lane == 0) a.ws.sums[piece] = make_float2(bm, bs);
  if (lane < a.beams) a.ws.best[piece * a.beams + lane] = make_int2(__float_as_int(list.v), list.i);
  __threadfence();  // before the ticket
  __syncwarp();
}

// The group's last block: log-sums of its rows, then the K best of all their lists, in 64 bits.
__device__ __forceinline__ void join_group(const SelectArgs& a, SelectShared& sh, int group) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.beams, S = a.splits;
  const int64_t row0 = (int64_t)group * K;
#pragma unroll 1
  for (int b = warp; b < K; b += kSelWarps) {
    const int done = a.done && a.done[row0 + b];
    double sum = 0;
    float m = -FLT_MAX;
    if (!done) {
      const float2* p = a.ws.sums + (row0 + b) * S;
#pragma unroll 1
      for (int k = lane; k < S; k += 32) m = fmaxf(m, __ldcg(&p[k].x));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 1
      for (int k = lane; k < S; k += 32) {
        const float2 q = __ldcg(p + k);
        sum += (double)q.y * (double)exp2_approx((q.x - m) * kLog2e);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
      sh.done[b] = done;
      // apart, so that rows of the type's lowest value keep their log-sum
      sh.max[b] = (double)m;
      sh.log_sum[b] = sum > 0 ? log(sum) : 0.0;  // nothing may follow: every candidate is -inf all the same
      sh.score[b] = (double)tame(a.scores[row0 + b]);
    }
  }
  __syncthreads();
  BestList<double> list;
  list.clear(-(double)INFINITY);
#pragma unroll 1
  for (int q = warp; q < K * S; q += kSelWarps) {
    const int b = q / S;
    if (sh.done[b]) {
      if (q == b * S) list.offer(sh.score[b], b * a.vocab + a.eos, lane == 0, K);
      continue;
    }
    int2 e = make_int2(0, INT_MAX);
    if (lane < K) e = __ldcg(a.ws.best + ((row0 + b) * S + (q - b * S)) * K + lane);
    const double c = sh.score[b] + (((double)__int_as_float(e.x) - sh.max[b]) - sh.log_sum[b]);
    list.offer(c, b * a.vocab + e.y, e.y != INT_MAX, K);
  }
  sh.dv[warp][lane] = list.v;
  sh.i[warp][lane] = list.i;
  __syncthreads();
  if (warp) return;
#pragma unroll 1
  for (int k = 1; k < kSelWarps; ++k) list.offer(sh.dv[k][lane], sh.i[k][lane], lane < K && sh.i[k][lane] != INT_MAX, K);
  if (lane < K) {
    const int b = list.i / a.vocab, t = list.i - b * a.vocab;
    a.scores_out[row0 + lane] = (float)list.v;
    a.tokens[row0 + lane] = t;
    a.parents[row0 + lane] = b;
    if (a.done_out) a.done_out[row0 + lane] = sh.done[b] || t == a.eos;
  }
}

template <int DT>
__global__ void __launch_bounds__(kSelThreads, 3) beam_select_kernel(const __grid_constant__ SelectArgs a) {
  using T = LogitType<DT>;
  __shared__ SelectShared sh;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int split = (int)(blockIdx.x - row * a.splits), group = (int)(row / a.beams), b = (int)(row - (int64_t)group * a.beams);
  if (threadIdx.x == 0) sh.bound = ordered(-INFINITY);
  grid_launch_dependents();
  grid_dependency_wait();
  __syncthreads();
  if (!(a.done && a.done[row])) {
    const char* p = a.logits + (group * a.group_stride + b * a.beam_stride) * T::BYTES;
    const int skew = (int)((uintptr_t)p & 15) / T::BYTES;  // elements between the 16-byte boundary and the row
    const int words = (a.vocab + T::PER - 1) / T::PER;
    const int per = (words + a.splits - 1) / a.splits;
    scan_row<DT>(a, sh, p, skew, min(split * per, words), min((split + 1) * per, words), row * a.splits + split);
  }
  if (threadIdx.x == 0) {
    sh.last = atomicAdd(a.ws.tickets + group, 1u) == (uint32_t)(a.beams * a.splits - 1);
  }
  __syncthreads();
  if (!sh.last) return;
  __threadfence();
  if (threadIdx.x == 0) a.ws.tickets[group] = 0;
  join_group(a, sh, group);
}

// Blocks a row: about one wave of four blocks an SM, each with at least 2048 logits to read.
int splits_of(int64_t rows, int vocab) {
  const int64_t want = (int64_t)sm_count() * 4 / std::max<int64_t>(1, rows);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, (int64_t)vocab / 2048, 1024}));
}

size_t select_ws(int groups, int beams, int vocab, void* base, SelectWs* w) {
  const int64_t rows = (int64_t)groups * beams, pieces = rows * splits_of(rows, vocab);
  const size_t sums = align_up(sizeof(uint32_t) * (size_t)groups), best = sums + align_up(sizeof(float2) * (size_t)pieces);
  if (w) {
    w->tickets = (uint32_t*)base;
    w->sums = (float2*)((char*)base + sums);
    w->best = (int2*)((char*)base + best);
  }
  return best + align_up(sizeof(int2) * (size_t)pieces * beams);
}

kvq_status check_select(int32_t groups, int32_t beams, int32_t vocab) {
  if (groups < 1 || beams < 1 || vocab < 1) return fail(KVQ_ERR_ARG, "groups, beams and vocab must be >= 1");
  if (beams > kMaxBeams) return fail(KVQ_ERR_UNSUPPORTED, "beams=%d > %d", beams, kMaxBeams);
  if (vocab > kMaxVocab) return fail(KVQ_ERR_UNSUPPORTED, "vocab=%d > %d", vocab, kMaxVocab);
  if ((int64_t)groups * beams > 1 << 24) return fail(KVQ_ERR_UNSUPPORTED, "%d x %d beams", groups, beams);
  return KVQ_OK;
}

kvq_status check_select_ws(int32_t groups, int32_t beams, int32_t vocab, void* ws, size_t bytes) {
  if (!ws) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = select_ws(groups, beams, vocab, nullptr, nullptr);
  if (bytes < need) return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", bytes, need);
  if (((uintptr_t)ws) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_beam_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, size_t* bytes) {
  const kvq_status st = check_select(n_groups, beams, vocab);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  *bytes = select_ws(n_groups, beams, vocab, nullptr, nullptr);
  return ok();
}

kvq_status kvq_beam_workspace_init(int32_t n_groups, int32_t beams, int32_t vocab, void* workspace, size_t ws_bytes,
                                   void* stream) {
  kvq_status st = check_select(n_groups, beams, vocab);
  if (st != KVQ_OK) return st;
  if ((st = check_select_ws(n_groups, beams, vocab, workspace, ws_bytes)) != KVQ_OK) return st;
  const cudaError_t e = cudaMemsetAsync(workspace, 0, align_up(sizeof(uint32_t) * (size_t)n_groups), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return ok();
}

kvq_status kvq_beam_select(const void* logits, int32_t dtype, int64_t group_stride, int64_t beam_stride, int32_t n_groups,
                           int32_t beams, int32_t vocab, const float* scores, const int32_t* done, int32_t eos,
                           float* scores_out, int32_t* tokens, int32_t* parents, int32_t* done_out, void* workspace,
                           size_t ws_bytes, void* stream) {
  kvq_status st = check_select(n_groups, beams, vocab);
  if (st != KVQ_OK) return st;
  if (dtype != KVQ_DT_F16 && dtype != KVQ_DT_BF16 && dtype != KVQ_DT_F32) return fail(KVQ_ERR_ARG, "dtype=%d", dtype);
  if (!logits || !scores || !scores_out || !tokens || !parents) return fail(KVQ_ERR_ARG, "logits, scores or an output is NULL");
  if (group_stride < 0 || beam_stride < 0) return fail(KVQ_ERR_ARG, "negative stride");
  if (eos < -1 || eos >= vocab) return fail(KVQ_ERR_ARG, "eos=%d outside [-1, %d)", eos, vocab);
  if (done && eos < 0) return fail(KVQ_ERR_ARG, "finished beams need an end token");
  if ((uintptr_t)logits % (dtype == KVQ_DT_F32 ? 4 : 2)) return fail(KVQ_ERR_ARG, "logits must be aligned to their elements");
  if (((uintptr_t)scores | (uintptr_t)done | (uintptr_t)scores_out | (uintptr_t)tokens | (uintptr_t)parents |
       (uintptr_t)done_out) & 3u)
    return fail(KVQ_ERR_ARG, "scores, done and outputs must be 4-byte aligned");
  if ((st = check_select_ws(n_groups, beams, vocab, workspace, ws_bytes)) != KVQ_OK) return st;
  SelectArgs a{};
  a.logits = (const char*)logits;
  a.group_stride = group_stride;
  a.beam_stride = beam_stride;
  a.scores = scores;
  a.done = done;
  a.scores_out = scores_out;
  a.tokens = tokens;
  a.parents = parents;
  a.done_out = done_out;
  a.beams = beams;
  a.vocab = vocab;
  a.eos = eos;
  const int64_t rows = (int64_t)n_groups * beams;
  a.splits = splits_of(rows, vocab);
  select_ws(n_groups, beams, vocab, workspace, &a.ws);
  const dim3 grid((unsigned)(rows * a.splits));
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == KVQ_DT_F32    ? launch_dependent(beam_select_kernel<KVQ_DT_F32>, grid, dim3(kSelThreads), 0, s, a)
                        : dtype == KVQ_DT_BF16 ? launch_dependent(beam_select_kernel<KVQ_DT_BF16>, grid, dim3(kSelThreads), 0, s, a)
                                               : launch_dependent(beam_select_kernel<KVQ_DT_F16>, grid, dim3(kSelThreads), 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "beam selection kernel");
  return ok();
}

}  // extern "C"
