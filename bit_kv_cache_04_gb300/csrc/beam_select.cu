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
// The K largest: a warp keeps its list sorted over its lanes.  A value and its place are one 64-bit key (larger value, then lower place),
// so a comparison decides both.  Of a turn's values (32 a lane) only those at or above a bound are looked at: the block's
// best known K-th value, in its first turn the K-th of its threads' largest, found bit by bit with votes.  Those join the list by
// rank: every lane counts how many of the few new keys are before its own.  Of n values in random order about K ln(n / K)
// ever enter a list, so the stream's cost is that of the maximum and the exponentials.
//
// On one GB300, one call a replayed graph: 1 x 4 beams over 32000 tokens 12.4 us (launch, one turn and two joins), 16 x 5 over 50257 (fp32) 18.5,
// 8 x 32 over 32001 32, 64 x 8 over 131072 (bf16) 50 us.  Called one behind another, each one's blocks beginning while the one before still
// runs: 12.9, 21.9, 41 and 47 us or 2.9 TB/s, with 68 % of the issue slots taken: 459 instructions for a warp's turn.
// Turns of masked values alone go through their terms twice (see kBig): 64 x 8 rows of nothing but -1e9 69 us.
// (Tried: sorting networks over the warp instead of ranks, 2200 cycles a time, and 64-bit floating-point comparisons in the last step, 5000: the smallest
// search 39 us, 20.8 us without them.  Every value offered by itself, unrolled, the large batch 144 us.  A first bound for each warp instead of
// one for the block: 8 x 32 beams 41 us.)
#include <algorithm>
#include <climits>
#include <cfloat>
#include <type_traits>

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
  int64_t* best;      // [rows][splits][beams]: keys of logits and tokens, descending
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

// fp32 as an int of the same order
__device__ __forceinline__ int ordered(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

// A logit and its token.
struct LogitKey {
  int64_t k;
  __device__ __forceinline__ static LogitKey none() { return LogitKey{INT64_MIN}; }
  __device__ __forceinline__ static LogitKey of(float v, int token) {
    return LogitKey{(int64_t)(((uint64_t)(uint32_t)ordered(v + 0.f) << 32) | (uint32_t)~token)};  // (-0 counts as 0)
  }
  __device__ __forceinline__ float value() const { return unordered((int)(k >> 32)); }
  __device__ __forceinline__ int token() const { return (int)~(uint32_t)k; }
  __device__ __forceinline__ bool before(const LogitKey& o) const { return k > o.k; }
  __device__ __forceinline__ bool real() const { return k != INT64_MIN; }
  __device__ __forceinline__ LogitKey of_lane(int l) const { return LogitKey{__shfl_sync(0xffffffffu, k, l)}; }
};
// A score, as an integer of the same order, and a place (beam * vocab + token).
struct alignas(16) ScoreKey {
  int64_t s;
  int at, pad;
  __device__ __forceinline__ static ScoreKey none() { return ScoreKey{INT64_MIN, INT_MAX, 0}; }
  __device__ __forceinline__ static ScoreKey of(double v, int at) {
    const int64_t b = __double_as_longlong(v + 0.0);
    return ScoreKey{b ^ ((b >> 63) & INT64_MAX), at, 0};
  }
  __device__ __forceinline__ double value() const { return __longlong_as_double(s ^ ((s >> 63) & INT64_MAX)); }
  __device__ __forceinline__ bool before(const ScoreKey& o) const { return (s > o.s) | ((s == o.s) & (at < o.at)); }
  __device__ __forceinline__ bool real() const { return at != INT_MAX; }
  __device__ __forceinline__ ScoreKey of_lane(int l) const {
    return ScoreKey{__shfl_sync(0xffffffffu, s, l), __shfl_sync(0xffffffffu, at, l), 0};
  }
};

// A number that at least K of the lanes' N (each) are not below: the K-th largest's bits from LOW on, two at a time.
template <int LOW, int N>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&x)[N], int K) {
  uint32_t t = 0;
  auto enough = [&](uint32_t c) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popc(__ballot_sync(0xffffffffu, x[i] >= c));
    return n >= K;
  };
#pragma unroll 1
  for (int at = 30; at >= LOW; at -= 2) {
    const uint32_t c1 = t | 1u << at, c2 = t | 2u << at, c3 = t | 3u << at;
    const bool e1 = enough(c1), e2 = enough(c2), e3 = enough(c3);
    t = e3 ? c3 : e2 ? c2 : e1 ? c1 : t;
  }
  return t;
}

// n <= 32 keys in shared memory join a warp's sorted list (entry i in lane i), by rank; `room`: 32 keys of scratch.
template <class Key>
__device__ __forceinline__ void join_found(Key& list, const Key* found, int n, Key* room) {
  const int lane = threadIdx.x & 31;
  const Key mine = lane < n ? found[lane] : Key::none();
  int at_list = lane, at_mine = 0;
#pragma unroll 2
  for (int j = 0; j < n; ++j) {
    const Key c = found[j];
    const bool b = c.before(list);
    at_list += b;
    at_mine += c.before(mine);
    const int ahead = __popc(__ballot_sync(0xffffffffu, !b));  // entries of the list before it
    if (lane == j) at_mine += ahead;
  }
  __syncwarp();
  if (at_list < 32) room[at_list] = list;
  if (lane < n && at_mine < 32) room[at_mine] = mine;
  __syncwarp();
  list = room[lane];
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// Sums of exponentials are of 2^(x kLog2e - r), one fused product a term, r = kLog2e times the largest value m, rounded: the same
// number in every term, taken off again at the end.  It is off by up to half a step of r, and so is every exponent.  Up to kBig that is
// 1/16 at most; beyond (from some 1e9 on all of a row's terms would overflow or vanish together: rows and tokens masked by
// -1e10, by the type's lowest value, infinities) terms are of 2^((x - m) kLog2e), two roundings each, where the
// difference is exact for all that count.
constexpr float kBig = 1e6f;
__device__ __forceinline__ bool big(float m) { return fabsf(m) > kBig; }
__device__ __forceinline__ float reference(float m) { return __fmul_rn(m, kLog2e); }
// What takes a sum from the reference of m to that of a larger value: r below kBig, m kLog2e itself beyond, in one fused
// product where they meet.  (Both rounded as in the terms: contracted to one
// fused product, m = to gave 2^(rounding of r) instead of 1, and rows 10000 away from zero scores up to 9e-4 off.)
__device__ __forceinline__ float rescale(float m, float to) {
  const float x = big(m) ? (big(to) ? (m - to) * kLog2e : __fmaf_rn(m, kLog2e, -reference(to)))
                         : (big(to) ? __fmaf_rn(-to, kLog2e, reference(m)) : __fsub_rn(reference(m), reference(to)));
  return exp2_approx(x);
}

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

// Natural logarithm, good to 2^-24: the exponent's share in 64 bits, the mantissa's in 32.
__device__ __forceinline__ double log_of(double x) {
  const int hi = __double2hiint(x), e = (hi >> 20 & 0x7ff) - 1023;
  const double f = __hiloint2double((hi & 0xfffff) | 0x3ff00000, __double2loint(x));
  const float g = (float)f;
  return e * 0.69314718055994531 + ((double)logf(g) + (double)((float)(f - (double)g) / g));
}

template <int DT>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {  // of a NaN and a number the number
  if constexpr (DT == KVQ_DT_BF16) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The largest of N words (-inf for NaN alone)
template <int DT, int N>
__device__ __forceinline__ float words_max(const uint4 (&w)[N]) {
  float top = -INFINITY;
  if constexpr (DT == KVQ_DT_F32) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                             fmaxf(__uint_as_float(w[u].z), __uint_as_float(w[u].w))));
  } else {
    uint32_t p = LogitType<DT>::LOWEST;
#pragma unroll
    for (int u = 0; u < N; ++u)
      p = pair_max<DT>(p, pair_max<DT>(pair_max<DT>(w[u].x, w[u].y), pair_max<DT>(w[u].z, w[u].w)));
    float x[LogitType<DT>::PER];
    LogitType<DT>::widen(make_uint4(p, p, p, p), x);
    top = fmaxf(top, fmaxf(x[0], x[1]));
  }
  return top;
}

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

// The same into shared memory, whole words of the row asynchronously (one group a turn, see scan_row).
template <int DT>
__device__ __forceinline__ void fetch_word(uint4* to, const char* row, int skew, int vocab, int w) {
  using T = LogitType<DT>;
  const int first = w * T::PER - skew;
  if (first >= 0 && first + T::PER <= vocab)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(row + (int64_t)first * T::BYTES)
                 : "memory");
  else
    *to = row_word<DT>(row, skew, vocab, w);
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

constexpr int kWords = 4;  // 16-byte words of a thread in flight, and looked at together

struct SelectShared {
  uint4 words[kSelWarps][2][kWords * 32 + 1];  // a warp's turn, and the next one on its way
  union {
    ScoreKey found[kSelWarps][64];             // (or 128 LogitKeys) on their way into a warp's list: 31, and two lanes' 32
    ScoreKey all[kSelWarps * kMaxBeams];
  };
  ScoreKey room[kSelWarps][32];
  uint32_t top[kSelThreads];           // the threads' largest of the first turn, as unsigned numbers of the same order
  int count;                           // candidates in `all`
  int bound;                           // ordered(): no value below it is among the block's K largest
  float m[kSelWarps], s[kSelWarps];
  double max[kMaxBeams], log_sum[kMaxBeams], score[kMaxBeams];
  int done[kMaxBeams];
  bool finished;                       // this block's beam
  bool last;
};

// The warps' lists joined, by rank, into the first K lanes of warp 0.
template <class Key>
__device__ __forceinline__ Key join_warps(SelectShared& sh, const Key& list, int K) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Key *const all = reinterpret_cast<Key*>(sh.all), *const out = reinterpret_cast<Key*>(sh.room[0]);
  __syncthreads();  // what the shared memory held before has been read
  if (lane < K) all[warp * K + lane] = list;
  if (threadIdx.x < 32) out[threadIdx.x] = Key::none();
  __syncthreads();
  const int n = kSelWarps * K;
  if ((int)threadIdx.x - lane < n) {
    const Key mine = (int)threadIdx.x < n ? all[threadIdx.x] : Key::none();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += all[j].before(mine);
    if (mine.real() && rank < K) out[rank] = mine;
  }
  __syncthreads();
  return out[lane];
}

// Words [w0, w1) of a row, counted from its start: the block's maximum, sum and K largest into the workspace.  A warp takes
// `up` times 32 words side by side, so that a row that starts off a 16-byte boundary has its words put together from the
// aligned ones of this lane and the next: which thread sums what, and with it every bit of the
// result, does not depend on where the row lies.
template <int DT>
__device__ __forceinline__ void scan_row(const SelectArgs& a, SelectShared& sh, const char* row, int skew, int w0, int w1,
                                         int64_t piece) {
  using T = LogitType<DT>;
  constexpr int U = kWords;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // finite, so that rows of -inf alone sum up to nothing instead of NaN
  float m = -FLT_MAX, s = 0.f;
  LogitKey list = LogitKey::none(), last = list;  // last: the K-th
  LogitKey *const found = reinterpret_cast<LogitKey*>(sh.found[warp]), *const room = reinterpret_cast<LogitKey*>(sh.room[warp]);
  const int up = min(U, (w1 - w0 + kSelThreads - 1) / kSelThreads), stride = up * kSelThreads;
  const uint4 none = make_uint4(T::LOWEST, T::LOWEST, T::LOWEST, T::LOWEST);
  const char* const at0 = row + ((int64_t)(w0 + warp * up * 32 + lane) * T::PER - skew) * T::BYTES;  // of this lane's first word
  const uint32_t to0 = (uint32_t)__cvta_generic_to_shared(&sh.words[warp][0][lane]);
  auto fetch = [&](int w, int slot) {  // (aligned words: one more where the row lies off the boundary)
    uint4* to = sh.words[warp][slot];
    const int wb = w - lane;  // the warp's
    if (up == U && wb * T::PER >= skew && (wb + U * 32 + 1) * T::PER <= a.vocab + skew && wb + U * 32 <= w1) {  // nothing but whole words
      const char* at = at0 + (int64_t)(w - (w0 + warp * up * 32 + lane)) * 16;
#pragma unroll
      for (int u = 0; u < U; ++u)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to0 + slot * (uint32_t)sizeof(sh.words[0][0]) + u * 512), "l"(at + u * 512)
                     : "memory");
      if (skew && lane == 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to0 + slot * (uint32_t)sizeof(sh.words[0][0]) + U * 512), "l"(at + U * 512)
                     : "memory");
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < up && w + u * 32 < w1 + (skew ? 1 : 0)) fetch_word<DT>(to + u * 32 + lane, row, skew, a.vocab, w + u * 32);
    if (skew && lane == 0 && w + up * 32 <= w1) fetch_word<DT>(to + up * 32, row, skew, a.vocab, w + up * 32);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  int w = w0 + warp * up * 32 + lane, slot = 0;
  bool first = true;
  fetch(w, 0);
#pragma unroll 1
  for (; first || w - lane < w1; w += stride, slot ^= 1) {  // whole warps; a first turn also where there is nothing to read
    fetch(w + stride, slot ^ 1);
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncwarp();
    const uint4* const in_slot = sh.words[warp][slot];
    uint4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      now[u] = none;  // (the next block's, or another warp's)
      if (u < up && w + u * 32 < w1) {
        now[u] = in_slot[u * 32 + lane];
        if (skew) now[u] = straddle(now[u], in_slot[u * 32 + lane + 1], skew * T::BYTES);
      }
    }
    float top = words_max<DT>(now);
    if (top == INFINITY) top = FLT_MAX;
    if (top > m) {
      s *= rescale(m, top);
      m = top;
    }
    const float r = reference(m);
    float t;
    {
      const uint64_t nr = pk2(-r, -r), c = pk2(kLog2e, kLog2e);
      uint64_t sum = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[T::PER];
        T::widen(now[u], x);
#pragma unroll
        for (int e = 0; e < T::PER; e += 2) {
          float e0, e1;
          upk2(fma2(pk2(x[e], x[e + 1]), c, nr), e0, e1);
          sum = add2(sum, pk2(exp2_approx(e0), exp2_approx(e1)));
        }
      }
      float t0, t1;
      upk2(sum, t0, t1);
      t = t0 + t1;
    }
    if (!(t <= (float)(U * T::PER)) || big(m)) {  // hardly ever: a NaN, infinities, masked values alone, or nothing yet
      t = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[T::PER];
        T::widen(now[u], x);
#pragma unroll
        for (int e = 0; e < T::PER; ++e) {
          const float y = tame(x[e]);
          t += exp2_approx(big(m) ? (y - m) * kLog2e : fmaf(y, kLog2e, -r));
        }
      }
    }
    s += t;
    float bound = unordered(*(volatile int*)&sh.bound);
    if (first) {
      // The block's K-th largest of its 256 threads' largest values: no value below that is among the K best.  (Of 8192 values in random
      // order some 8 come through for K = 8 and 34 for K = 32.)
      sh.top[threadIdx.x] = (uint32_t)ordered(top) ^ 0x80000000u;
      __syncthreads();
      uint32_t x[kSelWarps];
#pragma unroll
      for (int i = 0; i < kSelWarps; ++i) x[i] = sh.top[32 * i + lane];
      // (bits below -inf's are no number: then all values count)
      const int o = (int)(bound_of<18>(x, a.beams) ^ 0x80000000u);
      if (o > ordered(-INFINITY)) {
        bound = unordered(o);
        if (threadIdx.x == 0) atomicMax(&sh.bound, o);
      }
    }
    // (behind the first turn values like the K-th have higher places than it)
    uint32_t hits = __ballot_sync(0xffffffffu, top >= bound && (!last.real() || top > last.value()));
    if (hits) {
      // of lanes with -inf alone only the lowest places matter, and only as long as the list is not full
      if (first) hits &= __ballot_sync(0xffffffffu, top > -INFINITY) | (uint32_t)((1ull << (a.beams + T::PER - 1) / T::PER) - 1);
      // a lane's values side by side over the warp
      const int u = lane / T::PER, e = lane % T::PER, end = min(a.vocab, w1 * T::PER);
      int n = 0;  // candidates found
      auto look = [&](int src) {
        float x = -INFINITY;
        if (u < up) {
          const int i = (u * 32 + src) * T::PER + e + skew;
          if constexpr (DT == KVQ_DT_F32)
            x = reinterpret_cast<const float*>(in_slot)[i];
          else if constexpr (DT == KVQ_DT_BF16)
            x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(in_slot)[i] << 16);
          else
            x = __half2float(reinterpret_cast<const __half*>(in_slot)[i]);
        }
        return tame(x);
      };
      auto keep = [&](float x, int src, bool there) {
        const int at = (w - lane + src + u * 32) * T::PER + e;
        const LogitKey key = LogitKey::of(x, at);
        const bool in = there && u < up && x >= bound && at < end && key.before(last);
        const uint32_t pass = __ballot_sync(0xffffffffu, in);
        if (in) found[n + __popc(pass & ((1u << lane) - 1u))] = key;
        n += __popc(pass);
      };
#pragma unroll 1
      while (hits) {  // two lanes' at a time
        const int s0 = __ffs(hits) - 1;
        hits &= hits - 1;
        const bool two = hits != 0;
        const int s1 = two ? __ffs(hits) - 1 : s0;
        hits &= hits - 1;
        const float x0 = look(s0), x1 = look(s1);
        keep(x0, s0, true);
        keep(x1, s1, two);
#pragma unroll 1
        while (n >= 32 || (!hits && n > 0)) {
          const int take = min(n, 32);
          n -= take;
          __syncwarp();
          join_found(list, found + n, take, room);
          last = list.of_lane(a.beams - 1);
        }
      }
      if (lane == 0 && last.real()) atomicMax(&sh.bound, ordered(last.value()));
    }
    first = false;
    __syncwarp();  // before the slot is written again
  }
  // the block's
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  s *= rescale(m, wm);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    sh.m[warp] = wm;
    sh.s[warp] = s;
  }
  list = join_warps(sh, list, a.beams);
  if (warp) return;
  const float pm = lane < kSelWarps ? sh.m[lane] : -FLT_MAX, ps = lane < kSelWarps ? sh.s[lane] : 0.f;
  float bm = pm;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
  float bs = ps * rescale(pm, bm);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) bs += __shfl_xor_sync(0xffffffffu, bs, o);
  if (lane == 0) a.ws.sums[piece] = make_float2(bm, bs);
  if (lane < a.beams) a.ws.best[piece * a.beams + lane] = list.k;
  __syncwarp();  // before the ticket
}

// More candidates at one bound than shared memory takes: those of equal scores.  32 of them a warp at a time, those before its K-th so far.
template <class F>
__device__ __noinline__ ScoreKey join_ties(SelectShared& sh, int N, int K, const int64_t* from, const F& candidate) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ScoreKey list = ScoreKey::none(), last = list;
  ScoreKey* const found = sh.found[warp];
  int n = 0;
  __syncthreads();  // `found` is where the candidates were
#pragma unroll 1
  for (int c0 = warp * 32; c0 < N; c0 += kSelThreads) {
    const int c = c0 + lane;
    const ScoreKey x = c < N ? candidate(c, __ldcg(from + c)) : ScoreKey::none();
    const bool in = x.before(last);
    const uint32_t pass = __ballot_sync(0xffffffffu, in);
    if (in) found[n + __popc(pass & ((1u << lane) - 1u))] = x;
    n += __popc(pass);
    const bool end = c0 + kSelThreads >= N;
#pragma unroll 1
    while (n >= 32 || (end && n > 0)) {
      const int take = min(n, 32);
      n -= take;
      __syncwarp();
      join_found(list, found + n, take, sh.room[warp]);
      last = list.of_lane(K - 1);
    }
  }
  return join_warps(sh, list, K);
}

// The group's last block: log-sums of its rows, then the K best of all their lists, in 64 bits.
__device__ __forceinline__ void join_group(const SelectArgs& a, SelectShared& sh, int group) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.beams, S = a.splits;
  const int64_t row0 = (int64_t)group * K;
  const int N = K * S * K;
  const int64_t* from = a.ws.best + row0 * S * K;
  const int64_t mine_at_first = (int)threadIdx.x < N ? __ldcg(from + threadIdx.x) : INT64_MIN;
  {
    // all rows at a time, by 32 or 8 lanes each: 64-bit arithmetic is slow, and no faster for fewer lanes
    const int G = K <= kSelWarps ? 32 : 8, b = (warp * 32 + lane) / G, l = lane & (G - 1);
    const bool there = b < K;
    const float2* p = a.ws.sums + (row0 + (there ? b : 0)) * S;
    const int done = there && a.done ? a.done[row0 + b] != 0 : 0;
    const float score = there ? a.scores[row0 + b] : 0.f;
    const float2 q = l < S ? __ldcg(p + l) : make_float2(-FLT_MAX, 0.f);  // (of a finished beam: nothing that counts)
    float m = q.x;
#pragma unroll 1
    for (int k = l + G; k < S; k += G) m = fmaxf(m, __ldcg(&p[k].x));
#pragma unroll 1
    for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double sum = (double)q.y * (double)rescale(q.x, m);
#pragma unroll 1
    for (int k = l + G; k < S; k += G) {
      const float2 r = __ldcg(p + k);
      sum += (double)r.y * (double)rescale(r.x, m);
    }
#pragma unroll 1
    for (int o = min(G / 2, S > 16 ? 16 : S > 8 ? 8 : S > 1 ? 4 : 0); o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (there && l == 0) {
      sh.done[b] = done;
      // apart, so that rows of the type's lowest value keep their log-sum
      sh.max[b] = (double)m;
      // nothing may follow: every candidate is -inf all the same
      sh.log_sum[b] = sum > 0 ? log_of(sum) + (big(m) ? 0.0 : (double)reference(m) * (1.0 / (double)kLog2e) - (double)m) : 0.0;
      sh.score[b] = (double)tame(score);
    }
    if (threadIdx.x == 0) sh.count = 0;
    if (threadIdx.x < 32) sh.room[0][threadIdx.x] = ScoreKey::none();
  }
  __syncthreads();
  auto candidate = [&](int c, int64_t key) {
    const LogitKey e{key};
    const int b = min(c / (S * K), K - 1), i = c - b * S * K;
    if (sh.done[b]) return i == 0 ? ScoreKey::of(sh.score[b], b * a.vocab + a.eos) : ScoreKey::none();  // one candidate
    // an empty beam: all are -inf, whatever their logits
    if (sh.score[b] == -INFINITY) return i < min(K, a.vocab) ? ScoreKey::of(-INFINITY, b * a.vocab + i) : ScoreKey::none();
    if (!e.real()) return ScoreKey::none();
    return ScoreKey::of(sh.score[b] + (((double)e.value() - sh.max[b]) - sh.log_sum[b]), b * a.vocab + e.token());
  };
  auto order = [](const ScoreKey& x) { return (uint32_t)(x.s >> 32) ^ 0x80000000u; };
  // Candidates side by side in shared memory, and ranked there: all of them, or those at or above a bound that the best few of the
  // rows' pieces give (of 32 beams' 1024 some 100).
  int n = N;
  if (N <= kSelThreads) {
    if ((int)threadIdx.x < N) sh.all[threadIdx.x] = candidate(threadIdx.x, mine_at_first);
  } else {
    uint32_t x[4];
    const int lists = K * S;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int list = lists <= 32 ? lane : lane + 32 * i, c = list * K + (lists <= 32 ? i : 0);
      x[i] = list < lists && (lists > 32 || i < K) ? order(candidate(c, __ldcg(from + c))) : 0u;
    }
    const uint32_t t = bound_of<12>(x, K);
#pragma unroll 1
    for (int c0 = warp * 32; c0 < N; c0 += kSelThreads) {
      const int c = c0 + lane;
      const ScoreKey y = c >= N ? ScoreKey::none() : candidate(c, c0 < kSelThreads ? mine_at_first : __ldcg(from + c));
      const uint32_t pass = __ballot_sync(0xffffffffu, y.real() && order(y) >= t);
      int at = 0;
      if (lane == 0 && pass) at = atomicAdd(&sh.count, __popc(pass));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(pass & ((1u << lane) - 1u));
      if ((pass >> lane & 1) && at < kSelThreads) sh.all[at] = y;
    }
    __syncthreads();
    n = sh.count;
  }
  __syncthreads();
  ScoreKey list = ScoreKey::none();
  if (n <= kSelThreads) {
    if (warp * 32 < n) {
      const ScoreKey mine = (int)threadIdx.x < n ? sh.all[threadIdx.x] : ScoreKey::none();
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += sh.all[j].before(mine);
      if (mine.real() && rank < K) sh.room[0][rank] = mine;
    }
    __syncthreads();
    list = sh.room[0][lane];
  } else {
    list = join_ties(sh, N, K, from, candidate);
  }
  if (warp) return;
  if (lane < K) {
    const int b = list.at / a.vocab, t = list.at - b * a.vocab;
    a.scores_out[row0 + lane] = (float)list.value();
    a.tokens[row0 + lane] = t;
    a.parents[row0 + lane] = b;
    if (a.done_out) a.done_out[row0 + lane] = sh.done[b] || t == a.eos;
  }
}

template <int DT>
__global__ void __launch_bounds__(kSelThreads, 4) beam_select_kernel(const __grid_constant__ SelectArgs a) {
  using T = LogitType<DT>;
  __shared__ SelectShared sh;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int split = (int)(blockIdx.x - row * a.splits), group = (int)(row / a.beams), b = (int)(row - (int64_t)group * a.beams);
  if (threadIdx.x == 0) sh.bound = ordered(-INFINITY);
  grid_launch_dependents();
  grid_dependency_wait();
  // read once, before the ticket: behind the group's last one done_out is written, which may be done
  if (threadIdx.x == 0) sh.finished = a.done && a.done[row];
  __syncthreads();
  if (!sh.finished) {
    const char* p = a.logits + (group * a.group_stride + b * a.beam_stride) * T::BYTES;
    const int skew = (int)((uintptr_t)p & 15) / T::BYTES;  // elements between the 16-byte boundary and the row
    const int words = (a.vocab + T::PER - 1) / T::PER;
    const int per = (words + a.splits - 1) / a.splits;
    scan_row<DT>(a, sh, p, skew, min(split * per, words), min((split + 1) * per, words), row * a.splits + split);
  }
  if (threadIdx.x == 0) {  // releases warp 0's results, and acquires the other blocks' where this is the last one
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;\n" : "=r"(before) : "l"(a.ws.tickets + group) : "memory");
    sh.last = before == (uint32_t)(a.beams * a.splits - 1);
  }
  __syncthreads();
  if (!sh.last) return;
  if (threadIdx.x == 0) a.ws.tickets[group] = 0;
  join_group(a, sh, group);
}

// Blocks a row: up to two an SM in all, each with at least a turn of logits to read (8192 of two bytes); at most 4096 candidates a group.
// More of them read sooner and cost more in first turns and joins.  In us with 1, 2, 4, 8, 16 blocks a row, the rule's in brackets (bf16, one call a
// graph): 16 x 8 rows of 32000 20.0 [21.1] 31.3; 16 x 5 of 50257 22.9 21.4 [3: 20.9] 22.7 28.8; 8 x 8 of 131072 30.7 25.2 [27.6] 29.7 35.5;
// 8 x 32 of 32001 [35.6] 45.9 60.2; 4 x 4 of 131072 27.2 21.6 18.3 17.2 [21.3]; 1 x 4 of 131072 26.3 20.7 17.7 16.7 [18.7]; one row of
// 131072 23.3 18.6 15.7 14.6 [13.7].  So the rule is up to a tenth off the best count, a quarter for a few long rows.
int splits_of(int64_t rows, int beams, int vocab) {
  const int64_t want = (int64_t)sm_count() * 2 / std::max<int64_t>(1, rows);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, (int64_t)vocab / 8192, (int64_t)4096 / (beams * beams)}));
}

size_t select_ws(int groups, int beams, int vocab, void* base, SelectWs* w) {
  const int64_t rows = (int64_t)groups * beams, pieces = rows * splits_of(rows, beams, vocab);
  const size_t sums = align_up(sizeof(uint32_t) * (size_t)groups), best = sums + align_up(sizeof(float2) * (size_t)pieces);
  if (w) {
    w->tickets = (uint32_t*)base;
    w->sums = (float2*)((char*)base + sums);
    w->best = (int64_t*)((char*)base + best);
  }
  return best + align_up(sizeof(int64_t) * (size_t)pieces * beams);
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
  {
    // a group's results are written while other groups' inputs are still read
    const uintptr_t list = 4 * (uintptr_t)n_groups * beams, size = dtype == KVQ_DT_F32 ? 4 : 2;
    const uintptr_t all = size * (uintptr_t)((n_groups - 1) * group_stride + (beams - 1) * beam_stride + vocab);
    auto meet = [](const void* x, uintptr_t n, const void* y, uintptr_t m) {
      return x && y && (uintptr_t)x < (uintptr_t)y + m && (uintptr_t)y < (uintptr_t)x + n;
    };
    const void* const out[4] = {scores_out, tokens, parents, done_out};
    for (int i = 0; i < 4; ++i) {
      bool bad = meet(out[i], list, logits, all) || (meet(out[i], list, scores, list) && !(i == 0 && scores_out == scores)) ||
                 (meet(out[i], list, done, list) && !(i == 3 && done_out == done));
      for (int j = 0; j < i; ++j) bad |= meet(out[i], list, out[j], list);
      if (bad) return fail(KVQ_ERR_ARG, "an output overlaps another one or an input");
    }
  }
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
  a.splits = splits_of(rows, beams, vocab);
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
