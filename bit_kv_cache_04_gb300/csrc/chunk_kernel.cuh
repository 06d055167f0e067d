// The chunk attention kernel (design in chunk_attention.cuh).
#pragma once

#include <algorithm>
#include <type_traits>

#include "chunk_attention.cuh"

namespace kvq {
namespace {

// ---- mbarriers, TMEM and tcgen05 -------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kChunkPollNs)
      : "memory");
  return ok != 0;
}
// Waits, boundedly, for the phase of that parity.  After too many polls, or
// once another warp has given up, the answer is false and the caller leaves.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
#pragma unroll 1
  for (int i = 0; i < kChunkSpin; ++i) {
    if (bar_test(bar, parity)) return true;
    if (*gave_up) return false;
  }
  *gave_up = 1;
  return false;
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
// x of lane 0: equal in all lanes by construction, so that what follows from
// it stays in uniform registers (operands of products and copies, loop counters, addresses).
template <class T>
__device__ __forceinline__ T uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}
// One lane of a converged warp.  The instructions below and the bulk copies take their
// operands from uniform registers: issued by `lane == 0`, or by several lanes with
// operands of their own, each becomes a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[shared] B[shared]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[shared]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (DT == KVQ_DT_F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Shared-memory operand descriptor: 128-byte swizzle, `lead` and `stride` in
// bytes (K-major tiles: stride between groups of 8 rows, lead unused;
// MN-major tiles: stride between groups of 8 rows of the summed index, lead
// between runs of 64 values of the other one).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((lead >> 4) & 0x3fff) << 16) |
         ((uint64_t)((stride >> 4) & 0x3fff) << 32) | (1ull << 46) | (2ull << 61);
}

// Byte offset of 16-byte piece c (of 8) of row r in a swizzled tile of 128-byte rows.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Sign bits of a lane's four channels (4 lane ..) of a 128-chunk: fetched once per loop, since a
// lane's own word of the parameters is a serialized load.
__device__ __forceinline__ uint32_t lane_signs(const uint32_t* d, int lane) {
  const uint32_t lo = lane & 16 ? d[2] : d[0], hi = lane & 16 ? d[3] : d[1];
  return (lane & 8 ? hi : lo) >> (4 * (lane & 7));
}
// The transform of a 128-chunk held four channels a lane, between the signs s1 and s2 of lane_signs: forward with
// (d1, d2), inverse with (d2, d1).  `factor`: on the result.
__device__ __forceinline__ void rotate_lanes(float (&v)[4], uint32_t s1, uint32_t s2, float factor = 1.f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(__float_as_uint(v[e]) ^ ((s1 << (31 - e)) & 0x80000000u));
  warp_fwht128(v);
  const float c = hadamard_scale() * factor;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(__float_as_uint(v[e] * c) ^ ((s2 << (31 - e)) & 0x80000000u));
}

// ---- the units' line ---------------------------------------------------------------

struct Unit {
  int layer, h, b, rt;
  int n, T, cu;          // rows' tokens, cached tokens, first row of q
  int r0, rows;          // first query row (token * g + head) and rows of this row tile
  int p_lo, p_hi;        // positions of its first and last token
  int lo;                // first token of the window
  int sink;              // tokens [0, sink) visible besides
  int st, lo_tile, nt;   // sink tiles, first window tile, tiles
  // of a planned unit (SEG): b and T: the prefix; rt: its number; n: where its own tiles begin in the list; st: prefix tiles
};

// One CTA's run of a unit: tiles [t0, t1) of it.  Each warp keeps its own in shared memory: registers are short.
struct Run {
  Unit u;
  int t0, t1;
  int pos;               // place of the run's first tile on the line
  int first;             // the CTA's first run
};

struct LineStart {  // found once per CTA
  int lh, b, rt, tile;
  int begin, end;  // the CTA's stretch of the line
  int per_cta;
};

// r / g for query rows (g <= 8, r < 2^28: exact with the rounded-up reciprocal)
__device__ __forceinline__ int div_g(const ChunkArgs& a, int r) {
  return a.lo.g == 1 ? r : (int)__umulhi((uint32_t)r, a.g_magic);
}

__device__ __forceinline__ bool valid_seq(const ChunkArgs& a, int b, int* n, int* T, int* cu) {
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), t = __ldg(a.seq_lens + b);
  *cu = c0;
  *n = (int)((uint32_t)c1 - (uint32_t)c0);
  *T = t;
  return c0 >= 0 && c1 >= c0 && c1 <= a.total_q && c1 - c0 <= a.max_q && t >= c1 - c0 && t <= a.lo.max_T;
}

// (The plan is read past the first-level cache: this grid may begin while the plan is still being written, and what an
// SM has cached of an earlier one at that time would stay.  With non-coherent loads the roles of a CTA saw different units, now and then.)
// SEG: unit i of the plan; false where it is none.  What could lead outside the call's tensors is checked again.
template <int D, int RT>
__device__ __forceinline__ bool planned_unit(const ChunkArgs& a, int i, Unit& u) {
  constexpr int NT = chunk_tile(D);
  const int4 x = __ldcg(reinterpret_cast<const int4*>(a.units + i)), y = __ldcg(reinterpret_cast<const int4*>(a.units + i) + 1);
  u.rt = i;
  u.cu = x.x;
  u.r0 = x.y;
  u.rows = x.z;
  u.b = x.w;
  u.T = y.x;
  u.n = y.y;
  u.p_lo = y.w;
  u.p_hi = u.T - 1;
  u.lo = u.sink = u.lo_tile = 0;
  u.st = u.T / NT;
  u.nt = u.st + y.z;
  return u.rows > 0 && u.rows <= min(RT, a.most_rows) && u.r0 >= 0 && u.cu >= 0 && u.cu + div_g(a, u.r0 + u.rows - 1) < a.total_q &&
         (uint32_t)u.b < (uint32_t)a.lo.B && (uint32_t)u.T <= (uint32_t)a.lo.max_T && u.n >= 0 && y.z >= 0 && u.n <= a.own_tiles - y.z && u.nt > 0;
}
// Whether the plan is one for the call's sizes: then its units and tiles are where the call looks for them.
__device__ __forceinline__ bool plan_fits(const ChunkArgs& a) {
  const int4 x = __ldcg(reinterpret_cast<const int4*>(a.plan));
  return x.x == a.total_q && x.y == a.max_q && x.z == a.max_group_q && x.w == a.n_groups;
}
// Places on the line before a unit's tiles: what a unit costs whatever its length, in tiles (SEG).
template <bool SEG>
__device__ __forceinline__ int unit_cost(const ChunkArgs& a) {
  return SEG ? a.unit_cost : 0;
}

template <int D, int RT>
__device__ __forceinline__ void unit_tiles(const ChunkArgs& a, Unit& u) {
  constexpr int NT = chunk_tile(D);
  u.r0 = u.rt * RT;
  u.rows = min(RT, u.n * a.lo.g - u.r0);
  u.p_lo = u.T - u.n + div_g(a, u.r0);
  u.p_hi = u.T - u.n + div_g(a, u.r0 + u.rows - 1);
  u.lo = a.window ? max(0, u.p_lo - a.window + 1) : 0;
  u.sink = min(a.sinks, u.lo);
  u.lo_tile = u.lo / NT;
  u.st = min((u.sink + NT - 1) / NT, u.lo_tile);
  u.nt = u.st + u.p_hi / NT - u.lo_tile + 1;
}

template <int D, int RT>
__device__ __forceinline__ int seq_row_tiles(const ChunkArgs& a, int n) {
  return (n * a.lo.g + RT - 1) / RT;
}

// Tiles of sequence b (one layer and kv head): summed by one thread, or by the 32 lanes of a warp.  SEG: of unit b, one thread.
template <int D, int RT, bool SEG>
__device__ __forceinline__ int seq_tiles(const ChunkArgs& a, int b, int lane, int lanes, bool* bad) {
  Unit u;
  if constexpr (SEG) return planned_unit<D, RT>(a, b, u) ? u.nt + unit_cost<SEG>(a) : 0;
  if (!valid_seq(a, b, &u.n, &u.T, &u.cu)) {
    *bad = true;
    return 0;
  }
  int sum = 0;
  const int nrt = seq_row_tiles<D, RT>(a, u.n);
#pragma unroll 1
  for (u.rt = lane; u.rt < nrt; u.rt += lanes) {
    unit_tiles<D, RT>(a, u);
    sum += u.nt;
  }
  return sum;
}

// The CTA's first run (step 0) or the one after r; false past the last.  One lane of a warp.
template <int D, int RT, bool SEG>
__device__ __forceinline__ bool step_run(const ChunkArgs& a, const LineStart& s, Run& r, int step) {
  Unit u = r.u;
  int pos, t0;
  if constexpr (SEG) {
    const int cost = unit_cost<SEG>(a);
    if (step == 0) {
      pos = s.begin;
      if (pos >= s.end) return false;
      u.layer = s.lh / a.lo.H;
      u.h = s.lh % a.lo.H;
      (void)planned_unit<D, RT>(a, s.b, u);
      t0 = s.tile - cost;
      if (t0 < 0) {  // the stretch begins before the unit's tiles
        pos -= t0;
        t0 = 0;
      }
    } else {
      pos = r.pos + r.t1 - r.t0;
      if (pos >= s.end) return false;
      pos += cost;
      t0 = 0;
      int i = u.rt;
      do {
        if (++i == a.n_units) {
          i = 0;
          if (++u.h == a.lo.H) {
            u.h = 0;
            if (++u.layer == a.n_layers) return false;
          }
        }
      } while (!planned_unit<D, RT>(a, i, u));
    }
    if (pos >= s.end) return false;
    r.u = u;
    r.t0 = t0;
    r.t1 = min(u.nt, t0 + s.end - pos);
    r.pos = pos;
    r.first = step == 0;
    return true;
  }
  if (step == 0) {
    pos = s.begin;
    if (pos >= s.end) return false;
    u.layer = s.lh / a.lo.H;
    u.h = s.lh % a.lo.H;
    u.b = s.b;
    u.rt = s.rt;
    (void)valid_seq(a, s.b, &u.n, &u.T, &u.cu);
    t0 = s.tile;
  } else {
    pos = r.pos + r.t1 - r.t0;
    if (pos >= s.end) return false;
    t0 = 0;
    ++u.rt;
    if (u.rt >= seq_row_tiles<D, RT>(a, u.n)) {  // the next sequence with rows, of the same or the next kv head, layer
      u.rt = 0;
      bool found;
      do {
        if (++u.b == a.lo.B) {
          u.b = 0;
          if (++u.h == a.lo.H) {
            u.h = 0;
            if (++u.layer == a.n_layers) return false;  // only where lengths changed under the kernel
          }
        }
        found = valid_seq(a, u.b, &u.n, &u.T, &u.cu) && u.n > 0;
      } while (!found);
    }
  }
  unit_tiles<D, RT>(a, u);
  r.u = u;
  r.t0 = t0;
  r.t1 = min(u.nt, t0 + s.end - pos);
  r.pos = pos;
  r.first = step == 0;
  return true;
}
template <int D, int RT, bool SEG>
__device__ __forceinline__ bool warp_run(const ChunkArgs& a, const LineStart& s, Run& r, int step) {
  bool more = false;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) more = step_run<D, RT, SEG>(a, s, r, step);
  __syncwarp();  // the run is read by every lane
  return __shfl_sync(0xffffffffu, (int)more, 0) != 0;
}

// ---- dequantization --------------------------------------------------------------------

// 32 codes of BITS bits at p (2-byte aligned) as fp16 pairs, exact: signed
// codes, or the raw fields (RAW: asymmetric blocks).
__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// fields at bits [0, w) of each half, as fp16 integers minus the bias: 1024 + field is exact in fp16
// (BF: the same in bf16, where 128 + field is exact).  `one`: 1024 in both halves, whose last bit counts 1; or 64 or 4, whose
// last bit counts 2^-4 or 2^-8, for codes times that.
constexpr uint32_t kOnes = 0x64006400u;
template <bool BF = false>
__device__ __forceinline__ uint32_t field_pair(uint32_t x, uint32_t mask, uint32_t bias, uint32_t one = kOnes) {
  if constexpr (BF) {
    const uint32_t v = (x & mask) | 0x43004300u, b = 0x43004300u + bias * 0x10001u;
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  return hsub2u((x & mask) | one, one + bias * 0x10001u);
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint32_t v;
  asm volatile("{\n .reg .u16 t;\n ld.shared.u16 t, [%1];\n cvt.u32.u16 %0, t;\n}\n" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds_half(uint32_t at) { return __half2float(__ushort_as_half((uint16_t)lds16(at))); }
// n words from a 2-byte aligned shared address (aligned loads, shifted; the staging
// area has a word to spare behind its last slot)
template <int N>
__device__ __forceinline__ void load_words(uint32_t p, uint32_t (&w)[N]) {
  const uint32_t a = p & ~3u, sh = (p & 2) * 8;
  uint32_t x[N + 1];
#pragma unroll
  for (int i = 0; i <= N; ++i) x[i] = lds32(a + 4 * i);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], sh);
}
template <int BITS, bool RAW, bool BF = false>
__device__ __forceinline__ void codes32(uint32_t p, uint32_t (&h)[16], uint32_t one = kOnes) {
  uint32_t w[BITS];
  load_words(p, w);
  if constexpr (BITS == 4) {
    constexpr uint32_t bias = RAW ? 0 : 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = w[i] >> 4;
      h[4 * i] = field_pair<BF>(__byte_perm(w[i], v, 0x0400), 0x000f000fu, bias, one);
      h[4 * i + 1] = field_pair<BF>(__byte_perm(w[i], v, 0x1511), 0x000f000fu, bias, one);
      h[4 * i + 2] = field_pair<BF>(__byte_perm(w[i], v, 0x2622), 0x000f000fu, bias, one);
      h[4 * i + 3] = field_pair<BF>(__byte_perm(w[i], v, 0x3733), 0x000f000fu, bias, one);
    }
  } else if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = w[i] ^ 0x80808080u;
      h[2 * i] = hsub2u(__byte_perm(u, one, 0x5150), one + 0x00800080u);
      h[2 * i + 1] = hsub2u(__byte_perm(u, one, 0x5352), one + 0x00800080u);
    }
  } else if constexpr (BITS == 3) {
    const uint32_t g[4] = {w[0], __funnelshift_r(w[0], w[1], 24), __funnelshift_r(w[1], w[2], 16), w[2] >> 8};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t t = g[k] >> (6 * j);
        h[4 * k + j] = field_pair<BF>((t & 7u) | ((t & 0x38u) << 13), 0x00070007u, 4, one);
      }
  } else {
    constexpr uint32_t bias = RAW ? 0 : 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t x = (w[i] >> (8 * b)) & 0xffu;
        const uint32_t y = x | (x << 14);  // fields 0 and 2 low; 1 and 3 at bits 16 and 20
        h[8 * i + 2 * b] = field_pair<BF>(y, 0x00030003u, bias, one);
        h[8 * i + 2 * b + 1] = field_pair<BF>(y >> 4, 0x00030003u, bias, one);
      }
  }
}

__device__ __forceinline__ float2 half2_f(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// What a run's decoding needs of its format, in registers: fields of the
// kernel's parameters picked one by one (a reference picked at run time would be
// a chain of dependent loads).
struct RunFmt {
  int bits, group, bb, row;
  bool zp, codebook;
};
__device__ __forceinline__ RunFmt run_fmt(const Layout& lo, int which, bool cold) {
  RunFmt r;
  r.bits = which ? (cold ? lo.vc.bits : lo.vf.bits) : (cold ? lo.kc.bits : lo.kf.bits);
  r.group = which ? (cold ? lo.vc.group : lo.vf.group) : (cold ? lo.kc.group : lo.kf.group);
  r.bb = which ? (cold ? lo.vc.bb : lo.vf.bb) : (cold ? lo.kc.bb : lo.kf.bb);
  r.row = which ? (cold ? lo.vc.row : lo.vf.row) : (cold ? lo.kc.row : lo.kf.row);
  r.zp = (which ? (cold ? lo.vc.zp : lo.vf.zp) : (cold ? lo.kc.zp : lo.kf.zp)) != 0;
  r.codebook = !cold && (which ? lo.vf.codebook : lo.kf.codebook) != 0;
  return r;
}

// Scale and zero of a block; a scale that is not finite (the block's values are unspecified) counts as 0.
struct BlockScale {
  float s, z;
  bool big;  // a value may leave fp16's range
};
__device__ __forceinline__ BlockScale block_scale_of_run(uint32_t blk, const RunFmt& f) {
  BlockScale r;
  r.s = lds_half(blk);
  r.z = f.zp ? lds_half(blk + 2) : 0.f;
  if (!(fabsf(r.s) <= 65504.f)) r.s = 0.f;
  if (!(fabsf(r.z) <= 65504.f)) r.z = 0.f;
  const float top = f.codebook ? 1.f : f.zp ? (float)((1 << f.bits) - 1) : (float)(1 << (f.bits - 1));
  r.big = fabsf(r.s) * top + fabsf(r.z) > 65504.f;
  return r;
}

// codes (fp16 pairs, exact) -> values in the input dtype.  fp16: one rounding of code * scale (+ zero);
// bf16: through fp32, where the product is exact.
template <int DT, bool ZP>
__device__ __forceinline__ void scale32(uint32_t (&h)[16], uint32_t s16, uint32_t z16) {
  if constexpr (DT == KVQ_DT_F16) {
    const uint32_t ss = __byte_perm(s16, 0, 0x1010), zz = __byte_perm(z16, 0, 0x1010);
    const __half2 s2 = *reinterpret_cast<const __half2*>(&ss), z2 = *reinterpret_cast<const __half2*>(&zz);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 c = *reinterpret_cast<const __half2*>(&h[i]);
      const __half2 v = ZP ? __hfma2(c, s2, z2) : __hmul2(c, s2);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  } else {
    const float s = __half2float(__ushort_as_half((uint16_t)s16)), z = __half2float(__ushort_as_half((uint16_t)z16));
    const uint64_t s2 = pk2(s, s), z2 = pk2(z, z);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 c = half2_f(h[i]);
      const uint64_t c2 = pk2(c.x, c.y), v = ZP ? fma2(c2, s2, z2) : mul2(c2, s2);
      float x, y;
      upk2(v, x, y);
      h[i] = pack16<DT>(x, y);
    }
  }
}

// The same for bf16 codes of at most 4 bits, symmetric blocks, two instructions a pair: the scale is the exact sum of
// two bf16 (11 bits: 8 and the rest), a code times the rest is exact (4 + 3 bits), and the fused product rounds
// once, so the values are those of the fp32 path bit for bit (1000-token chunk of 256-channel heads, when keys took it too:
// 756 -> 709 us).
__device__ __forceinline__ void scale32_bf(uint32_t (&h)[16], uint32_t s16) {
  const float s = __half2float(__ushort_as_half((uint16_t)s16));
  const __nv_bfloat16 hi = __float2bfloat16_rn(s), lo = __float2bfloat16_rn(s - __bfloat162float(hi));
  const __nv_bfloat162 hi2 = __halves2bfloat162(hi, hi), lo2 = __halves2bfloat162(lo, lo);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat162 c = *reinterpret_cast<const __nv_bfloat162*>(&h[i]);
    const __nv_bfloat162 v = __hfma2(c, hi2, __hmul2(c, lo2));
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <int DT>
__device__ __forceinline__ float keep_range(float x) {
  if constexpr (DT == KVQ_DT_F16) return isinf(x) || isnan(x) ? x : fminf(fmaxf(x, -65504.f), 65504.f);
  return x;
}

// The scores' operands are fp16 whatever the input's type: 11 bits instead of bf16's 8, where it counts most (with a
// 15-fold outlier channel a bf16 key is off by 2^-9 of the score).  Keys of a bf16 cache go in times k_pre, 2^-4
// (2^-8 with 8-bit codes), which takes in all that their fp16 scales can hold, and turned queries times q_pre, 2^-4 (the
// turn makes a value up to 11.4 times the largest); the scores are multiplied back.
__device__ __forceinline__ uint32_t score_pack(float x, float y) {
  if (fmaxf(fabsf(x), fabsf(y)) > 65504.f) {  // hardly ever
    x = keep_range<KVQ_DT_F16>(x);
    y = keep_range<KVQ_DT_F16>(y);
  }
  return pack16<KVQ_DT_F16>(x, y);
}
// four channels of a turned query
template <int DT>
__device__ __forceinline__ uint2 query_pack(const float (&v)[4]) {
  if constexpr (DT == KVQ_DT_F16) return make_uint2(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]));
  return make_uint2(score_pack(v[0], v[1]), score_pack(v[2], v[3]));
}
// a pair of the input's type
template <int DT>
__device__ __forceinline__ uint32_t score_pair(uint32_t w, float pre) {
  if constexpr (DT == KVQ_DT_F16) return w;
  return score_pack(__uint_as_float(w << 16) * pre, __uint_as_float(w & 0xffff0000u) * pre);
}

struct TileTokens {
  int t0;        // first token of the tile
  int v0, v1;    // tokens of the tile that some row sees lie in [v0, v1)
};

template <int D>
__device__ __forceinline__ TileTokens tile_tokens(const Unit& u, int j) {
  constexpr int NT = chunk_tile(D);
  TileTokens r;
  const bool sink = j < u.st;
  r.t0 = (sink ? j : u.lo_tile + (j - u.st)) * NT;
  const int lo = sink || u.sink > r.t0 ? 0 : u.lo;  // a window tile may hold sink tokens too
  const int hi = sink ? u.sink : u.p_hi + 1;
  r.v0 = max(r.t0, lo);
  r.v1 = min(r.t0 + NT, hi);
  return r;
}

// The part of a unit that addresses the cache, by value for the calls below.
struct CachePos {
  int layer, b, h, T, qe, ce;
};

// SEG: a tile's entry says where it is.  Of a unit's `nt` tiles the `n` own ones are spread evenly among those of the prefix, so that every
// CTA's stretch has its share of them: they cost more (pages of another sequence each, ragged ends, 16-bit windows: 8 prompts with 8 beams each
// behind 16-bit windows of 128 tokens took 301 us with the own tiles in a row, 255 us so, when a window still took twice as long).  The loader goes through the unit, and leaves every
// tile's entry in shared memory for the other roles.
struct TileOrder {
  int own, err;  // own tiles before this one; its place times n, less own times nt
  __device__ __forceinline__ void start(const Unit& u, int j) {
    const uint64_t x = (uint64_t)j * (uint32_t)(u.nt - u.st);
    own = (int)(x / (uint32_t)u.nt);
    err = (int)(x - (uint64_t)own * (uint32_t)u.nt);
  }
  // tile j's entry (rows -1: of the prefix, which every row sees), and on to the next one
  __device__ __forceinline__ int4 entry(const ChunkArgs& a, const Unit& u, int j, int NT) {
    const int before = own, n = u.nt - u.st;
    if (j >= u.nt) return make_int4(0, 0, 0, 0);
    err -= u.nt - n;  // (err + n may pass 31 bits where both are large)
    if (err >= 0) {
      ++own;
      return __ldcg(reinterpret_cast<const int4*>(a.own + u.n + before));
    }
    err += u.nt;
    return make_int4(u.b, (j - before) * NT, u.T, -1);
  }
};
template <int D>
__device__ __forceinline__ TileTokens listed_tile(const ChunkArgs& a, const Unit& u, const int4& entry, CachePos& at) {
  constexpr int NT = chunk_tile(D);
  TileTokens r;
  at.layer = u.layer + a.layer0;
  at.h = u.h;
  at.b = entry.x;
  at.T = entry.z;
  at.qe = entry.w < 0 ? at.T : q_end_of(a.lo, at.T);  // a prefix is packed to its end
  at.ce = 0;
  r.t0 = r.v0 = entry.y;
  r.v1 = min(r.t0 + NT, at.T);
  return r;
}

// Tile j of a unit: its tokens, and where they are.
template <int D, bool SEG>
__device__ __forceinline__ TileTokens unit_tile(const ChunkArgs& a, const Unit& u, int j, CachePos& at, const int4* entry) {
  at.layer = u.layer + a.layer0;
  at.h = u.h;
  if constexpr (SEG) {
    return listed_tile<D>(a, u, *entry, at);
  } else {
    at.b = u.b;
    at.T = u.T;
    at.qe = q_end_of(a.lo, u.T);
    at.ce = c_end_of(a.lo, u.T);
    return tile_tokens<D>(u, j);
  }
}
// Position of the unit's row r: the last token that it sees.
template <bool SEG>
__device__ __forceinline__ int row_pos(const ChunkArgs& a, const Unit& u, int r) {
  const int tok = div_g(a, u.r0 + r);
  return SEG ? __ldcg(&a.where[u.cu + tok].x) : u.T - u.n + tok;
}

// Where the runs of 32 values of a tensor's tile sit.  Rows of the tile in
// shared memory are tokens (per-token blocks, runs along channels) or
// channels (per-channel blocks, runs along tokens).  A piece is half a tile: 256 runs, four a
// lane of its two warps.  Consecutive lanes take consecutive rows of one run, so that their
// 16-byte stores fall into different banks.
template <int D>
struct RunPlace {
  static constexpr int NT = chunk_tile(D), PIECE = NT / 2;
  // run i of lane `lane` of the piece's warp `part`: first token from the piece's, row and run in the tile's first half.
  // i steps along rows.  Per-channel: a warp takes a 32-token group (of two) or half of the channels.
  // Per-token: four runs of a row side by side; a warp takes half of the tokens, or of the channels (D = 256).
  __device__ __forceinline__ static void of(bool per_channel, int part, int i, int lane, int* toff, int* row, int* run) {
    if (per_channel) {
      *row = i * 32 + lane + (D == 128 ? 0 : 128 * part);
      *run = D == 128 ? part : 0;
      *toff = 32 * *run;
    } else {
      *row = *toff = (lane & 7) + 8 * i + (D == 128 ? 32 * part : 0);
      *run = (lane >> 3) + (D == 128 ? 0 : 4 * part);
    }
  }
  // block and codes of a run (channel `row` of a 32-token group, or run `run` of a token) in the staged piece
  __device__ __forceinline__ static void at(bool per_channel, const RunFmt& f, int sub_bytes, int t, int row, int run,
                                            uint32_t* b, uint32_t* c) {
    const uint32_t sub = (t >> 5) * sub_bytes;
    if (per_channel) {
      *b = sub + row * f.bb;
      *c = *b + (f.zp ? 4 : 2);
    } else {
      const bool one = f.group == 32;  // a block is one run, or four
      *b = sub + (t & 31) * f.row + (one ? run : run >> 2) * f.bb;
      *c = *b + (f.zp ? 4 : 2) + (one ? 0 : (run & 3) * 4 * f.bits);
    }
  }
  // shared-memory row of a run in the tile
  __device__ __forceinline__ static uint32_t line_at(uint32_t dst, int row, int run, int rows) {
    return dst + (uint32_t)(run >> 1) * rows * 128 + row * 128;
  }
};

__device__ __forceinline__ void store_run(uint32_t line, int row, int run, const uint32_t (&h)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(line + ((((run & 1) * 4 + j) ^ (row & 7)) << 4)),
                 "r"(h[4 * j]), "r"(h[4 * j + 1]), "r"(h[4 * j + 2]), "r"(h[4 * j + 3])
                 : "memory");
}

// 16-bit window values as they are; in V's tile values that are not finite become 0 (see add_nonfinite)
template <int DT>
__device__ __forceinline__ uint32_t clean(uint32_t w, int which, volatile uint32_t* nonfinite) {
  if (which == 0) return w;
  constexpr uint32_t E = DT == KVQ_DT_F16 ? 0x7c00u : 0x7f80u;
  if ((w & E) == E) {
    *nonfinite = 1;
    w &= 0xffff0000u;
  }
  if (((w >> 16) & E) == E) {
    *nonfinite = 1;
    w &= 0x0000ffffu;
  }
  return w;
}

// 32 channels of window token t (zeros past the length)
template <int DT>
__device__ __forceinline__ void raw_token_run(const ChunkArgs& a, const CachePos& u, int which, int t, int run,
                                              volatile uint32_t* nonfinite, uint32_t (&h)[16]) {
  if (t >= u.T) {  // no address is formed: a cache without a window has no slots (and comes by here behind its last token)
#pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = 0;
    return;
  }
  const uint4* p = reinterpret_cast<const uint4*>(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t)) + run * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = p[j];
    h[4 * j] = clean<DT>(v.x, which, nonfinite);
    h[4 * j + 1] = clean<DT>(v.y, which, nonfinite);
    h[4 * j + 2] = clean<DT>(v.z, which, nonfinite);
    h[4 * j + 3] = clean<DT>(v.w, which, nonfinite);
  }
}
// channel c of window tokens t .. t + 31 (zeros past the length)
template <int DT>
__device__ __forceinline__ void raw_channel_run(const ChunkArgs& a, const CachePos& u, int which, int t, int c,
                                                volatile uint32_t* nonfinite, uint32_t (&h)[16]) {
  const uint16_t* p = resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t) + c;
  const int D = a.lo.D, ring = a.lo.ring;
  int left = ring - t % ring;  // slots until the ring wraps
  uint32_t x[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    x[j] = *p;  // slots past the length exist, and count as zeros below
    --left;
    p += left == 0 ? (int64_t)D - (int64_t)ring * D : (int64_t)D;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (t + j >= u.T) x[j] = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) h[j] = clean<DT>(x[2 * j] | (x[2 * j + 1] << 16), which, nonfinite);
}

// Window tokens [t0, t1) of a rotated format, turned into the rotated domain by one warp.
template <int D, int DT>
__device__ __forceinline__ void rotated_window(const ChunkArgs& a, const CachePos& u, int which, int part, uint32_t dst,
                                               int tile0, int a0, int t0, int t1, int lane, volatile uint32_t* nonfinite) {
  constexpr int NT = chunk_tile(D);
  for (int t = t0; t < t1; ++t) {
    if (D == 128 && ((t - a0) >> 5) != part) continue;  // D = 128: the warp's 32 tokens
    const uint2* p = reinterpret_cast<const uint2*>(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t));
#pragma unroll
    for (int c = 0; c < D / 128; ++c) {
      if (D == 256 && c != part) continue;  // D = 256: the warp's 128 channels
      const uint2 w = p[32 * c + lane];
      const uint32_t w0 = clean<DT>(w.x, which, nonfinite), w1 = clean<DT>(w.y, which, nonfinite);
      float v[4] = {in_to_f32((uint16_t)w0, DT), in_to_f32((uint16_t)(w0 >> 16), DT), in_to_f32((uint16_t)w1, DT),
                    in_to_f32((uint16_t)(w1 >> 16), DT)};
      rotate_lanes(v, lane_signs(a.lo.d1, lane), lane_signs(a.lo.d2, lane));
      const int ch = 128 * c + 4 * lane;
      const uint32_t at = dst + (uint32_t)(ch >> 6) * NT * 128 + swz(t - tile0, (ch & 63) >> 3) + (ch & 4) * 2;
      uint32_t o0, o1;
      if (DT == KVQ_DT_F16 || which) {
        o0 = pack16<DT>(keep_range<DT>(v[0]), keep_range<DT>(v[1]));
        o1 = pack16<DT>(keep_range<DT>(v[2]), keep_range<DT>(v[3]));
      } else {
        o0 = score_pack(v[0] * a.k_pre, v[1] * a.k_pre);
        o1 = score_pack(v[2] * a.k_pre, v[3] * a.k_pre);
      }
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at), "r"(o0), "r"(o1) : "memory");
    }
  }
}

// rotate_lanes of four rows, eight lanes a row: lane 8 r + q holds channels 32 j + 4 q + e of row r.  The same operations in the same
// order, with 48 shuffles where a row at a time takes 80.  Bits 4 j + e of s1 and s2: the signs.
__device__ __forceinline__ void rotate_rows(float (&v)[4][4], uint32_t s1, uint32_t s2) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[j][e] = __uint_as_float(__float_as_uint(v[j][e]) ^ ((s1 << (31 - 4 * j - e)) & 0x80000000u));
    const float a0 = v[j][0] + v[j][1], a1 = v[j][0] - v[j][1], a2 = v[j][2] + v[j][3], a3 = v[j][2] - v[j][3];
    v[j][0] = a0 + a2;
    v[j][2] = a0 - a2;
    v[j][1] = a1 + a3;
    v[j][3] = a1 - a3;
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const float sign = lane & m ? -1.f : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = fmaf(v[j][e], sign, __shfl_xor_sync(0xffffffffu, v[j][e], m));  // exact: v + o or o - v, rounded once
  }
  const float c = hadamard_scale();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a0 = v[0][e] + v[1][e], a1 = v[0][e] - v[1][e], a2 = v[2][e] + v[3][e], a3 = v[2][e] - v[3][e];
    v[0][e] = a0 + a2;
    v[2][e] = a0 - a2;
    v[1][e] = a1 + a3;
    v[3][e] = a1 - a3;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[j][e] = __uint_as_float(__float_as_uint(v[j][e] * c) ^ ((s2 << (31 - 4 * j - e)) & 0x80000000u));
}

// 16 bytes from global memory to shared, in flight until copies_land.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_land() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// The same (SEG).  All tokens' values are first copied, as they are, to where the turned ones will stand, so that one load's latency
// is paid a piece; then four tokens are turned at a time, by eight lanes each.
// (One token at a time, with a load's and the shuffles' latencies each, a tile of 128 window tokens took some 40 us.  8 prompts with 8 beams
// each behind 16-bit windows of 128 tokens took 208 us with four tokens' loads in flight, 186 us with all of them, 172 us
// with four rows by eight lanes each instead of one row by 32.)
template <int D, int DT>
__device__ __forceinline__ void rotated_window4(const ChunkArgs& a, const CachePos& u, int which, int part, uint32_t dst,
                                               int tile0, int a0, int t0, int t1, int lane, volatile uint32_t* nonfinite) {
  constexpr int NT = chunk_tile(D);
  const int c = D == 256 ? part : 0;  // D = 256: the warp's 128 channels
  if (D == 128) {                     // D = 128: its 32 tokens
    t0 = max(t0, a0 + 32 * part);
    t1 = min(t1, a0 + 32 * part + 32);
  }
  if (t0 >= t1) return;
  dst += 2 * c * NT * 128;
  // a lane's window row, passed on by shuffles: one division by the ring's size for all tokens
  const uint64_t mine = (uint64_t)(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, min(t0 + lane, t1 - 1)) + 128 * c);
  const int ch = lane & 15;  // a 16-byte piece
#pragma unroll 4
  for (int i = 0; i < t1 - t0; i += 2) {
    const int t = i + (lane >> 4);
    const uint64_t row = __shfl_sync(0xffffffffu, mine, t & 31);
    if (t < t1 - t0) copy_16(dst + (uint32_t)(ch >> 3) * NT * 128 + swz(t0 + t - tile0, ch & 7), (const char*)row + 16 * ch);
  }
  const int q = lane & 7, r = lane >> 3;
  uint32_t s1 = 0, s2 = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s1 |= (a.lo.d1[j] >> (4 * q) & 15) << (4 * j);
    s2 |= (a.lo.d2[j] >> (4 * q) & 15) << (4 * j);
  }
  copies_land();
  __syncwarp();
  // rows 0, 1, 4, 5 of eight, then 2, 3, 6, 7: their swizzled pieces lie in all banks
#pragma unroll 1
  for (int i = 0; i < t1 - t0; i += (i & 2) ? 6 : 2) {
    const int t = t0 + i + (r & 1) + 4 * (r >> 1), row = min(t, t1 - 1) - tile0;
    uint32_t at[4];
    float v[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at[j] = dst + (uint32_t)(j >> 1) * NT * 128 + swz(row, 4 * (j & 1) + (q >> 1)) + 8 * (q & 1);
      uint32_t w0, w1;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(w0), "=r"(w1) : "r"(at[j]) : "memory");
      w0 = clean<DT>(w0, which, nonfinite);
      w1 = clean<DT>(w1, which, nonfinite);
      v[j][0] = in_to_f32((uint16_t)w0, DT);
      v[j][1] = in_to_f32((uint16_t)(w0 >> 16), DT);
      v[j][2] = in_to_f32((uint16_t)w1, DT);
      v[j][3] = in_to_f32((uint16_t)(w1 >> 16), DT);
    }
    rotate_rows(v, s1, s2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o0, o1;
      if (DT == KVQ_DT_F16 || which) {
        o0 = pack16<DT>(keep_range<DT>(v[j][0]), keep_range<DT>(v[j][1]));
        o1 = pack16<DT>(keep_range<DT>(v[j][2]), keep_range<DT>(v[j][3]));
      } else {
        o0 = score_pack(v[j][0] * a.k_pre, v[j][1] * a.k_pre);
        o1 = score_pack(v[j][2] * a.k_pre, v[j][3] * a.k_pre);
      }
      if (t < t1) asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at[j]), "r"(o0), "r"(o1) : "memory");
    }
  }
}

// Window tokens [t0, t1) (whole 32-token groups) of a per-channel tensor: a
// lane per token reads 8 channels at a time, and a warp's 2-byte stores of one
// channel are 64 bytes of one row.
template <int D, int DT>
__device__ __forceinline__ void window_groups(const ChunkArgs& a, const CachePos& u, int which, int part, uint32_t dst, int tile0,
                                              int t0, int t1, int lane, volatile uint32_t* nonfinite) {
  for (int g = t0; g < t1; g += 32) {
    if (D == 128 && ((g - tile0) >> 5 & 1) != part) continue;  // D = 128: the warp's group of the piece
    const int t = g + lane, col = t - tile0;  // column of the channel rows
    const bool in = t < u.T;
    const uint4* p = reinterpret_cast<const uint4*>(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, in ? t : g));
    const uint32_t blk = dst + (uint32_t)(col >> 6) * D * 128 + (col & 7) * 2;
    const int c16 = (col & 63) >> 3;
#pragma unroll 1
    for (int c0 = D == 128 ? 0 : part * 16; c0 < (D == 128 ? 16 : part * 16 + 16); c0 += 4) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = p[c0 + k];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4] = {clean<DT>(in ? v[k].x : 0u, which, nonfinite), clean<DT>(in ? v[k].y : 0u, which, nonfinite),
                         clean<DT>(in ? v[k].z : 0u, which, nonfinite), clean<DT>(in ? v[k].w : 0u, which, nonfinite)};
        if (which == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = score_pair<DT>(w[e], a.k_pre);
        }
        const int row = (c0 + k) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)  // row + e has low bits e
          asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(blk + (row + e) * 128 + ((c16 ^ e) << 4)),
                       "h"((uint16_t)(w[e >> 1] >> (16 * (e & 1))))
                       : "memory");
      }
    }
  }
}

// The values of one run in fp32 from its codes, whatever the format; values past fp16's range
// saturate in fp16 (an infinity would turn a masked token's zero probability into NaN).
template <int DT>
__device__ __forceinline__ void general_run(RunFmt f, uint32_t blk, uint32_t codes, const uint32_t* pair_table,
                                         uint32_t line, int row, int run, bool key, float pre) {
  uint32_t h[16];
  if (f.codebook) {
    uint32_t w[4];
    load_words(codes, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = pair_table[(w[i / 4] >> (8 * (i % 4))) & 0xff];
  } else if (f.bits == 4) {
    codes32<4, true>(codes, h);
  } else if (f.bits == 8) {
    codes32<8, true>(codes, h);
  } else if (f.bits == 3) {
    codes32<3, true>(codes, h);
  } else {
    codes32<2, true>(codes, h);
  }
  const float bias = f.zp || f.codebook ? 0.f : f.bits == 4 ? 8.f : f.bits == 2 ? 2.f : 0.f;  // 8- and 3-bit codes are signed already
  const BlockScale b = block_scale_of_run(blk, f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 c = half2_f(h[i]);
    float x = fmaf(c.x - bias, b.s, b.z), y = fmaf(c.y - bias, b.s, b.z);
    if constexpr (DT == KVQ_DT_F16) {
      x = fminf(fmaxf(x, -65504.f), 65504.f);
      y = fminf(fmaxf(y, -65504.f), 65504.f);
    }
    h[i] = DT == KVQ_DT_F16 || !key ? pack16<DT>(x, y) : score_pack(x * pre, y * pre);
  }
  store_run(line, row, run, h);
}

// One lane's four runs of a piece that lies in one format, wholly in view:
// the hot path.  Its loop is kept short, and everything else out of line: the five roles run
// different code at the same time, and what they run has to fit the instruction cache (with
// this loop unrolled eight times the single tokens of 64 sequences took 1.3 times as long).
struct PiecePlace {
  uint32_t blk, codes, step;  // first run's block and codes in the staged piece; to the next run
  uint32_t line, line_step;   // the same in the tile
  uint32_t piece16[4];        // swizzled places of the run's four 16-byte parts
  int tok;                    // the first run's token of the piece (per-token blocks; the next ones' are 8 apart)
};
// False when a block's values leave fp16's range, or its scale is not finite (the piece is then done again).
// KEY: keys of a bf16 cache, fp16 values times k_pre (`one` is a.k_one); their codes take the factor, exactly.
// RAGGED: only the first `valid` tokens of the piece are there (per-token blocks); the others' values are zeros.
template <int DT, bool KEY, int BITS, bool ZP, bool RAGGED>
__device__ __forceinline__ bool fill_piece(const PiecePlace& q, uint32_t staged, uint32_t tile, int valid, uint32_t one = kOnes) {
  uint32_t most = 0, blk = staged + q.blk, line = tile + q.line;
  int tok = RAGGED ? q.tok : 0;
  const uint32_t codes = q.codes - q.blk;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    uint32_t s16 = lds16(blk), z16 = ZP ? lds16(blk + 2) : 0u;
    if constexpr (RAGGED) {
      if (tok >= valid) s16 = z16 = 0;
      tok += 8;
    }
    uint32_t h[16];
    constexpr bool BF = DT == KVQ_DT_BF16 && !KEY && !ZP && BITS < 8;
    codes32<BITS, ZP, BF>(blk + codes, h, KEY ? one : kOnes);
    most = max(most, s16 & 0x7fffu);
    // the zero's bound is four times the scale's
    if (ZP) most = max(most, DT == KVQ_DT_F16 ? max(z16 & 0x7fffu, 0x800u) - 0x800u : z16 & 0x7fffu);
    if constexpr (BF)
      scale32_bf(h, s16);
    else if constexpr (KEY)  // (0x2800: from 1024, 64 or 4 to 1, 2^-4 or 2^-8)
      scale32<KVQ_DT_F16, ZP>(
          h, s16, ZP ? __half_as_ushort(__hmul(__ushort_as_half((uint16_t)z16), __ushort_as_half((uint16_t)(one - 0x2800u)))) : 0u);
    else
      scale32<DT, ZP>(h, s16, z16);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(line + q.piece16[k]), "r"(h[4 * k]),
                   "r"(h[4 * k + 1]), "r"(h[4 * k + 2]), "r"(h[4 * k + 3])
                   : "memory");
    blk += q.step;
    line += q.line_step;
  }
  // bf16: finite is enough.  fp16: |scale| below 2^15 / the largest code's bound (and a zero below 2^15), so that
  // every value stays below 2^16 less a rounding
  constexpr uint32_t LIMIT = DT != KVQ_DT_F16 ? 0x7c00u : (uint32_t)(15 - (ZP ? BITS : BITS - 1) + 15) << 10;
  return !__any_sync(0xffffffffu, most >= LIMIT);
}

// Half of a piece whose tokens differ in tier, are partly out of view, include pages out of range or the
// 16-bit window, or whose blocks are TBQ4 or hold values past the range: run by run.
template <int D, int DT, bool SEG>
__device__ __forceinline__ void mixed_piece(const ChunkArgs& a, const CachePos& u, int which, int half, int part, int lane,
                                         bool per_channel, bool rotated, int a0, int v0, int v1, uint32_t staged,
                                         uint32_t bad, uint32_t dst, int tile0, bool fresh, const uint32_t* pair_table,
                                         volatile uint32_t* nonfinite) {
  constexpr int NT = chunk_tile(D);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    int toff, row, run;
    RunPlace<D>::of(per_channel, part, i, lane, &toff, &row, &run);
    const int t = a0 + toff, row_t = row + (per_channel ? 0 : half * (NT / 2)), run_t = run + (per_channel ? half * (NT / 64) : 0);
    const uint32_t line = RunPlace<D>::line_at(dst, row_t, run_t, per_channel ? D : NT);
    const bool in = t >= v0 && t < v1;
    if (in && t < u.qe && !((bad >> (toff >> a.copy_shift)) & 1u)) {
      const RunFmt f = run_fmt(a.lo, which, t < u.ce);
      uint32_t blk, codes;
      RunPlace<D>::at(per_channel, f, a.sub_bytes, toff, row, run, &blk, &codes);
      general_run<DT>(f, staged + blk, staged + codes, pair_table, line, row_t, run_t, which == 0, a.k_pre);
    } else if (in && t >= u.qe && !per_channel && !(rotated && t < u.T)) {
      uint32_t h[16];
      raw_token_run<DT>(a, u, which, t, run, nonfinite, h);
      if (which == 0) {
#pragma unroll
        for (int k = 0; k < 16; ++k) h[k] = score_pair<DT>(h[k], a.k_pre);
      }
      store_run(line, row_t, run_t, h);
    } else if ((in && t < u.qe) || fresh) {
      // a page out of range; or a run out of view in a buffer that V has not filled yet: what shared
      // memory held before the kernel must not meet a zero probability
      uint32_t h[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) h[k] = 0;
      store_run(line, row_t, run_t, h);
    }
  }
  // the window tokens of this warp's own half: the same rows or channels as its runs
  if (rotated) {
    __syncwarp();
    const int w0 = max(max(u.qe, a0), v0), w1 = min(min(u.T, a0 + NT / 2), v1);
    if constexpr (SEG)
      rotated_window4<D, DT>(a, u, which, part, dst, tile0, a0, w0, w1, lane, nonfinite);
    else
      rotated_window<D, DT>(a, u, which, part, dst, tile0, a0, w0, w1, lane, nonfinite);
  }
  if (per_channel && v1 > max(u.qe, a0)) {
    __syncwarp();
    window_groups<D, DT>(a, u, which, part, dst, tile0, max(max(u.qe, a0), v0), min(a0 + NT / 2, v1), lane, nonfinite);
  }
}

// Values of a run as code pairs with (scale, zero), or as pairs of the input dtype (window tokens), for the turn in fp32
template <int DT>
struct Loose {
  uint32_t h[16];
  float s, z;
  bool raw;
  __device__ __forceinline__ float2 value(int i) const {
    if (raw) {
      if constexpr (DT == KVQ_DT_F16) return half2_f(h[i]);
      return make_float2(__uint_as_float(h[i] << 16), __uint_as_float(h[i] & 0xffff0000u));
    }
    const float2 c = half2_f(h[i]);
    return make_float2(fmaf(c.x, s, z), fmaf(c.y, s, z));
  }
};

// cos and sin of a 64-bit turn fraction
__device__ __forceinline__ float2 cos_sin(uint64_t turn) {
  float s, c;
  sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// Keys stored pre-RoPE: a piece's runs of channels i and i + D/2 together.
template <int D, int DT>
__device__ __forceinline__ void turned_piece(const ChunkArgs& a, const CachePos& u, const TileTokens& tt, int a0, uint32_t staged,
                                          uint32_t bad, uint32_t dst, int e0, volatile uint32_t* nonfinite) {
  constexpr int NT = chunk_tile(D), PIECE = NT / 2, THREADS = 64;  // the piece's two warps
  const bool per_channel = a.lo.kf.axis == KVQ_AXIS_CHANNEL;
  auto loose = [&](int t, int row, int run, Loose<DT>& l) {
    l.raw = t >= u.qe || ((bad >> ((t - a0) >> a.copy_shift)) & 1u);
    if (!l.raw) {
      const RunFmt f = run_fmt(a.lo, 0, t < u.ce);
      uint32_t blk, codes;
      RunPlace<D>::at(per_channel, f, a.sub_bytes, t - a0, row, run, &blk, &codes);
      const BlockScale b = block_scale_of_run(staged + blk, f);
      l.s = b.s;
      l.z = b.z;
      if (f.bits == 4)
        codes32<4, true>(staged + codes, l.h);
      else if (f.bits == 8)
        codes32<8, true>(staged + codes, l.h);
      else if (f.bits == 3)
        codes32<3, true>(staged + codes, l.h);
      else
        codes32<2, true>(staged + codes, l.h);
      if (!f.zp) l.z = -b.s * (f.bits == 4 ? 8.f : f.bits == 2 ? 2.f : 0.f);  // the bias of raw fields: exact products

    } else if (t < u.qe) {  // a page out of range
#pragma unroll
      for (int i = 0; i < 16; ++i) l.h[i] = 0;
    } else if (per_channel) {
      raw_channel_run<DT>(a, u, 0, t, row, nonfinite, l.h);
    } else {
      raw_token_run<DT>(a, u, 0, t, run, nonfinite, l.h);
    }
  };
  if (per_channel) {
    constexpr int G = PIECE / 32;  // token groups of the piece
    for (int e = e0; e < (D / 2) * G; e += THREADS) {
      const int c = (e & 7) | ((e / (8 * G)) << 3), t = a0 + 32 * ((e >> 3) % G), run = (t - tt.t0) >> 5;
      if (t + 32 <= tt.v0 || t >= tt.v1) continue;
      Loose<DT> x, y;
      loose(t, c, 0, x);
      loose(t, c + D / 2, 0, y);
      const uint64_t f = a.turns[c];
      // token after token the angle grows by the same step: a complex
      // product each, 31 times from an exact start (error below 31 x 2^-22)
      float2 k = cos_sin((uint64_t)t * f);
      const float2 step = cos_sin(f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 xa = x.value(i), ya = y.value(i);
        const float x0 = xa.x * k.x - ya.x * k.y, y0 = ya.x * k.x + xa.x * k.y;
        k = make_float2(k.x * step.x - k.y * step.y, k.y * step.x + k.x * step.y);
        const float x1 = xa.y * k.x - ya.y * k.y, y1 = ya.y * k.x + xa.y * k.y;
        k = make_float2(k.x * step.x - k.y * step.y, k.y * step.x + k.x * step.y);
        x.h[i] = score_pack(x0 * a.k_pre, x1 * a.k_pre);
        y.h[i] = score_pack(y0 * a.k_pre, y1 * a.k_pre);
      }
      store_run(RunPlace<D>::line_at(dst, c, run, D), c, run, x.h);
      store_run(RunPlace<D>::line_at(dst, c + D / 2, run, D), c + D / 2, run, y.h);
    }
  } else {
    constexpr int R = D / 64;  // runs of half a row
    for (int e = e0; e < PIECE * R; e += THREADS) {
      const int run = (e >> 3) % R, t = a0 + ((e & 7) | ((e / (8 * R)) << 3)), row = t - tt.t0;
      if (t < (tt.v0 & ~31) || t >= ((tt.v1 + 31) & ~31)) continue;
      Loose<DT> x, y;
      loose(t, row, run, x);
      loose(t, row, run + R, y);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 k0 = cos_sin((uint64_t)t * a.turns[32 * run + 2 * i]);
        const float2 k1 = cos_sin((uint64_t)t * a.turns[32 * run + 2 * i + 1]);
        const float2 xa = x.value(i), ya = y.value(i);
        x.h[i] = score_pack((xa.x * k0.x - ya.x * k0.y) * a.k_pre, (xa.y * k1.x - ya.y * k1.y) * a.k_pre);
        y.h[i] = score_pack((ya.x * k0.x + xa.x * k0.y) * a.k_pre, (ya.y * k1.x + xa.y * k1.y) * a.k_pre);
      }
      store_run(RunPlace<D>::line_at(dst, row, run, NT), row, run, x.h);
      store_run(RunPlace<D>::line_at(dst, row, run + R, NT), row, run + R, y.h);
    }
  }
}

// ---- staging -----------------------------------------------------------------------------

// Two loader warps, one for K and one for V, bring the packed bytes of their
// pieces into a common ring of shared-memory slots: bulk copies of 32-token subtiles (of pages,
// when those are smaller).  A tile's two pieces are worked out side by side, 16 lanes
// a piece: one lane's addresses are a long chain of dependent instructions.
// Piece i (K, K, V, V) of tile kt is number 4 kt + i and goes to slot number mod slots; its
// barriers are the piece kind's, kt mod kChunkBars: each warp sees every
// phase of the barriers that it waits on, and the ring never spans kChunkBars tiles.
template <int D>
struct Loader {
  static constexpr int NT = chunk_tile(D), PIECE = NT / 2;

  int which, half, ln;       // this lane's piece and its place among the piece's lanes
  const uint8_t *main0, *cold0;  // first row of the unit's (layer, sequence, kv head); of page 0 when paged
  int64_t page_stride;
  int row_main, row_cold;    // bytes per token (per-token) or per 32-token group (per-channel)
  int ring;                  // hot ring in rows (tiers), else 0
  bool per_channel;

  __device__ __forceinline__ void lanes(const ChunkArgs& a, int tensor, int lane) {
    which = tensor;
    half = lane >> 4;
    ln = lane & 15;
    per_channel = (which ? a.lo.vf.axis : a.lo.kf.axis) == KVQ_AXIS_CHANNEL;
    row_main = which ? a.lo.vf.row : a.lo.kf.row;
    row_cold = which ? a.lo.vc.row : a.lo.kc.row;
    ring = a.lo.tiered ? (which ? a.lo.hot_ring_v : a.lo.hot_ring_k) : 0;
  }
  __device__ __forceinline__ void unit(const ChunkArgs& a, const CachePos& u) {
    const uint8_t* m = which ? a.cp.v_main : a.cp.k_main;
    if (a.lo.paged) {
      page_stride = (int64_t)a.lo.H * a.lo.pt * row_main;
      main0 = m + (int64_t)u.layer * a.lo.n_pages * page_stride + (int64_t)u.h * a.lo.pt * row_main;
      cold0 = nullptr;
    } else {
      const int64_t lbh = ((int64_t)u.layer * a.lo.B + u.b) * a.lo.H + u.h;
      main0 = m + lbh * (which ? a.lo.rows_v_main : a.lo.rows_k_main) * row_main;
      cold0 = (which ? a.cp.v_cold : a.cp.k_cold) + lbh * (which ? a.lo.rows_v_cold : a.lo.rows_k_cold) * row_cold;
    }
  }
  // page id of copy c of this lane's piece of a tile (-1 where none is read)
  __device__ __forceinline__ int page_id(const ChunkArgs& a, const CachePos& u, int tile0, int c) const {
    const int t = tile0 + half * PIECE + (c << a.copy_shift);
    if (!a.lo.paged || c >= (PIECE >> a.copy_shift) || t >= u.qe) return -1;
    return __ldg(a.cp.block_table + (int64_t)u.b * a.lo.max_pages + t / a.lo.pt);
  }
  // source and bytes of copy c of this lane's piece (0 bytes: nothing to copy)
  __device__ __forceinline__ int source(const ChunkArgs& a, const CachePos& u, const TileTokens& tt, int c, int pid,
                                        const uint8_t** src, int* at, bool* bad) const {
    const int t = tt.t0 + half * PIECE + (c << a.copy_shift), sub = t & ~31;
    if (c >= (PIECE >> a.copy_shift) || t >= u.qe || sub + 32 <= tt.v0 || sub >= tt.v1) return 0;
    const bool cold = t < u.ce;
    const int row = cold ? row_cold : row_main;
    *at = ((t - tt.t0 - half * PIECE) >> 5) * a.sub_bytes + (per_channel ? 0 : (t & 31) * row);
    if (a.lo.paged) {
      if (pid < 0 || pid >= a.lo.n_pages) {
        *bad = true;
        return 0;
      }
      *src = main0 + pid * page_stride + (int64_t)(t % a.lo.pt) * row;
    } else {
      int r = per_channel ? t >> 5 : t;
      if (ring && !cold) r %= ring;
      *src = (cold ? cold0 : main0) + (int64_t)r * row;
    }
    const int bytes = per_channel ? row : row << a.copy_shift;
    [[maybe_unused]] const CachePtrs& cp = a.cp;
    if (!KVQ_CHECK(*at + bytes <= a.slot_bytes)) return 0;
    return span_ok(a.lo, a.cp, which + (cold ? 2 : 0), *src, bytes) ? bytes : 0;
  }
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, uint32_t src_lo, uint32_t src_hi, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n .reg .b64 src;\n mov.b64 src, {%1, %2};\n"
      " cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [src], %3, [%4];\n}\n" ::"r"(dst),
      "r"(src_lo), "r"(src_hi), "r"(bytes), "r"(bar)
      : "memory");
}

// ---- the kernel ----------------------------------------------------------------------

struct ChunkShared;
struct FewShared;
// SEG: the list's entries of the tiles in flight, written by the loader with a piece: [piece kind][tile mod kChunkBars].  A slot is
// written again eight tiles later: by then the piece four tiles back has been read, the scores six tiles back are
// issued, and with them the outputs eight tiles back, whose softmax was the last to look.
struct TileEntries {
  int4 at[4 * kChunkBars];
};

template <int D, int MODE>
struct ChunkShape {
  static constexpr bool PAIRED = MODE == kChunkPaired, FEW = MODE == kChunkFew;
  using Shared = std::conditional_t<FEW, FewShared, ChunkShared>;
  static constexpr int NT = chunk_tile(D);
  static constexpr int STREAMS = FEW ? 1 : chunk_streams(D);
  static constexpr int QTILES = PAIRED ? 2 : 1;
  static constexpr int RT = 128 * QTILES;  // rows of a row tile
  static constexpr int SOFT_WARPS = FEW ? 8 : 4 * STREAMS;
  static constexpr int LOAD_WARP = SOFT_WARPS + 8, MMA_WARP = LOAD_WARP + 2;  // two loaders: K, V
  static constexpr int WARPS = MMA_WARP + 1;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr uint32_t Q_BYTES = 128u * D * 2;
  static constexpr uint32_t TILE_BYTES = (uint32_t)NT * D * 2;  // 32 KiB
  static constexpr uint32_t FRONT = FEW ? 3 * kFewBytes : QTILES * Q_BYTES;  // queries; FEW: and two tiles' P
  static constexpr uint32_t FIXED = 1024 + FRONT + 4 * TILE_BYTES;  // the rest of the SM's is staging
  static constexpr uint32_t S_COL = 0, O_COL = 256, L_COL = O_COL + kFewRows,
                            ONE_COL = L_COL + kFewRows;  // columns of TMEM
};

struct ChunkShared {
  uint64_t raw_full[4 * kChunkBars], raw_empty[4 * kChunkBars];  // [piece kind][tile mod kChunkBars]
  uint32_t bad_pages[4 * kChunkBars];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], s_full[2], p_full[2], o_full, pv_done, soft, drained,
      never;
  uint32_t tmem;
  uint32_t gave_up;
  uint32_t nonfinite;
  uint32_t last;  // this CTA joins the unit's partials
  LineStart start;
  Run runs[19];   // one per warp
  uint4 orders[2][32];  // the loaders' copies: source, place, bytes
  int scan[32];
  uint32_t pair_table[256];  // TBQ4: centroids of a byte's two indices
};

struct FewShared : ChunkShared {
  Run next;  // the softmax warps' runs are here and in runs[0] in turn
  alignas(16) float few_part[8][16], few_mneg[8][16], few_fac[8][16], few_sum[kFewRows];
  int few_pos[8][16];
};

// The loader's work for pages whose rows are no whole 16-byte words, or do not divide a subtile: piece
// by piece, 2 bytes at a time.  A page out of range reads as blocks of scale 0 (and zero 0).
template <int D, int RT, bool SEG>
__device__ __noinline__ void load_direct(const ChunkArgs& a, ChunkShared& sh, Run& run, bool more, uint32_t raw_at, int lane,
                                         TileEntries* entries) {
  uint32_t kt = 0, slot = 0, n = 0;
  for (; more; more = warp_run<D, RT, SEG>(a, sh.start, run, 1)) {
    TileOrder order;
    if (SEG) order.start(run.u, run.t0);
    for (int j = run.t0; j < run.t1; ++j, ++kt) {
      CachePos u;
      const int4 entry = SEG ? order.entry(a, run.u, j, chunk_tile(D)) : make_int4(0, 0, 0, 0);
      const TileTokens tt = unit_tile<D, SEG>(a, run.u, j, u, &entry);
      for (int piece = 0; piece < 4; ++piece, ++n) {
        const int which = piece >> 1, a0 = tt.t0 + (piece & 1) * (chunk_tile(D) / 2), row = which ? a.lo.vf.row : a.lo.kf.row;
        if (n >= (uint32_t)a.slots) {  // the slot's last piece must have been read
          const uint32_t last = n - a.slots, bar = (last & 3) * kChunkBars + ((last >> 2) & (kChunkBars - 1));
          if (!__all_sync(0xffffffffu, bar_wait(smem_addr(&sh.raw_empty[bar]), (last >> 2) / kChunkBars & 1, &sh.gave_up))) return;
        }
        for (int i = 0; i < chunk_tile(D) / 2; ++i) {
          const int t = a0 + i;
          if (t >= u.qe || (t & ~31) + 32 <= tt.v0 || (t & ~31) >= tt.v1) continue;
          bool bad = false;
          const uint8_t* src = main_row(a.lo, a.cp, which, u.layer, u.b, u.h, t, &bad);
          const uint32_t to = raw_at + slot * a.slot_bytes + (i >> 5) * a.sub_bytes + (t & 31) * row;
          for (int e = 2 * lane; e < row; e += 64) {
            const uint16_t v = bad ? (uint16_t)0 : *reinterpret_cast<const uint16_t*>(src + e);
            asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(to + e), "h"(v) : "memory");
          }
          if (bad && lane == 0) atomicOr(a.status, KVQ_DEV_PAGE);
        }
        __syncwarp();
        if (lane == 0) {
          const int bar = piece * kChunkBars + (kt & (kChunkBars - 1));
          sh.bad_pages[bar] = 0;
          if (SEG) entries->at[bar] = entry;
          bar_arrive(smem_addr(&sh.raw_full[bar]));
        }
        if (++slot == (uint32_t)a.slots) slot = 0;
      }
    }
  }
}

// A dequantizing warp's half of a piece that the hot path does not cover: one
// call with few arguments (the caller's registers are short), everything else worked out again.
template <int D, int DT, bool SEG>
__device__ __forceinline__ void cold_piece(const ChunkArgs& a, ChunkShared& sh, const Run& run, uint32_t tiles_at,
                                        uint32_t raw_at, int dw, uint32_t kt, uint32_t slot, int j, const TileEntries* entries) {
  constexpr int NT = chunk_tile(D);
  const int piece = dw >> 1, which = dw >> 2, half = piece & 1, part = dw & 1, lane = threadIdx.x & 31;
  const bool per_channel = (which ? a.lo.vf.axis : a.lo.kf.axis) == KVQ_AXIS_CHANNEL;
  CachePos u;
  const TileTokens tt = unit_tile<D, SEG>(a, run.u, j, u, SEG ? &entries->at[piece * kChunkBars + (kt & (kChunkBars - 1))] : nullptr);
  const int a0 = tt.t0 + half * (NT / 2);
  const uint32_t staged = raw_at + slot * a.slot_bytes, bad = sh.bad_pages[piece * kChunkBars + (kt & (kChunkBars - 1))];
  const uint32_t dst = tiles_at + (kt & 1) * (uint32_t)NT * D * 2;
  if (which == 0 && (a.lo.flags & KVQ_K_PRE_ROPE))
    turned_piece<D, DT>(a, u, tt, a0, staged, bad, dst, part * 32 + lane, &sh.nonfinite);
  else
    mixed_piece<D, DT, SEG>(a, u, which, half, part, lane, per_channel, (a.lo.flags & (which ? KVQ_ROTATE_V : KVQ_ROTATE_K)) != 0, a0,
                       tt.v0 & ~31, (tt.v1 + 31) & ~31, staged, bad, dst, tt.t0, which == 1 && kt < 2, sh.pair_table,
                       &sh.nonfinite);
}

// SEG: a dequantizing warp's share of the 16-bit window's tokens of a piece whose packed tokens it has filled in.
template <int D, int DT>
__device__ __forceinline__ void window_tokens(const ChunkArgs& a, ChunkShared& sh, const Run& run, uint32_t tiles_at, int dw,
                                              uint32_t kt, const TileEntries* entries) {
  constexpr int NT = chunk_tile(D);
  const int piece = dw >> 1, which = dw >> 2, half = piece & 1, part = dw & 1, lane = threadIdx.x & 31;
  CachePos u;
  const TileTokens tt = listed_tile<D>(a, run.u, entries->at[piece * kChunkBars + (kt & (kChunkBars - 1))], u);
  const int a0 = tt.t0 + half * (NT / 2), t0 = max(a0, u.qe), t1 = min(a0 + NT / 2, u.T);
  const uint32_t dst = tiles_at + (kt & 1) * (uint32_t)NT * D * 2;
  __syncwarp();  // the zeros of its other lanes are there
  if (a.lo.flags & (which ? KVQ_ROTATE_V : KVQ_ROTATE_K)) {
    rotated_window4<D, DT>(a, u, which, part, dst, tt.t0, a0, t0, t1, lane, &sh.nonfinite);
    return;
  }
  // as in rotated_window4: copied into place, then put right there
  auto each = [&](auto f) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      int toff, row, run32;
      RunPlace<D>::of(false, part, i, lane, &toff, &row, &run32);
      if (a0 + toff < t0 || a0 + toff >= t1) continue;
      row += half * (NT / 2);
      const uint32_t line = RunPlace<D>::line_at(dst, row, run32, NT);
#pragma unroll
      for (int k = 0; k < 4; ++k) f(line + ((((run32 & 1) * 4 + k) ^ (row & 7)) << 4), a0 + toff, 32 * run32 + 8 * k);
    }
  };
  each([&](uint32_t at, int t, int ch) { copy_16(at, resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t) + ch); });
  copies_land();
  if (which == 0 && DT == KVQ_DT_F16) return;  // (keys stand as they are)
  each([&](uint32_t at, int, int) {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = which ? clean<DT>(w[e], which, &sh.nonfinite) : score_pair<DT>(w[e], a.k_pre);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  });
}

// Sum over the block's threads of x, and the exclusive prefix.
template <int THREADS>
__device__ __forceinline__ int block_sum(int x, int* scan, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = y;
  __syncthreads();
  // every warp sums the warps' totals by itself
  const int s = lane < THREADS / 32 ? scan[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, s);
  return __reduce_add_sync(0xffffffffu, lane < warp ? s : 0) + y - x;
}

// Finds this CTA's stretch of the line of tiles and the unit it starts in.
template <int D, int RT, int THREADS, bool SEG>
__device__ __forceinline__ void find_start(const ChunkArgs& a, ChunkShared& sh) {
  const int lane = a.by_warp ? threadIdx.x & 31 : 0, lanes = a.by_warp ? 32 : 1;
  const int group = a.by_warp ? threadIdx.x >> 5 : threadIdx.x, groups = a.by_warp ? THREADS / 32 : THREADS;
  const int owners = SEG ? (plan_fits(a) ? a.n_units : 0) : a.lo.B;
  bool bad = false;
  int line = 0, mine = 0, at = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < owners; b0 += groups) {
    const int b = b0 + group;
    mine = b < owners ? seq_tiles<D, RT, SEG>(a, b, lane, lanes, &bad) : 0;
    int sum;
    at = line + block_sum<THREADS>(mine, sh.scan, &sum);
    line += sum;
  }
  if (SEG && blockIdx.x == 0 && threadIdx.x == 0 && !owners) atomicOr(a.status, KVQ_DEV_SEQ);
  if (!SEG && blockIdx.x == 0) {
    if (threadIdx.x == 0 && __ldg(a.cu_q) != 0) bad = true;
    if (bad) atomicOr(a.status, KVQ_DEV_LENGTH);
  }
  const int all = line * a.n_layers * a.lo.H;
  // at least two tiles a run: joining costs about as much
  const int per = max((all + (int)gridDim.x - 1) / (int)gridDim.x, 2);
  const int begin = (int)min((int64_t)all, (int64_t)per * blockIdx.x), end = min(all - begin, per) + begin;
  if (threadIdx.x == 0) {
    sh.start.begin = begin;
    sh.start.end = end;
    sh.start.per_cta = per;
  }
  if (begin >= end) return;
  const int lh = begin / line, x = begin - lh * line;  // place within one (layer, kv head)
  int base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < owners && base <= x; b0 += groups) {
    const int b = b0 + group;
    if (owners > groups) {  // else the sums of the pass above are still there
      bool ignore = false;
      mine = b < owners ? seq_tiles<D, RT, SEG>(a, b, lane, lanes, &ignore) : 0;
      int sum;
      at = base + block_sum<THREADS>(mine, sh.scan, &sum);
      base += sum;
    } else {
      base = line;
    }
    const int tiles = a.by_warp ? __reduce_add_sync(0xffffffffu, mine) : mine;  // the sequence's, seen from lane 0
    if (lane == 0 && b < owners && x >= at && x < at + tiles) {
      Unit u;
      int left = x - at;
      if constexpr (SEG) {
        u.rt = 0;
      } else {
        (void)valid_seq(a, b, &u.n, &u.T, &u.cu);
#pragma unroll 1
        for (u.rt = 0;; ++u.rt) {
          unit_tiles<D, RT>(a, u);
          if (left < u.nt) break;
          left -= u.nt;
        }
      }
      sh.start.lh = lh;
      sh.start.b = b;
      sh.start.rt = u.rt;
      sh.start.tile = left;
    }
  }
}

// Row r of a row tile: where its query (or output) starts.
__device__ __forceinline__ int64_t query_row(const ChunkArgs& a, const Unit& u, int r) {
  const int row = u.r0 + r, tok = div_g(a, row);
  return (((int64_t)u.layer * a.total_q + u.cu + tok) * a.lo.Hq + u.h * a.lo.g + (row - tok * a.lo.g)) * a.lo.D;
}

// V's values that are not finite were left out of the products: every row
// that sees such a window token gets them afterwards (an infinity stays one
// under any positive weight, a NaN stays NaN).  What a row gets depends on the kinds that it sees in a channel,
// not on how many: the tokens that all rows of a run's unit see are gone through once a warp, and a
// row adds the few that only some see.  (Gone through by every row, one such value in a 16-bit window of 16K tokens
// held a call of 128 rows of 256 channels up for 585 ms.)

// Kinds among window tokens [t0, t1) of this lane's channels (4 lane .. of every 128-chunk): of chunk c, bits
// 12 c + e: +inf in channel e, + 4: -inf, + 8: NaN.
template <int D, int DT>
__device__ __forceinline__ uint32_t sequence_kinds(const ChunkArgs& a, int layer, int b, int h, int T, int t0, int t1) {
  constexpr uint32_t E = DT == KVQ_DT_F16 ? 0x7c00u : 0x7f80u;
  constexpr int N = D / 128, U = 16 / N;  // loads in flight
  const int lane = threadIdx.x & 31;
  uint32_t kinds = 0;
#pragma unroll 1
  for (int t = max(t0, q_end_of(a.lo, T)); t < t1; t += U) {
    uint2 v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint2* p = reinterpret_cast<const uint2*>(
                           resid_row(a.lo, a.cp, 1, layer + a.layer0, b, h, min(t + u, t1 - 1))) + lane;
#pragma unroll
      for (int c = 0; c < N; ++c) v[u][c] = p[32 * c];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < N; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = e & 2 ? v[u][c].y : v[u][c].x, x = e & 1 ? w >> 16 : w & 0xffffu;
          if ((x & E) == E) kinds |= 1u << (12 * c + e + (x & (0x7fffu & ~E) ? 8 : x >> 15 ? 4 : 0));
        }
  }
  return kinds;
}
template <int D, int DT>
__device__ __noinline__ uint32_t window_kinds(const ChunkArgs& a, const Run& run, int t0, int t1) {
  return sequence_kinds<D, DT>(a, run.u.layer, run.u.b, run.u.h, run.u.T, t0, t1);
}
// of sequence b of T tokens (SEG)
template <int D, int DT>
__device__ __noinline__ uint32_t window_kinds_of(const ChunkArgs& a, const Run& run, int b, int T, int t0, int t1) {
  return sequence_kinds<D, DT>(a, run.u.layer, b, run.u.h, T, t0, t1);
}
// Adds them to the unit's output rows r0, r0 + step, .. below r1, which this warp has written.
template <int D, int DT, bool SEG>
__device__ __noinline__ void add_nonfinite(const ChunkArgs& a, const Run& run, int r0, int r1, int step) {
  const Unit& u = run.u;
  const int lo = a.window ? max(0, u.p_hi - a.window + 1) : 0;
  __syncwarp();
  if (r0 >= r1) return;
  // what every row of the unit sees (SEG: every row of one of its sequences)
  uint32_t common = SEG ? 0 : window_kinds<D, DT>(a, run, 0, u.sink) | window_kinds<D, DT>(a, run, lo, u.p_lo + 1);
  int seq = -1, from = 0, T = 0;  // SEG: the sequence of `common`, its first row's position, its length
#pragma unroll 1
  for (int r = r0; r < r1; r += step) {
    const int p = row_pos<SEG>(a, u, r);
    uint32_t kinds;
    if constexpr (SEG) {
      const int b = __ldcg(&a.where[u.cu + div_g(a, u.r0 + r)].y);
      if (b != seq) {
        seq = b;
        from = p;
        T = __ldcg(a.lens + b);
        common = window_kinds_of<D, DT>(a, run, b, T, 0, p + 1);
      }
      kinds = common | window_kinds_of<D, DT>(a, run, b, T, from + 1, p + 1);
    } else {
      const int w = a.window ? max(0, p - a.window + 1) : 0;
      // and the row alone: the sinks that have left its window, what is before and behind the common tokens
      kinds = common | window_kinds<D, DT>(a, run, u.sink, min(a.sinks, w)) |
              window_kinds<D, DT>(a, run, w, min(lo, p + 1)) |
              window_kinds<D, DT>(a, run, max(u.p_lo + 1, w), p + 1);
    }
    uint16_t* out = a.out + query_row(a, u, r) + 4 * (threadIdx.x & 31);
#pragma unroll 1
    for (int e = 0; e < D / 32; ++e) {  // channel e & 3 of chunk e >> 2
      const uint32_t k = kinds >> (12 * (e >> 2) + (e & 3));
      if (!(k & 0x111u)) continue;
      uint16_t* o = out + 128 * (e >> 2) + (e & 3);
      float x = in_to_f32(*o, DT);
      if (k & 1u) x += INFINITY;
      if (k & 0x10u) x -= INFINITY;
      if (k & 0x100u) x = NAN;
      *o = (uint16_t)pack16<DT>(x, 0.f);
    }
  }
  __syncwarp();
}

// All softmax warps meet (boundedly, like every wait): false once a warp has given up.
__device__ __forceinline__ bool soft_sync(uint32_t bar, uint32_t& phase, volatile uint32_t* gave_up) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(bar);
  const bool ok = __all_sync(0xffffffffu, bar_wait(bar, phase & 1, gave_up));
  ++phase;
  return ok;
}

// One output row, four channels of a 128-chunk a lane: acc / L, out of the rotated domain.  (s1, s2): the lane's signs.
template <int D, int DT>
__device__ __forceinline__ void write_row(const ChunkArgs& a, const Run& run, int r, float (&acc)[D / 128][4], float L, uint32_t s1,
                                          uint32_t s2) {
  const int lane = threadIdx.x & 31;
  uint16_t* dst = a.out + query_row(a, run.u, r);
  const float inv = 1.f / L;
#pragma unroll
  for (int c = 0; c < D / 128; ++c) {
    float v[4] = {acc[c][0] * inv, acc[c][1] * inv, acc[c][2] * inv, acc[c][3] * inv};
    if (a.lo.flags & KVQ_ROTATE_V) rotate_lanes(v, s2, s1);
    *reinterpret_cast<uint2*>(dst + 128 * c + 4 * lane) = make_uint2(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]));
  }
}

// The softmax warps of FEW meet, N of them: whether p holds for any thread.  A hardware barrier, so all of them come
// by it equally often, also when one has given up waiting for another role.
template <int N>
__device__ __forceinline__ bool few_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "n"(32 * N)
      : "memory");
  return r != 0;
}

// Joins of planned units (SEG): warp w of `warps` takes rows w, w + warps, .. below `rows`, RW of them side by side, so that their loads
// are in flight together.  (Row after row, the joins of units of 32 rows in 3 parts took 15 us, of 256 rows in 10 parts 45 us.)
// part(i, r): row r of part i.
template <int D, int RW, class Part, class Write>
__device__ __forceinline__ void join_rows(int parts, int rows, int warps, const Part& part, const Write& write) {
  constexpr int N = D / 128, U = RW * N >= 4 ? 1 : 4 / (RW * N);  // parts in flight of each row
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r0 = threadIdx.x >> 5; r0 < rows; r0 += warps * RW) {
    float M[RW], L[RW], acc[RW][N][4];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      M[k] = -INFINITY;
      L[k] = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) acc[k][c][0] = acc[k][c][1] = acc[k][c][2] = acc[k][c][3] = 0.f;
    }
    auto row = [&](int k) { return min(r0 + k * warps, rows - 1); };
#pragma unroll 1
    for (int i = lane; i - lane < parts; i += 32)
#pragma unroll
      for (int k = 0; k < RW; ++k)
        if (i < parts) M[k] = fmaxf(M[k], __ldcg(part(i, row(k)) + D));
#pragma unroll
    for (int k = 0; k < RW; ++k)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M[k] = fmaxf(M[k], __shfl_xor_sync(0xffffffffu, M[k], o));
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += 32) {
      float w[RW];
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(min(i0 + lane, parts - 1), row(k)) + D));
        // a part that saw none of the row's tokens has m = -inf, or the lowest reference, and l = 0
        const bool none = i0 + lane >= parts || ml.y == 0.f;
        w[k] = none ? 0.f : ex2(ml.x - M[k]);
        L[k] += none ? 0.f : w[k] * ml.y;
      }
#pragma unroll 1
      for (int i = 0; i < min(32, parts - i0); i += U) {
        float4 v[RW][U][N];
#pragma unroll
        for (int k = 0; k < RW; ++k)
#pragma unroll
          for (int q = 0; q < U; ++q)
#pragma unroll
            for (int c = 0; c < N; ++c)
              v[k][q][c] = __ldcg(reinterpret_cast<const float4*>(part(min(i0 + i + q, parts - 1), row(k))) + 32 * c + lane);
#pragma unroll
        for (int k = 0; k < RW; ++k)
#pragma unroll
          for (int q = 0; q < U; ++q) {
            const float wk = __shfl_sync(0xffffffffu, w[k], (i + q) & 31);
            if (i0 + i + q < parts && wk != 0.f) {
#pragma unroll
              for (int c = 0; c < N; ++c) {
                acc[k][c][0] = fmaf(wk, v[k][q][c].x, acc[k][c][0]);
                acc[k][c][1] = fmaf(wk, v[k][q][c].y, acc[k][c][1]);
                acc[k][c][2] = fmaf(wk, v[k][q][c].z, acc[k][c][2]);
                acc[k][c][3] = fmaf(wk, v[k][q][c].w, acc[k][c][3]);
              }
            }
          }
      }
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L[k] += __shfl_xor_sync(0xffffffffu, L[k], o);
      if (r0 + k * warps < rows) write(r0 + k * warps, acc[k], L[k]);
    }
  }
}

// Joins the partial rows of one unit and writes its output rows; all softmax
// threads.  scratch: 8 rows of D + 4 floats in shared memory.  False once a warp has given up.
template <int D, int DT, int MODE, bool SEG>
__device__ __forceinline__ bool join_unit(const ChunkArgs& a, const Run& run, const LineStart& line, bool cut, bool fix,
                                          float* scratch, uint32_t soft, uint32_t& syncs, uint32_t* gave_up) {
  using C = ChunkShape<D, MODE>;
  constexpr bool PAIRED = C::PAIRED;
  constexpr int N = D / 128;
  constexpr int PR = chunk_part_row(D), SLOT = chunk_slot_rows(D) * PR;
  const Unit& u = run.u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit_pos = run.pos - run.t0;
  const int c0 = cut ? unit_pos / line.per_cta : blockIdx.x;
  const int c1 = cut ? (unit_pos + u.nt - 1) / line.per_cta : blockIdx.x;
  const int slot0 = !cut ? 2 : unit_pos - unit_cost<SEG>(a) <= c0 * line.per_cta ? 0 : 1;  // of the first CTA; the others' is 0
  constexpr bool ONE = PAIRED || C::FEW;
  constexpr int copies = ONE ? 1 : C::STREAMS, copies_log = copies - 1;  // partial rows of one query row in one slot
  const int parts = (c1 - c0 + 1) * copies;
  auto part = [&](int i, int r) {
    const int c = i >> copies_log, row = ((i & (copies - 1)) << 7) + r;  // a stream's 128 rows after the other's
    return a.partials + ((int64_t)(c0 + c) * kChunkSlots + (c ? 0 : slot0)) * SLOT + row * PR;
  };
  const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
  auto write = [&](int r, float (&acc)[N][4], float L) { write_row<D, DT>(a, run, r, acc, L, s1, s2); };
  if (PAIRED && parts <= 4) {
    // Many rows of few parts: a lane works out the weights of one row of the
    // warp's 32; then row by row, the next row's loads in flight.
    const int r0 = 32 * warp, mine = min(r0 + lane, u.rows - 1);
    float w[4], M = -INFINITY, L = 0.f;
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i < parts) ml[i] = __ldcg(reinterpret_cast<const float2*>(part(i, mine) + D));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // a part that saw none of the row's tokens has m = -inf and l = 0
      const bool none = ml[i].x == -INFINITY && ml[i].y == 0.f;
      w[i] = none ? 0.f : ex2(ml[i].x - M);
      L += none ? 0.f : w[i] * ml[i].y;
    }
    float4 next[4][N];
    auto load = [&](int r) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (i < parts) next[i][c] = __ldcg(reinterpret_cast<const float4*>(part(i, min(r, u.rows - 1))) + 32 * c + lane);
    };
    load(r0);
#pragma unroll 1
    for (int r = r0; r < min(r0 + 32, u.rows); ++r) {
      float acc[N][4];
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float wk = __shfl_sync(0xffffffffu, w[i], r - r0);
        if (i < parts && wk != 0.f) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            acc[c][0] = fmaf(wk, next[i][c].x, acc[c][0]);
            acc[c][1] = fmaf(wk, next[i][c].y, acc[c][1]);
            acc[c][2] = fmaf(wk, next[i][c].z, acc[c][2]);
            acc[c][3] = fmaf(wk, next[i][c].w, acc[c][3]);
          }
        }
      }
      load(r + 1);
      write(r, acc, __shfl_sync(0xffffffffu, L, r - r0));
    }
    if (fix) add_nonfinite<D, DT, SEG>(a, run, r0, min(r0 + 32, u.rows), 1);
    return true;
  }
  if constexpr (SEG) {
    if (u.rows > 4) {
      if (u.rows <= C::SOFT_WARPS)
        join_rows<D, 1>(parts, u.rows, C::SOFT_WARPS, part, write);
      else if (u.rows <= 2 * C::SOFT_WARPS)
        join_rows<D, 2>(parts, u.rows, C::SOFT_WARPS, part, write);
      else
        join_rows<D, 4>(parts, u.rows, C::SOFT_WARPS, part, write);
      if (fix) add_nonfinite<D, DT, SEG>(a, run, warp, u.rows, C::SOFT_WARPS);
      return true;
    }
  }
  // Few rows: `wpr` warps share a row's parts and join their sums in shared memory.
  const int wpr = u.rows >= C::SOFT_WARPS ? 1 : u.rows > C::SOFT_WARPS / 2 ? 1 : u.rows > C::SOFT_WARPS / 4 ? 2 : u.rows > 1 || C::SOFT_WARPS == 4 ? 4 : 8;
  const int sub = warp & (wpr - 1), len = (parts + wpr - 1) / wpr, i0 = sub * len, i1 = min(parts, i0 + len);
  const int per = C::SOFT_WARPS / wpr;  // rows at a time
#pragma unroll 1
  for (int rr = warp / wpr; rr < (u.rows + per - 1) / per * per; rr += per) {
    const int r = min(rr, u.rows - 1);
    float M = -INFINITY, L = 0.f, acc[N][4];
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
#pragma unroll 4
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(part(i, r) + D));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
      const float* p = part(min(i + lane, parts - 1), r);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + D));
      // a part that saw none of the row's tokens has m = -inf and l = 0
      const bool none = i + lane >= i1 || (ml.x == -INFINITY && ml.y == 0.f);
      const float w = none ? 0.f : ex2(ml.x - M);
      L += none ? 0.f : w * ml.y;
      const uint32_t off = (uint32_t)((p - a.partials) >> 2);  // in 16-byte words
      const int k1 = min(32, i1 - i);
      constexpr int U = 8 / N;  // loads in flight
#pragma unroll 1
      for (int k = 0; k < k1; k += U) {
        float4 v[U][N];
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const float4* o4 = reinterpret_cast<const float4*>(a.partials) + __shfl_sync(0xffffffffu, off, min(k + q, 31)) + lane;
#pragma unroll
          for (int c = 0; c < N; ++c) v[q][c] = __ldcg(o4 + 32 * c);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const float wk = __shfl_sync(0xffffffffu, w, min(k + q, 31));
          if (k + q < k1 && wk != 0.f) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
              acc[c][0] = fmaf(wk, v[q][c].x, acc[c][0]);
              acc[c][1] = fmaf(wk, v[q][c].y, acc[c][1]);
              acc[c][2] = fmaf(wk, v[q][c].z, acc[c][2]);
              acc[c][3] = fmaf(wk, v[q][c].w, acc[c][3]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (wpr > 1) {
      float* mine = scratch + warp * (D + 4);
#pragma unroll
      for (int c = 0; c < N; ++c)
        *reinterpret_cast<float4*>(mine + 128 * c + 4 * lane) = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
      if (lane == 0) mine[D] = L;
      if constexpr (C::FEW)
        (void)few_any<8>(3, false);
      else if (!soft_sync(soft, syncs, gave_up))
        return false;
      if (sub) continue;  // one turn: fewer rows than warps
#pragma unroll 1
      for (int k = 1; k < wpr; ++k) {
        const float* o = mine + k * (D + 4);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(o + 128 * c + 4 * lane);
          acc[c][0] += v.x;
          acc[c][1] += v.y;
          acc[c][2] += v.z;
          acc[c][3] += v.w;
        }
        L += o[D];
      }
    }
    if (rr < u.rows) write(r, acc, L);
  }
  if (fix && sub == 0) add_nonfinite<D, DT, SEG>(a, run, warp / wpr, u.rows, per);
  return true;
}

// The butterflies of the 128-point transform on TMEM columns [col, col + 128)
// of this lane, in place, after the signs of d2 and `factor`: strides below 16 within 16
// columns, the others between two sets of 16.  Short loops: this runs once per row tile, and code
// that runs once costs its fetch.
__device__ __forceinline__ void unrotate_columns(const ChunkArgs& a, uint32_t col, float factor) {
  const float f = factor * hadamard_scale();
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    uint32_t r[16];
    tmem_ld16(col + c, r);
    const uint32_t signs = a.lo.d2[c >> 5] >> (c & 16);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f) ^ ((signs << (31 - i)) & 0x80000000u);
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(i & h)) {
          const float u = __uint_as_float(r[i]), v = __uint_as_float(r[i + h]);
          r[i] = __float_as_uint(u + v);
          r[i + h] = __float_as_uint(u - v);
        }
    tmem_st16(col + c, r);
  }
#pragma unroll 1
  for (int h = 16; h < 128; h <<= 1) {
    tmem_wait_st();
#pragma unroll 1
    for (int k = 0; k < 64; k += 16) {
      const int c = (k & ~(h - 1)) * 2 + (k & (h - 1));  // the k-th column set whose bit h is clear
      uint32_t p[16], q[16];
      tmem_ld16(col + c, p);
      tmem_ld16(col + c + h, q);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float u = __uint_as_float(p[i]), v = __uint_as_float(q[i]);
        p[i] = __float_as_uint(u + v);
        q[i] = __float_as_uint(u - v);
      }
      tmem_st16(col + c, p);
      tmem_st16(col + c + h, q);
    }
  }
  tmem_wait_st();
}

// ---- softmax of one tile, one row per thread ----------------------------------------

struct RowSeen {
  int pos, win_lo, sinks;  // visible tokens: [win_lo, pos] and [0, sinks)
};
template <bool MASKED>
__device__ __forceinline__ void hide(uint32_t (&x)[32], int t, const RowSeen& see) {
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (t + i > see.pos || (t + i < see.win_lo && t + i >= see.sinks)) x[i] = 0xff800000u;
  }
}
// largest score of the row's columns of S at s_col (tile's first token t0)
template <int NT, bool MASKED>
__device__ __forceinline__ float tile_max(uint32_t s_col, int t0, const RowSeen& see) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < NT; c += 32) {
    uint32_t x[32];
    tmem_ld32(s_col + c, x);
    tmem_wait_ld();
    hide<MASKED>(x, t0 + c, see);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      m0 = fmaxf(m0, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
      m1 = fmaxf(m1, fmaxf(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])));
    }
  }
  return fmaxf(m0, m1);
}
// P = 2^(S sc + mneg) over S, in the input dtype; the sum of P
template <int DT, int NT, bool MASKED>
__device__ __forceinline__ float tile_exp(uint32_t s_col, int t0, const RowSeen& see, float sc, float mneg) {
  const uint64_t sc2 = pk2(sc, sc), mneg2 = pk2(mneg, mneg);  // packed pairs: half the instructions
  uint64_t la = 0, lb = 0;
#pragma unroll 1
  for (int c = 0; c < NT; c += 32) {
    uint32_t x[32];
    tmem_ld32(s_col + c, x);
    tmem_wait_ld();
    hide<MASKED>(x, t0 + c, see);
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float e0, e1;
      upk2(fma2(pk2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc2, mneg2), e0, e1);
      e0 = ex2(e0);
      e1 = ex2(e1);
      if (i & 1)
        la = add2(la, pk2(e0, e1));
      else
        lb = add2(lb, pk2(e0, e1));
      p[i] = pack16<DT>(e0, e1);
    }
    tmem_st16(s_col + c / 2, p);
  }
  float l0, l1;
  upk2(add2(la, lb), l0, l1);
  return l0 + l1;
}
template <int D>
__device__ __forceinline__ void rescale_columns(uint32_t o_col, float f) {
  uint32_t x[32];
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    tmem_ld32(o_col + c, x);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
    tmem_st32(o_col + c, x);
  }
  tmem_wait_st();
}

// ---- few rows ------------------------------------------------------------------------
// At most 32 query rows a sequence, D = 128: the products are turned over, S^T = K Q^T and O^T = V^T P^T, so that
// the rows are columns (16 or 32 of them) and not lanes: both products cost a quarter or an eighth, and the
// accumulator, its rescaling and its output shrink with them.  A thread holds one token of a tile, then
// one channel of the output; P goes through shared memory.  Row sums come from a third product, ones times
// P^T, so that no thread keeps 16 of them (32 registers of sums spilled: 8-token drafts of 16
// sequences took 414 us).  The rows' reference maxima are common to a group's four warps.
// Against rows as lanes: one token over one long window 34 -> 29 us, single tokens of 64 sequences 265 -> 228 us,
// drafts of 16 sequences 291 -> 274 us; 16 columns instead of 32 for the single tokens 238 -> 229 us.  (More than 32 rows are not two
// groups of 16 a thread any more, and there the lanes are full enough.)  Bound now by the dequantizing warps' issue slots and the shared memory's bandwidth (a tile's
// values are written once and read by the products once: 128 KiB of shared-memory traffic for 17 KiB of cache).

// A run's queries into shared memory (row r of 64 channels a block of kFewBytes / 2), a warp a row.
template <int DT>
__device__ __forceinline__ void few_queries(const ChunkArgs& a, const Unit& u, uint32_t q_at, int w, int lane) {
  const bool turn = a.lo.flags & KVQ_ROTATE_K;
  const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
  const int rows = u.rows, ch = 4 * lane;
  const uint32_t col = q_at + (uint32_t)(ch >> 6) * (kFewBytes / 2) + (ch & 4) * 2;
  uint2 x = make_uint2(0, 0);
  if (w < rows) x = __ldcg(reinterpret_cast<const uint2*>(a.q + query_row(a, u, w)) + lane);
#pragma unroll 1
  for (int r = w; r < rows; r += 8) {
    uint2 next = x;
    if (r + 8 < rows) next = __ldcg(reinterpret_cast<const uint2*>(a.q + query_row(a, u, r + 8)) + lane);
    if (turn) {
      float v[4] = {in_to_f32((uint16_t)x.x, DT), in_to_f32((uint16_t)(x.x >> 16), DT), in_to_f32((uint16_t)x.y, DT),
                    in_to_f32((uint16_t)(x.y >> 16), DT)};
      rotate_lanes(v, s1, s2, a.q_pre);
      x = query_pack<DT>(v);
    } else {
      x = make_uint2(score_pair<DT>(x.x, 1.f), score_pair<DT>(x.y, 1.f));
    }
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(col + swz(r, (ch & 63) >> 3)), "r"(x.x), "r"(x.y) : "memory");
    x = next;
  }
  proxy_fence();
  __syncwarp();
}

// Over the warp's lanes, row by row: lane r and lane r + 16 get row r's maximum.
__device__ __forceinline__ float max_across(float (&x)[16], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i], got = __shfl_xor_sync(0xffffffffu, give, o);
      x[i] = fmaxf(keep, got);
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, x[0], 16);
  return fmaxf(x[0], got);
}

// The softmax warps' work of FEW: two groups of four warps, 16 rows each.
template <int DT, bool SEG>
__device__ __forceinline__ void few_rows(const ChunkArgs& a, FewShared& sh, bool more, uint8_t* smem, uint32_t tmem,
                                         const TileEntries* entries) {
  constexpr int D = 128, NT = 128, PR = chunk_part_row(D);
  using C = ChunkShape<D, kChunkFew>;
  const int lane = threadIdx.x & 31;
  int w = threadIdx.x >> 5;
  asm volatile("" : "+r"(w));
  const int quad = w & 3, row0 = (w >> 2) * 16;  // rows [row0, row0 + 16)
  const int my = 32 * quad + lane;               // token of a tile; channel of the output
  const uint32_t q_at = smem_addr(smem), lane_base = tmem + ((uint32_t)(32 * quad) << 16) + row0, o_col = lane_base + C::O_COL;
  const float sc = a.score_scale;
  uint32_t* const gave_up = &sh.gave_up;
  float* const mneg = sh.few_mneg[w];  // minus the references
  float* const fac = sh.few_fac[w];
  int* const pos = sh.few_pos[w];
  float* const stage = reinterpret_cast<float*>(smem + kFewBytes);  // outputs [row][channel], where P was
  // this thread's token in P: row r's 64 tokens are 128 bytes, their 16-byte parts swizzled by r mod 8
  const uint32_t p_at = q_at + kFewBytes + (uint32_t)(my >> 6) * (kFewBytes / 2) + row0 * 128 + (my & 63) * 2;
  uint32_t ns0 = 0, ns1 = 0, runs = 0, steps = 0, syncs = 0;
  asm volatile("" : "+r"(ns0), "+r"(ns1), "+r"(runs), "+r"(steps));
  if (w < 4) {  // the left operand of the sums: 16 ones a lane
    uint32_t one[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) one[i] = DT == KVQ_DT_F16 ? 0x3c003c00u : 0x3f803f80u;
    tmem_st16(lane_base + C::ONE_COL, one);
    tmem_wait_st();
  }
  // the warps follow one run: their barriers must match whatever the lengths in memory do meanwhile
  Run *now = &sh.runs[0], *after = &sh.next;
  more = few_any<8>(3, w == 0 && more);
  if (more) {
    few_queries<DT>(a, now->u, q_at, w, lane);
    if (lane == 0) bar_arrive(smem_addr(&sh.q_full[0]));
  }
  while (more) {
    const Run& run = *now;
    const int rows = run.u.rows - row0, t0 = run.t0, t1 = run.t1;  // the group's: 16 or fewer, none
    bool ok = true;
    // row row0 + lane's reference; and minus all rows'.  +inf past the rows: it never moves.  The lowest to begin with is
    // finite, so that a score of -inf alone in a run counts nothing instead of making a NaN.
    constexpr float LOWEST = -3e38f;
    float m = lane < rows ? LOWEST : INFINITY;
    if (row0 < a.cols) {
      const int st = run.u.st, skip = run.u.lo_tile - st, p_lo = run.u.p_lo, p_hi = run.u.p_hi;
      float n[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) n[r] = r < rows ? -LOWEST : -INFINITY;
      __syncwarp();
      if (lane < 16) pos[lane] = row_pos<SEG>(a, run.u, min(row0 + lane, run.u.rows - 1));
      __syncwarp();
#pragma unroll 1
      for (int j = t0; j < t1; ++j, ++steps) {
        const int b = (j - t0) & 1;
        int tile0 = (j < st ? j : j + skip) * NT;
        const uint32_t s_col = lane_base + C::S_COL + b * kFewRows;
        const bool here = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.s_full[b]), (b ? ns1 : ns0) & 1, gave_up));
        ns0 += b ^ 1;
        ns1 += b;
        [[maybe_unused]] int r_lo = 0, r_hi = 0;  // SEG: rows of the group that see an own tile
        bool masked;
        if constexpr (SEG) {
          const int4 x = entries->at[steps & (kChunkBars - 1)];
          masked = false;  // of the prefix every row sees every token
          if (x.w >= 0) {
            tile0 = x.y;
            r_lo = (x.w & 0xffff) - row0;
            r_hi = (x.w >> 16) - row0;
            masked = tile0 + NT - 1 > p_lo || r_lo > 0 || r_hi < rows;
          }
        } else {
          masked = tile0 + NT - 1 > p_lo || (a.window && tile0 <= p_hi - a.window && tile0 + NT > a.sinks);
        }
        // -inf where this thread's token is out of a row's view
        auto hide = [&](float (&x)[16]) {
          const int t = tile0 + my, window = a.window ? a.window : 1 << 30;
          const bool sink = t < a.sinks;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int p = pos[i];
            if constexpr (SEG) {
              if (t > p || i < r_lo || i >= r_hi) x[i] = -INFINITY;
            } else {
              if (t > p || (t <= p - window && !sink)) x[i] = -INFINITY;
            }
          }
        };
        // log2 P
        auto powers = [&](float (&x)[16]) {
          uint32_t s16[16];
          tmem_ld16(s_col, s16);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(__uint_as_float(s16[i]), sc, n[i]);
          if (masked) hide(x);
        };
        float x[16], most = -INFINITY;
        if (here) {
          tc_fence_after();
          powers(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) most = fmaxf(most, x[i]);
        }
        // The references follow when some score passes its row's by 2^8 (P stays below 2^8): then the group's all go to their rows' maxima so far and the accumulator is
        // rescaled.  References are whole numbers: factors are powers of two, and P rounds alike whatever the reference.
        if (few_any<4>(1 + (w >> 2), most > 8.f || !here)) {
          if (here) {
            uint32_t s16[16];
            tmem_ld16(s_col, s16);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(s16[i]);
            if (masked) hide(x);
            const float top = max_across(x, lane) * sc;
            if (lane < 16) sh.few_part[w][lane] = top;
          }
          // the products of the step before must have left the accumulator
          const bool left = here && (j == t0 || __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.pv_done), (steps - 1) & 1, gave_up)));
          if (few_any<4>(1 + (w >> 2), !left)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float top = m;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, floorf(sh.few_part[(w & 4) + k][lane & 15]));
          if (lane < 16) {
            fac[lane] = top == m ? 1.f : ex2(m - top);
            mneg[lane] = -top;
          }
          m = top;
          __syncwarp();
          if (j > t0) {
#pragma unroll 1
            for (int c = 0; c < 2 * kFewRows; c += kFewRows) {  // outputs, then sums
              uint32_t o[16];
              tmem_ld16(o_col + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac[i]);
              tmem_st16(o_col + c, o);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(mneg + i);
            n[i] = v.x;
            n[i + 1] = v.y;
            n[i + 2] = v.z;
            n[i + 3] = v.w;
          }
          powers(x);
          __syncwarp();
        }
        // P, eight rows at a time (that of the columns behind the last rows is what it was)
        const uint32_t p_row = p_at + b * kFewBytes;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (8 * q < rows) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = pack16<DT>(ex2(x[q * 8 + 2 * i]), ex2(x[q * 8 + 2 * i + 1]));
#pragma unroll
            for (int i = 0; i < 4; ++i)  // rows 8 q + 2 i and the next: 2 i and 2 i + 1 are their swizzles
              asm volatile("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n st.shared.b16 [%0], lo;\n st.shared.b16 [%1], hi;\n}\n" ::"r"(
                               (p_row ^ (32 * i)) + (8 * q + 2 * i) * 128),
                           "r"((p_row ^ (32 * i + 16)) + (8 * q + 2 * i + 1) * 128), "r"(p[i]));
          }
        proxy_fence();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.p_full[b]));
      }
    }
    // ---- the run's outputs ---------------------------------------------------------------
    const bool here = ok && __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.o_full), runs & 1, gave_up));
    if (few_any<8>(3, !here)) break;
    ++runs;
    tc_fence_after();
    // the next run's queries first: its scores are worked out meanwhile
    static_assert(sizeof(Run) % 4 == 0 && sizeof(Run) <= 128, "a word a lane");
    if (w == 0) {
      if (lane < (int)sizeof(Run) / 4) reinterpret_cast<int*>(after)[lane] = reinterpret_cast<const int*>(now)[lane];
      more = warp_run<D, 128, SEG>(a, sh.start, *after, 1);
    }
    more = few_any<8>(3, w == 0 && more);
    if (more) {
      few_queries<DT>(a, after->u, q_at, w, lane);
      if (lane == 0) bar_arrive(smem_addr(&sh.q_full[0]));
    }
    uint32_t x[16];
    float L = 0.f;  // row row0 + lane's sum, from TMEM lane 0
    if (quad == 0 && rows > 0) {
      tmem_ld16(lane_base + C::L_COL, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = __uint_as_float(__shfl_sync(0xffffffffu, x[i], 0));
        if (lane == i) L = v;
      }
    }
    if (rows > 0) {
      tmem_ld16(o_col, x);
      tmem_wait_ld();
    }
    if (t0 == 0 && t1 == run.u.nt) {
      if (rows > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) stage[(row0 + i) * D + my] = __uint_as_float(x[i]);
        if (quad == 0 && lane < 16) sh.few_sum[row0 + lane] = L;
      }
      (void)few_any<8>(3, false);
      const bool fix = *(volatile uint32_t*)&sh.nonfinite != 0;
      const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
#pragma unroll 1
      for (int r = w; r < run.u.rows; r += 8) {
        const float4 v = *reinterpret_cast<const float4*>(stage + r * D + 4 * lane);
        float acc[1][4] = {{v.x, v.y, v.z, v.w}};
        write_row<D, DT>(a, run, r, acc, sh.few_sum[r], s1, s2);
      }
      if (fix) add_nonfinite<D, DT, SEG>(a, run, w, run.u.rows, 8);
    } else {
      float* part = a.partials + ((int64_t)blockIdx.x * kChunkSlots + (run.first ? 0 : 1)) * chunk_slot_rows(D) * PR + row0 * PR;
      if (quad == 0 && lane < min(rows, 16)) *reinterpret_cast<float2*>(part + lane * PR + D) = make_float2(m, L);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < rows) part[i * PR + my] = __uint_as_float(x[i]);
      __threadfence();
      (void)few_any<8>(3, false);
      const int unit_pos = run.pos - t0, c0 = unit_pos / sh.start.per_cta;  // the unit's ticket: as below
      const int tick = c0 * kChunkTickets + (unit_pos - unit_cost<SEG>(a) <= c0 * sh.start.per_cta ? 0 : 1);
      bool last = false;
      if (w == 0 && lane == 0) {
        if (*(volatile uint32_t*)&sh.nonfinite) atomicOr(a.nonfinite + tick, 1u);
        __threadfence();
        last = atomicAdd(a.tickets + tick, 1u) == (uint32_t)((unit_pos + run.u.nt - 1) / sh.start.per_cta - c0);
      }
      if (few_any<8>(3, last)) {
        __threadfence();
        const bool fix = __ldcg(a.nonfinite + tick) != 0;
        (void)join_unit<D, DT, kChunkFew, SEG>(a, run, sh.start, true, fix, stage, 0, syncs, gave_up);
        (void)few_any<8>(3, false);
        if (w == 0 && lane == 0) {
          a.tickets[tick] = 0;
          a.nonfinite[tick] = 0;
        }
      }
    }
    // (the next P over the staged outputs: behind the next run's first barriers)
    (void)few_any<8>(3, false);
    Run* const t = now;
    now = after;
    after = t;
  }
}

template <int D, int DT, int MODE, bool SEG>
__global__ void __launch_bounds__(ChunkShape<D, MODE>::THREADS, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkArgs a) {
  using C = ChunkShape<D, MODE>;
  constexpr bool PAIRED = C::PAIRED, FEW = C::FEW;
  constexpr int NT = C::NT, RT = C::RT;
  extern __shared__ uint8_t raw_smem[];
  __shared__ typename C::Shared sh;
  __shared__ std::conditional_t<SEG, TileEntries, uint32_t> entry_slots;
  TileEntries* const entries = SEG ? reinterpret_cast<TileEntries*>(&entry_slots) : nullptr;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = smem_addr(smem), k_at = q_at + C::FRONT, v_at = k_at + 2 * C::TILE_BYTES;
  const uint32_t raw_at = v_at + 2 * C::TILE_BYTES;

  // set-up that needs nothing of the stream's earlier work
  if (warp == 1) {
    bar_init(smem_addr(&sh.raw_full[lane]), 1);
    bar_init(smem_addr(&sh.raw_empty[lane]), 2);  // a piece's two warps
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  static_assert(4 * kChunkBars == 32, "one barrier a lane");
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sh.k_full[i]), 4);
      bar_init(smem_addr(&sh.v_full[i]), 4);
      bar_init(smem_addr(&sh.k_empty[i]), 1);
      bar_init(smem_addr(&sh.v_empty[i]), 1);
      bar_init(smem_addr(&sh.q_full[i]), FEW ? 8 : 4);
      bar_init(smem_addr(&sh.s_full[i]), 1);
      bar_init(smem_addr(&sh.p_full[i]), FEW ? a.cols / 4 : 4);
    }
    bar_init(smem_addr(&sh.o_full), 1);
    bar_init(smem_addr(&sh.pv_done), 1);
    bar_init(smem_addr(&sh.soft), C::SOFT_WARPS);
    bar_init(smem_addr(&sh.drained), 1);
    bar_init(smem_addr(&sh.never), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    sh.gave_up = 0;
    sh.nonfinite = 0;
  }
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  // query rows that no unit writes are zeros
#pragma unroll 1
  for (uint32_t e = tid * 16; e < C::FRONT; e += C::THREADS * 16)
    *reinterpret_cast<uint4*>(smem + e) = make_uint4(0, 0, 0, 0);
  if (a.lo.flags & (KVQ_TBQ4_K | KVQ_TBQ4_V))
    for (int i = tid; i < 256; i += C::THREADS) {
      const __half2 p = __floats2half2_rn(a.lo.cb[i & 15], a.lo.cb[i >> 4]);
      sh.pair_table[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  grid_launch_dependents();
  grid_dependency_wait();
  find_start<D, RT, C::THREADS, SEG>(a, sh);
  proxy_fence();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sh.tmem);
  Run& run = sh.runs[warp];
  uint32_t* const gave_up = &sh.gave_up;
  const bool k_chan = a.lo.kf.axis == KVQ_AXIS_CHANNEL, v_chan = a.lo.vf.axis == KVQ_AXIS_CHANNEL;
  bool more = warp_run<D, RT, SEG>(a, sh.start, run, 0);
  // Test mode (kvq_test_force_stall): in every second CTA one of the four roles first waits on a barrier that
  // nothing completes, gives up and leaves; the CTAs between finish their runs.
  if (a.stall_polls && (blockIdx.x & 1) && more) {
    const int role = warp == C::MMA_WARP ? 0 : warp >= C::LOAD_WARP ? 1 : warp >= C::SOFT_WARPS ? 2 : 3;
    if (role == (int)(blockIdx.x >> 1 & 3)) {
#pragma unroll 1
      for (int i = 0; i < a.stall_polls && !bar_test(smem_addr(&sh.never), 0); ++i) {
      }
      *(volatile uint32_t*)gave_up = 1;
      __syncwarp();
      more = false;
    }
  }

  if (warp == C::MMA_WARP) {
    // ---- products: one thread ----------------------------------------------------
    constexpr uint32_t F = DT == KVQ_DT_F16 ? 0 : 1;
    constexpr uint32_t half = (1u << 4) | ((128u >> 4) << 24), base = half | (F << 7) | (F << 10);
    // FEW: keys and values are the left operands, the rows the columns of both products
    const uint32_t qk_desc = half | ((uint32_t)k_chan << (FEW ? 15 : 16)) | ((uint32_t)((FEW ? a.cols : NT) >> 3) << 17);
    const uint32_t pv_desc = base | ((uint32_t)!v_chan << (FEW ? 15 : 16)) | ((uint32_t)((FEW ? a.cols : D) >> 3) << 17);
    const uint64_t p_desc = operand_desc(q_at + kFewBytes, 0, 1024);
    const uint32_t sum_desc = base | ((uint32_t)(a.cols >> 3) << 17);
    const uint64_t q_desc = operand_desc(q_at, 0, 1024), k_desc = operand_desc(k_at, k_chan ? D * 128 : 0, 1024),
                   v_desc = operand_desc(v_at, v_chan ? 0 : NT * 128, 1024);
    uint32_t kt = 0;             // tiles of this CTA so far
    uint32_t np0 = 0, np1 = 0;   // steps of each S buffer so far
    uint32_t runs = 0;
    bool ok = true;
    for (; more && ok; more = warp_run<D, RT, SEG>(a, sh.start, run, 1), ++runs) {
      const int tiles = uniform(run.t1 - run.t0), steps = PAIRED ? 2 * tiles : tiles;
      {
#pragma unroll 1
        for (int i = 0; i < 2 * steps + 2 && ok; ++i) {
          // order: scores of steps 0 and 1, then outputs of step s and scores of s + 2 in turn
          const int s = i < 2 ? i : (i & 1) ? (i - 3) / 2 + 2 : (i - 2) / 2;
          const bool scores = i < 2 || (i & 1);
          if (s >= steps) continue;
          const uint32_t t = kt + (PAIRED ? s >> 1 : s), st = t & 1, b = s & 1;
          const uint32_t s_col = tmem + C::S_COL + b * (FEW ? kFewRows : NT);
          if (scores) {
            if (s < C::QTILES) ok = bar_wait(smem_addr(&sh.q_full[s]), runs & 1, gave_up);
            ok = __all_sync(0xffffffffu, ok && bar_wait(smem_addr(&sh.k_full[st]), (t >> 1) & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            // descriptors differ in their address alone: steps of 16 summed values
            const uint64_t da = q_desc + (PAIRED ? b * (C::Q_BYTES >> 4) : 0), db = k_desc + st * (C::TILE_BYTES >> 4);
            if (elect_one()) {
              if constexpr (FEW) {
                const uint64_t dk = k_chan ? 128 : 2, dk4 = k_chan ? 512 : NT * 8;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_ss(s_col, db + (k >> 2) * dk4 + (k & 3) * dk, da + (k >> 2) * (kFewBytes >> 5) + (k & 3) * 2, qk_desc, k > 0);
              } else if (k_chan) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_ss(s_col, da + (k >> 2) * 1024 + (k & 3) * 2, db + k * 128, qk_desc, k > 0);
              } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_ss(s_col, da + (k >> 2) * 1024 + (k & 3) * 2, db + (k >> 2) * (NT * 8) + (k & 3) * 2, qk_desc, k > 0);
              }
              tc_commit(smem_addr(&sh.s_full[b]));
              if (!PAIRED || b) tc_commit(smem_addr(&sh.k_empty[st]));
            }
            __syncwarp();
          } else {
            const uint32_t done = b ? np1 : np0;
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.v_full[st]), (t >> 1) & 1, gave_up) &&
                                             bar_wait(smem_addr(&sh.p_full[b]), done & 1, gave_up));
            if (!ok) break;
            np0 += b ^ 1;
            np1 += b;
            tc_fence_after();
            const uint64_t db = v_desc + st * (C::TILE_BYTES >> 4);
            const uint32_t o = tmem + C::O_COL + (C::STREAMS == 2 ? b * D : 0);
            const bool add = C::STREAMS == 2 ? s >= 2 : s > 0;
            if (elect_one()) {
              if constexpr (FEW) {
                const uint64_t dv = v_chan ? 2 : 128, dv4 = v_chan ? D * 8 : 512, dp = p_desc + b * (kFewBytes >> 4);
#pragma unroll
                for (int k = 0; k < NT / 16; ++k)
                  mma_ss(o, db + (k >> 2) * dv4 + (k & 3) * dv, dp + (k >> 2) * (kFewBytes >> 5) + (k & 3) * 2, pv_desc,
                         add || k > 0);
                // the rows' sums of P, in every lane
#pragma unroll
                for (int k = 0; k < NT / 16; ++k)
                  mma_ts(tmem + C::L_COL, tmem + C::ONE_COL, dp + (k >> 2) * (kFewBytes >> 5) + (k & 3) * 2, sum_desc, add || k > 0);
              } else if (v_chan) {
#pragma unroll
                for (int k = 0; k < NT / 16; ++k)
                  mma_ts(o, s_col + k * 8, db + (k >> 2) * (D * 8) + (k & 3) * 2, pv_desc, add || k > 0);
              } else {
#pragma unroll
                for (int k = 0; k < NT / 16; ++k) mma_ts(o, s_col + k * 8, db + k * 128, pv_desc, add || k > 0);
              }
              if (C::STREAMS == 1) tc_commit(smem_addr(&sh.pv_done));
              if (!PAIRED || b) tc_commit(smem_addr(&sh.v_empty[st]));
            }
            __syncwarp();
          }
        }
        if (ok && elect_one()) tc_commit(smem_addr(&sh.o_full));
        __syncwarp();
      }
      kt += tiles;
    }
    // Every product issued has left its operands, its accumulators and its barriers before the CTA's
    // shared memory and TMEM go, also after a wait that gave up (else the softmax warps have waited already).
    if (elect_one()) tc_commit(smem_addr(&sh.drained));
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < kChunkSpin && !bar_test(smem_addr(&sh.drained), 0); ++i) {
    }
    __syncwarp();
  } else if (warp >= C::LOAD_WARP && a.direct) {
    if (warp == C::LOAD_WARP) load_direct<D, RT, SEG>(a, sh, run, more, raw_at, lane, entries);
  } else if (warp >= C::LOAD_WARP) {
    // ---- staging ------------------------------------------------------------------------
    int w = warp;
    asm volatile("" : "+r"(w));
    Loader<D> ld;
    ld.lanes(a, w - C::LOAD_WARP, lane);
    const int piece = 2 * ld.which + ld.half;
    const uint32_t slots = a.slots;
    uint4* const orders = sh.orders[w - C::LOAD_WARP];
    uint32_t kt = 0, slot = piece, todo = 3;  // tiles so far; this lane's piece's slot; pieces to ask for
    while (slot >= slots) slot -= slots;
    bool ok = true;
    for (; more && ok; more = warp_run<D, RT, SEG>(a, sh.start, run, 1)) {
      CachePos u;
      // (entries of the list load two tiles ahead, page ids one)
      TileOrder order;
      int4 entry = make_int4(0, 0, 0, 0), next_entry = entry;
      if constexpr (SEG) {
        order.start(run.u, run.t0);
        entry = order.entry(a, run.u, run.t0, NT);
        next_entry = order.entry(a, run.u, run.t0 + 1, NT);
      }
      TileTokens tt = unit_tile<D, SEG>(a, run.u, run.t0, u, &entry);
      ld.unit(a, u);
      const int t1 = run.t1;
      int pid = ld.page_id(a, u, tt.t0, ld.ln);
#pragma unroll 1
      for (int j = run.t0; j < t1; ++j, ++kt) {
        // the next tile's page ids load while this one waits for slots
        CachePos next_u = u;
        int4 after_next = next_entry;
        if constexpr (SEG) after_next = order.entry(a, run.u, j + 2, NT);
        const TileTokens next = SEG ? unit_tile<D, SEG>(a, run.u, min(j + 1, t1 - 1), next_u, &next_entry) : tile_tokens<D>(run.u, min(j + 1, t1 - 1));
        const int next_pid = ld.page_id(a, next_u, next.t0, ld.ln);
        // A lane works out a copy and notes it; one lane then asks for all of a piece's.  (Operands passed by
        // shuffles took 200 to 500 cycles a copy, queued behind the dequantizing warps' shared-memory
        // traffic; an odd chunk of 256-channel heads took 824 us so, 773 us with the notes.)
        const uint8_t* src = nullptr;
        int at = 0;
        bool bad = false;
        const int bytes = ld.source(a, u, tt, ld.ln, pid, &src, &at, &bad);
        const uint32_t bads = __ballot_sync(0xffffffffu, bad) >> (16 * ld.half) & 0xffffu;
        const uint32_t copies = __ballot_sync(0xffffffffu, bytes != 0);
        const uint32_t total0 = __reduce_add_sync(0xffffffffu, ld.half ? 0u : (uint32_t)bytes),
                       total1 = __reduce_add_sync(0xffffffffu, ld.half ? (uint32_t)bytes : 0u);
        if (bytes) {
          const uint64_t from = reinterpret_cast<uint64_t>(src);
          orders[16 * ld.half + __popc(copies >> (16 * ld.half) & ((1u << ld.ln) - 1))] =
              make_uint4((uint32_t)from, (uint32_t)(from >> 32), raw_at + slot * a.slot_bytes + at, (uint32_t)bytes);
        }
        __syncwarp();
        const uint32_t number = 4 * kt + piece, bar = piece * kChunkBars + (kt & (kChunkBars - 1));
        const uint32_t full0 = smem_addr(&sh.raw_full[2 * ld.which * kChunkBars + (kt & (kChunkBars - 1))]);
        // the slot's last piece must have been read
        const uint32_t last = number - slots;
        const uint32_t empty = smem_addr(&sh.raw_empty[(last & 3) * kChunkBars + ((last >> 2) & (kChunkBars - 1))]);
        todo = 3;
#pragma unroll 1
        for (int spin = 0; todo; ++spin) {
          const bool ready = ld.ln == 0 && (todo >> ld.half & 1) &&
                             (number < slots || bar_test(empty, (last >> 2) / kChunkBars & 1));
          const uint32_t b = __ballot_sync(0xffffffffu, ready), now = (b & 1) | (b >> 15 & 2);
          if (ready) {
            sh.bad_pages[bar] = bads;
            if (SEG) entries->at[bar] = entry;
            if (bads) atomicOr(a.status, KVQ_DEV_PAGE);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_addr(&sh.raw_full[bar])),
                         "r"(ld.half ? total1 : total0)
                         : "memory");
          }
          __syncwarp();
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int n = now >> h & 1 ? __popc(copies >> (16 * h) & 0xffffu) : 0;
            if (elect_one()) {
#pragma unroll 4
              for (int c = 0; c < n; ++c) {
                const uint4 x = orders[16 * h + c];
                bulk_copy(x.z, x.x, x.y, x.w, full0 + h * (8 * kChunkBars));
              }
            }
            __syncwarp();
          }
          todo &= ~now;
          if (!now && (spin > kChunkSpin || __any_sync(0xffffffffu, *(volatile uint32_t*)gave_up != 0))) {
            if (lane == 0) *(volatile uint32_t*)gave_up = 1;
            ok = false;
            break;
          }
        }
        if (!ok) break;
        pid = next_pid;
        tt = next;
        if constexpr (SEG) {
          u = next_u;
          entry = next_entry;
          next_entry = after_next;
        }
        slot += 4;
        while (slot >= slots) slot -= slots;
      }
    }
    // the copies in flight land before the CTA ends, also when a warp has
    // given up (then `todo` are the last tile's pieces that were not asked for)
    if (ld.ln == 0) {
#pragma unroll 1
      for (uint32_t back = ok || (todo >> ld.half & 1) ? 1 : 0; back <= 4 && back <= kt; ++back) {
        const uint32_t t = kt - back, bar = smem_addr(&sh.raw_full[piece * kChunkBars + (t & (kChunkBars - 1))]);
        for (int k = 0; k < kChunkSpin && !bar_test(bar, t / kChunkBars & 1); ++k) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= C::SOFT_WARPS) {
    // ---- dequantization ---------------------------------------------------------------
    // Two warps for each piece (half tile of K or V).
    uint32_t kt = 0, slot = (warp - C::SOFT_WARPS) >> 1, slots = a.slots;
    asm volatile("" : "+r"(kt), "+r"(slot));  // not uniform registers: they live across a call
    while (slot >= slots) slot -= slots;
    bool ok = true;
    for (; more && ok; more = warp_run<D, RT, SEG>(a, sh.start, run, 1)) {
      int j = run.t0;
#pragma unroll 1
      while (ok) {
        // What the hot loop keeps in registers is worked out here, after the
        // call below, and hidden from hoisting: kept across the call it would live in local memory.
        int dw = warp - C::SOFT_WARPS;
        asm volatile("" : "+r"(dw));
        const int piece = dw >> 1, which = dw >> 2, half = piece & 1, part = dw & 1, j1 = run.t1;
        const bool per_channel = which ? v_chan : k_chan;
        const uint32_t empty_at = smem_addr(which ? &sh.v_empty[0] : &sh.k_empty[0]),
                       filled_at = smem_addr(which ? &sh.v_full[0] : &sh.k_full[0]);
        const uint32_t full_at = smem_addr(&sh.raw_full[piece * kChunkBars]), read_at = smem_addr(&sh.raw_empty[piece * kChunkBars]);
        const int T = run.u.T, q_last = SEG ? T : q_end_of(a.lo, T), ce = SEG ? 0 : c_end_of(a.lo, T);
        const bool cold = !SEG && j < j1 && tile_tokens<D>(run.u, j).t0 + half * (NT / 2) < ce;
        const RunFmt f = run_fmt(a.lo, which, cold);
        // the hot path's format: bits, 16 for asymmetric blocks; 0: none
        const int kind = (which == 0 && (a.lo.flags & KVQ_K_PRE_ROPE)) || f.codebook ? 0 : f.bits + (f.zp ? 16 : 0);
        PiecePlace q;
        {
          int toff, row, run32;
          RunPlace<D>::of(per_channel, part, 0, lane, &toff, &row, &run32);
          RunPlace<D>::at(per_channel, f, a.sub_bytes, toff, row, run32, &q.blk, &q.codes);
          q.tok = toff;
          q.step = per_channel ? 32 * f.bb : 8 * f.row;
          q.line_step = (per_channel ? 32 : 8) * 128;
          const int tile_row = row + (per_channel ? 0 : half * (NT / 2)), tile_run = run32 + (per_channel ? half * (NT / 64) : 0);
          q.line = RunPlace<D>::line_at(which ? v_at : k_at, tile_row, tile_run, per_channel ? D : NT);
#pragma unroll
          for (int k = 0; k < 4; ++k) q.piece16[k] = (((tile_run & 1) * 4 + k) ^ (row & 7)) << 4;
        }
        bool landed = false;
        [[maybe_unused]] bool filled = false;  // SEG: all but the window's tokens
        // tiles behind the window's first lie in one format and in view up to this token (to whole 32-token subtiles)
        const int st0 = run.u.st, safe = min(cold ? ce : q_last, run.u.p_hi + 32);
        auto stretch = [&](auto fill) {
        int a1 = 1 << 30;  // the piece's end
#pragma unroll 1
        for (; j < j1; ++j, ++kt) {
          const uint32_t st = kt & 1, bar = kt & (kChunkBars - 1);
          bool plain = true;
          int valid = NT / 2;  // SEG: packed tokens of the piece (per-token blocks; the others become zeros)
          [[maybe_unused]] bool raw = false;  // SEG: and tokens of the 16-bit window behind them
          a1 += NT;
          if (!SEG && (j <= st0 || a1 > safe)) {
            const TileTokens tt = tile_tokens<D>(run.u, j);
            const int a0 = tt.t0 + half * (NT / 2), qe = q_last;
            a1 = a0 + NT / 2;
            if ((a0 < ce) != cold) break;  // the other tier's format
            // of one format, wholly in view (to whole 32-token subtiles) and in range: the common case
            plain = a0 + 31 >= tt.v0 && a1 - 31 <= tt.v1 && a1 <= qe && (!cold || a1 <= ce);
          }
          ok = __all_sync(0xffffffffu, bar_wait(empty_at + 8 * st, ((kt >> 1) & 1) ^ 1, gave_up) &&
                                           bar_wait(full_at + 8 * bar, kt / kChunkBars & 1, gave_up));
          if (!ok) break;
          landed = true;
          if (SEG) {
            const int4 entry = entries->at[piece * kChunkBars + bar];
            if (entry.w >= 0) {
              const int a0 = entry.y + half * (NT / 2), qe = q_end_of(a.lo, entry.z);
              valid = qe - a0;
              raw = valid < NT / 2 && max(a0, qe) < entry.z;
            }
          }
          if (!plain || *(volatile uint32_t*)&sh.bad_pages[piece * kChunkBars + bar]) break;
          if (!fill(raw_at + slot * a.slot_bytes, st * C::TILE_BYTES, valid)) break;
          if (SEG && raw) {
            filled = true;
            break;
          }
          proxy_fence();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(read_at + 8 * bar);
            bar_arrive(filled_at + 8 * st);
          }
          slot += 4;
          while (slot >= slots) slot -= slots;
          landed = false;
        }
        };
        // (a loop a format: the formats' branches are outside of it)
        auto by_kind = [&](auto key) {
          constexpr bool KEY = decltype(key)::value;
          const uint32_t one = KEY ? a.k_one : kOnes;
          if (kind == 4)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 4, false, SEG>(q, staged, dst, valid, one); });
          else if (kind == 8)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 8, false, SEG>(q, staged, dst, valid, one); });
          else if (kind == 2)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 2, false, SEG>(q, staged, dst, valid, one); });
          else if (kind == 3)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 3, false, SEG>(q, staged, dst, valid, one); });
          else if (kind == 20)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 4, true, SEG>(q, staged, dst, valid, one); });
          else if (kind == 18)
            stretch([&](uint32_t staged, uint32_t dst, int valid) { return fill_piece<DT, KEY, 2, true, SEG>(q, staged, dst, valid, one); });
          else
            stretch([&](uint32_t, uint32_t, int) { return false; });
        };
        if (DT == KVQ_DT_BF16 && which == 0)
          by_kind(std::integral_constant<bool, DT == KVQ_DT_BF16>{});
        else
          by_kind(std::false_type{});
        if (!ok || j >= j1) break;
        if (landed) {
          if (SEG && filled)
            window_tokens<D, DT>(a, sh, run, which ? v_at : k_at, dw, kt, entries);
          else
            cold_piece<D, DT, SEG>(a, sh, run, which ? v_at : k_at, raw_at, dw, kt, slot, j, entries);
          proxy_fence();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(smem_addr(&sh.raw_empty[piece * kChunkBars + (kt & (kChunkBars - 1))]));
            bar_arrive(smem_addr(which ? &sh.v_full[kt & 1] : &sh.k_full[kt & 1]));
          }
          slot += 4;
          while (slot >= slots) slot -= slots;
          ++j;
          ++kt;
        }
      }
    }
  } else if constexpr (FEW) {
    few_rows<DT, SEG>(a, sh, more, smem, tmem, entries);
  } else {
    // ---- softmax and outputs -----------------------------------------------------------
    uint32_t ns0 = 0, ns1 = 0, runs = 0, steps_done = 0, syncs = 0;
    [[maybe_unused]] int tiles_done = 0;  // of the runs before
    asm volatile("" : "+r"(ns0), "+r"(ns1), "+r"(runs), "+r"(steps_done), "+r"(syncs));  // as above
    bool ok = true;
    for (; more && ok; more = warp_run<D, RT, SEG>(a, sh.start, run, 1), ++runs) {
      int w = warp;  // worked out anew for every run: see the dequantizing warps
      asm volatile("" : "+r"(w));
      const int stream = w >> 2, quad = w & 3;
      const int my_lane = quad * 32 + lane;  // TMEM lane: row of the 128-row tile
      const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
      const uint32_t o_col = lane_base + C::O_COL + (C::STREAMS == 2 ? stream * D : 0);
      const int my_row = (PAIRED ? stream * 128 : 0) + my_lane;  // query row of the row tile
      const float sc = a.score_scale;
      // queries into shared memory
      if (PAIRED || stream == 0) {
        const int first = PAIRED ? stream * 128 : 0, n = min(128, run.u.rows - first);  // rows
        const uint32_t q0 = q_at + (PAIRED ? stream * C::Q_BYTES : 0);
        if (a.turn_here) {
          // few rows, turned into the rotated domain here: a warp a row
          const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
          constexpr int NC = D / 128;
#pragma unroll 1
          for (int e = quad; e < n * NC; e += 4) {
            const int r = e / NC, c = e % NC;
            uint2 w = __ldcg(reinterpret_cast<const uint2*>(a.q + query_row(a, run.u, first + r) + 128 * c) + lane);
            float v[4] = {in_to_f32((uint16_t)w.x, DT), in_to_f32((uint16_t)(w.x >> 16), DT),
                          in_to_f32((uint16_t)w.y, DT), in_to_f32((uint16_t)(w.y >> 16), DT)};
            rotate_lanes(v, s1, s2, a.q_pre);
            w = query_pack<DT>(v);
            const int ch = 128 * c + 4 * lane;
            const uint32_t at = q0 + (uint32_t)(ch >> 6) * 16384 + swz(r, (ch & 63) >> 3) + (ch & 4) * 2;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at), "r"(w.x), "r"(w.y) : "memory");
          }
        } else {
          constexpr int LPR = D / 8, RPT = 32 / LPR, U = 4;  // lanes a row, rows a turn, turns in flight
          const int ch = 8 * (lane & (LPR - 1)), sub = lane / LPR;
          const uint32_t col = q0 + (uint32_t)(ch >> 6) * 16384;
#pragma unroll 1
          for (int r0 = quad * RPT + sub; r0 - sub < n; r0 += 4 * RPT * U) {
            uint4 w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const int r = r0 + 4 * RPT * i;
              w[i] = make_uint4(0, 0, 0, 0);
              if (r < n) w[i] = __ldcg(reinterpret_cast<const uint4*>(a.q + query_row(a, run.u, first + r) + ch));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const int r = r0 + 4 * RPT * i;
              if (DT == KVQ_DT_BF16 && !(a.lo.flags & KVQ_ROTATE_K))  // (turned queries are fp16 already)
                w[i] = make_uint4(score_pair<DT>(w[i].x, 1.f), score_pair<DT>(w[i].y, 1.f), score_pair<DT>(w[i].z, 1.f),
                                  score_pair<DT>(w[i].w, 1.f));
              if (r < n)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(col + swz(r, (ch & 63) >> 3)), "r"(w[i].x),
                             "r"(w[i].y), "r"(w[i].z), "r"(w[i].w)
                             : "memory");
            }
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.q_full[PAIRED ? stream : 0]));
      }
      RowSeen row_sees;
      row_sees.pos = row_pos<SEG>(a, run.u, SEG ? min(my_row, run.u.rows - 1) : my_row);
      row_sees.win_lo = !SEG && a.window ? max(0, row_sees.pos - a.window + 1) : 0;
      row_sees.sinks = a.sinks;
      const int steps = (PAIRED ? 2 : 1) * (run.t1 - run.t0), first_tile = run.t0;
      const int st = run.u.st, skip = run.u.lo_tile - st, p_lo = run.u.p_lo, p_hi = run.u.p_hi;
      float m = -INFINITY, l = 0.f;
      bool first_step = true;
#pragma unroll 1
      for (int s = C::STREAMS == 2 ? stream : 0; s < steps; s += C::STREAMS) {
        const int b = s & 1;
        const int j = first_tile + (PAIRED ? s >> 1 : s);
        int t0 = (j < st ? j : j + skip) * NT;
        bool masked = t0 + NT - 1 > p_lo || (a.window && t0 <= p_hi - a.window && t0 + NT > a.sinks);
        const uint32_t s_col = lane_base + C::S_COL + b * NT;
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.s_full[b]), (b ? ns1 : ns0) & 1, gave_up));
        if (!ok) break;
        RowSeen see = row_sees;
        if constexpr (SEG) {
          const int4 x = entries->at[(tiles_done + (j - first_tile)) & (kChunkBars - 1)];
          masked = false;  // of the prefix every row sees every token
          if (x.w >= 0) {
            const int r_lo = x.w & 0xffff, r_hi = x.w >> 16;
            t0 = x.y;
            masked = t0 + NT - 1 > p_lo || r_lo > 0 || r_hi < run.u.rows;
            if (my_row < r_lo || my_row >= r_hi) see.pos = -1;
            // none of the warp's rows: P is zeros (drafts of 32 chats 243 -> 238 us)
            if (my_row - lane >= r_hi || my_row - lane + 32 <= r_lo) {
              ns0 += b ^ 1;
              ns1 += b;
              tc_fence_after();
              uint32_t zero[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll
              for (int c = 0; c < NT / 2; c += 16) tmem_st16(s_col + c, zero);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) bar_arrive(smem_addr(&sh.p_full[b]));
              ++steps_done;
              first_step = false;
              continue;
            }
          }
        }
        ns0 += b ^ 1;
        ns1 += b;
        tc_fence_after();
        const float mt = sc * (masked ? tile_max<NT, true>(s_col, t0, see) : tile_max<NT, false>(s_col, t0, see));
        // the reference maximum follows only when it falls behind by 2^8: P
        // stays below 2^8 and the accumulator is rescaled rarely
        const bool grow = mt > m + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
          const float nm = grow ? mt : m;
          const float f = m == -INFINITY ? 0.f : ex2(m - nm);
          l = l == 0.f ? 0.f : l * f;
          m = nm;
          if (!first_step) {
            if (C::STREAMS == 1) {
              // the products of the step before must have left the accumulator
              ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.pv_done), (steps_done - 1) & 1, gave_up));
              if (!ok) break;
              tc_fence_after();
            }
            rescale_columns<D>(o_col, f);
          }
        }
        first_step = false;
        const float mneg = m == -INFINITY ? 0.f : -m;
        l += masked ? tile_exp<DT, NT, true>(s_col, t0, see, sc, mneg) : tile_exp<DT, NT, false>(s_col, t0, see, sc, mneg);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.p_full[b]));
        ++steps_done;
      }
      if constexpr (SEG) tiles_done += run.t1 - first_tile;
      // ---- the run's outputs -----------------------------------------------------------
      if (!ok) break;
      ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.o_full), runs & 1, gave_up));
      if (!ok) break;
      tc_fence_after();
      const bool cut = run.t0 > 0 || run.t1 < run.u.nt, mine = my_row < run.u.rows;
      const bool direct = !cut && (PAIRED || C::STREAMS == 1);
      uint32_t x[16];
      if (direct) {
        const bool rotated = (a.lo.flags & KVQ_ROTATE_V) != 0, fix = *(volatile uint32_t*)&sh.nonfinite != 0;
        const float inv = 1.f / l, f = rotated ? 1.f : inv;
        if (rotated) {
#pragma unroll 1
          for (int c = 0; c < D; c += 128) unrotate_columns(a, o_col + c, inv);
        }
        uint16_t* dst = a.out + query_row(a, run.u, mine ? my_row : 0);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          tmem_ld16(o_col + c, x);
          const uint32_t signs = rotated ? a.lo.d1[c >> 5 & 3] >> (c & 16) : 0u;
          tmem_wait_ld();
          if (mine) {
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              p[i] = pack16<DT>(__uint_as_float(x[2 * i] ^ ((signs << (31 - 2 * i)) & 0x80000000u)) * f,
                                __uint_as_float(x[2 * i + 1] ^ ((signs << (30 - 2 * i)) & 0x80000000u)) * f);
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(p[0], p[1], p[2], p[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(p[4], p[5], p[6], p[7]);
          }
          __syncwarp();
        }
        if (fix) add_nonfinite<D, DT, SEG>(a, run, my_row - lane, min(my_row - lane + 32, run.u.rows), 1);
        __syncwarp();
        tc_fence_before();
      } else {
        const int slot = !cut ? 2 : run.first ? 0 : 1;
        float* part = a.partials + (((int64_t)blockIdx.x * kChunkSlots + slot) * chunk_slot_rows(D) + stream * 128 + my_lane) *
                                       chunk_part_row(D);
        // a stream without a step of this run has no accumulator
        const bool none = C::STREAMS == 2 && stream >= steps;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          tmem_ld16(o_col + c, x);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(part + c + i) =
                  none ? make_uint4(0, 0, 0, 0) : make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
          __syncwarp();
        }
        if (mine) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
        tc_fence_before();
        const uint32_t soft = smem_addr(&sh.soft);
        bool join = !cut, fix = false;
        // a unit's ticket belongs to its first CTA: entry 0 when the unit
        // starts with that CTA's stretch, else 1
        const int unit_pos = run.pos - run.t0, c0 = unit_pos / sh.start.per_cta;
        const int tick = c0 * kChunkTickets + (unit_pos - unit_cost<SEG>(a) <= c0 * sh.start.per_cta ? 0 : 1);
        if (cut) __threadfence();
        if (!(ok = soft_sync(soft, syncs, gave_up))) break;
        if (cut) {
          if (tid == 0) {
            if (*(volatile uint32_t*)&sh.nonfinite) atomicOr(a.nonfinite + tick, 1u);
            __threadfence();
            const int c1 = (unit_pos + run.u.nt - 1) / sh.start.per_cta;
            sh.last = atomicAdd(a.tickets + tick, 1u) == (uint32_t)(c1 - c0);
          }
          if (!(ok = soft_sync(soft, syncs, gave_up))) break;
          join = *(volatile uint32_t*)&sh.last != 0;
          if (join) {
            __threadfence();
            fix = __ldcg(a.nonfinite + tick) != 0;
          }
        } else {
          fix = *(volatile uint32_t*)&sh.nonfinite != 0;
        }
        // (the queries' shared memory is free: the run's products are done)
        if (join && !(ok = join_unit<D, DT, MODE, SEG>(a, run, sh.start, cut, fix, reinterpret_cast<float*>(smem), soft, syncs, gave_up)))
          break;
        if (!(ok = soft_sync(soft, syncs, gave_up))) break;
        if (join && cut && tid == 0) {
          a.tickets[tick] = 0;
          a.nonfinite[tick] = 0;
        }
      }
    }
  }
  // every role ends here, also after a wait that gave up
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    if (sh.gave_up) atomicOr(a.status, KVQ_DEV_STALL);
    // Every CTA comes by here, whether its waits held or not.  The last one takes back what a stalled call has
    // counted: its cut units have tickets that no CTA draws any more, and the next call would count on from them.
    __threadfence();
    const uint32_t before = atomicAdd(a.left, sh.gave_up ? 0x10001u : 1u);
    if ((before & 0xffffu) == gridDim.x - 1) {
      __threadfence();
      if (sh.gave_up || before >> 16)
        for (int i = 0; i < (int)gridDim.x * kChunkTickets; ++i) a.tickets[i] = a.nonfinite[i] = 0;
      *a.left = 0;
    }
  }
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

// Queries of a rotated format turned into the rotated domain, into their rows
// of `out` (which a row's outputs replace when everything that reads it has been read): a
// warp per (layer, row).  With many rows a sequence, turning them as they are loaded kept the products
// waiting a fifth of the time.
template <int D, int DT>
__global__ void __launch_bounds__(256) turn_queries_kernel(const __grid_constant__ ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)a.n_layers * a.total_q) return;
  const int row = (int)(w % a.total_q);
  int lo = 0, hi = a.lo.B;  // the last b with cu_q[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(a.cu_q + mid) <= row)
      lo = mid;
    else
      hi = mid;
  }
  int n, T, cu;
  if (!valid_seq(a, lo, &n, &T, &cu) || row < cu || row >= cu + n) return;  // rows of no sequence stay as they are
  const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
  const uint2* src = reinterpret_cast<const uint2*>(a.q + w * a.lo.Hq * D) + lane;
  uint2* dst = reinterpret_cast<uint2*>(a.out + w * a.lo.Hq * D) + lane;
  const int chunks = a.lo.Hq * (D / 128);
#pragma unroll 1
  for (int c0 = 0; c0 < chunks; c0 += 4) {
    uint2 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k < chunks) x[k] = __ldcg(src + 32 * (c0 + k));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k < chunks) {
        float v[4] = {in_to_f32((uint16_t)x[k].x, DT), in_to_f32((uint16_t)(x[k].x >> 16), DT),
                      in_to_f32((uint16_t)x[k].y, DT), in_to_f32((uint16_t)(x[k].y >> 16), DT)};
        rotate_lanes(v, s1, s2, a.q_pre);
        dst[32 * (c0 + k)] = query_pack<DT>(v);
      }
  }
}

// The same for planned units: a block a unit, its tokens' heads four 128-chunks a warp at a time.  (A token of two units is turned twice.)
template <int D, int DT, int RT>
__global__ void __launch_bounds__(256) turn_units_kernel(const __grid_constant__ ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  Unit u;
  if (!plan_fits(a) || !planned_unit<D, RT>(a, blockIdx.x, u)) return;
  const uint32_t s1 = lane_signs(a.lo.d1, lane), s2 = lane_signs(a.lo.d2, lane);
  const int chunks = a.lo.Hq * (D / 128), per = (chunks + 3) / 4;
  const int tok0 = div_g(a, u.r0), n = div_g(a, u.r0 + u.rows - 1) - tok0 + 1;
  const int64_t items = (int64_t)a.n_layers * n * per;
#pragma unroll 1
  for (int64_t i = blockIdx.y * 8 + (threadIdx.x >> 5); i < items; i += gridDim.y * 8) {
    const int c0 = (int)(i % per) * 4;
    const int64_t r = i / per, row = r / n * a.total_q + u.cu + tok0 + r % n;
    const uint2* src = reinterpret_cast<const uint2*>(a.q + row * a.lo.Hq * D) + lane;
    uint2* dst = reinterpret_cast<uint2*>(a.out + row * a.lo.Hq * D) + lane;
    uint2 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k < chunks) x[k] = __ldcg(src + 32 * (c0 + k));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k < chunks) {
        float v[4] = {in_to_f32((uint16_t)x[k].x, DT), in_to_f32((uint16_t)(x[k].x >> 16), DT),
                      in_to_f32((uint16_t)x[k].y, DT), in_to_f32((uint16_t)(x[k].y >> 16), DT)};
        rotate_lanes(v, s1, s2, a.q_pre);
        dst[32 * (c0 + k)] = query_pack<DT>(v);
      }
  }
}

template <int D, int DT, int MODE, bool SEG = false>
cudaError_t launch_chunk(ChunkArgs a, int grid, cudaStream_t s) {
  using C = ChunkShape<D, MODE>;
  // all of the SM's shared memory that the tiles leave is staging
  const uint32_t all = 227 * 1024 - (uint32_t)sizeof(typename C::Shared) - (SEG ? (uint32_t)sizeof(TileEntries) : 0);
  const uint32_t left = all - C::FIXED - 16;
  a.slots = (int)(left / a.slot_bytes);
  if (a.slots > kChunkMaxSlots) a.slots = kChunkMaxSlots;
  if (a.slots < 1) return cudaErrorInvalidConfiguration;
  const uint32_t smem = C::FIXED + 16 + a.slots * a.slot_bytes;
  // The attribute belongs to the function and the current device, so it is set on every call, and always to the same
  // value: another thread's call, of another format, may come between this and the launch.  Before the queries
  // are turned: a failure here leaves `out` as it was.
  cudaError_t e = cudaFuncSetAttribute(chunk_attention_kernel<D, DT, MODE, SEG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)all);
  if (e != cudaSuccess) return e;
  if ((a.lo.flags & KVQ_ROTATE_K) && !a.turn_here) {
    if constexpr (SEG) {
      const int64_t items = (int64_t)a.n_layers * C::RT / a.lo.g * ((a.lo.Hq * (D / 128) + 3) / 4);
      const unsigned parts = (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + 7) / 8, 4 * grid / a.n_units + 1));
      e = launch_dependent(turn_units_kernel<D, DT, C::RT>, dim3(a.n_units, parts), dim3(256), 0, s, a);
    } else {
      const int64_t rows = (int64_t)a.n_layers * a.total_q;
      e = launch_dependent(turn_queries_kernel<D, DT>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a);
    }
    if (e != cudaSuccess) return e;
    a.q = a.out;
  }
  return launch_dependent(chunk_attention_kernel<D, DT, MODE, SEG>, dim3(grid), dim3(C::THREADS), smem, s, a);
}

}  // namespace
}  // namespace kvq
