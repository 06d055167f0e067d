// The chunk attention kernel (design in chunk_attention.cuh).
#pragma once

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
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits, boundedly, for the phase of that parity.  After too many polls, or
// once another warp has given up, the answer is false and the caller leaves.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
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

// ---- the units' line ---------------------------------------------------------------

struct Unit {
  int layer, h, b, rt;
  int n, T, cu;          // rows' tokens, cached tokens, first row of q
  int r0, rows;          // first query row (token * g + head) and rows of this row tile
  int p_lo, p_hi;        // positions of its first and last token
  int lo;                // first token of the window
  int sink;              // tokens [0, sink) visible besides
  int st, lo_tile, nt;   // sink tiles, first window tile, tiles
};

__device__ __forceinline__ bool valid_seq(const ChunkArgs& a, int b, int* n, int* T, int* cu) {
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), t = __ldg(a.seq_lens + b);
  *cu = c0;
  *n = c1 - c0;
  *T = t;
  return c0 >= 0 && c1 >= c0 && c1 <= a.total_q && c1 - c0 <= a.max_q && t >= c1 - c0 && t <= a.lo.max_T;
}

template <int D, int RT>
__device__ __forceinline__ void unit_tiles(const ChunkArgs& a, Unit& u) {
  constexpr int NT = chunk_tile(D);
  u.r0 = u.rt * RT;
  u.rows = min(RT, u.n * a.lo.g - u.r0);
  u.p_lo = u.T - u.n + u.r0 / a.lo.g;
  u.p_hi = u.T - u.n + (u.r0 + u.rows - 1) / a.lo.g;
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

// Tiles of sequence b (one layer and kv head): summed by one thread, or by the 32 lanes of a warp.
template <int D, int RT>
__device__ __forceinline__ int64_t seq_tiles(const ChunkArgs& a, int b, int lane, int lanes, bool* bad) {
  Unit u;
  u.b = b;
  if (!valid_seq(a, b, &u.n, &u.T, &u.cu)) {
    *bad = true;
    return 0;
  }
  int64_t sum = 0;
  const int nrt = seq_row_tiles<D, RT>(a, u.n);
  for (u.rt = lane; u.rt < nrt; u.rt += lanes) {
    unit_tiles<D, RT>(a, u);
    sum += u.nt;
  }
  return sum;
}

// The unit after u (of the same or the next sequence, kv head, layer); false
// past the last one (only where lengths changed under the kernel).
template <int D, int RT>
__device__ __forceinline__ bool next_unit(const ChunkArgs& a, Unit& u) {
  ++u.rt;
  if (u.rt >= seq_row_tiles<D, RT>(a, u.n)) {
    u.rt = 0;
    bool ok;
    do {
      if (++u.b == a.lo.B) {
        u.b = 0;
        if (++u.h == a.lo.H) {
          u.h = 0;
          if (++u.layer == a.n_layers) return false;
        }
      }
      ok = valid_seq(a, u.b, &u.n, &u.T, &u.cu) && u.n > 0;
    } while (!ok);
  }
  unit_tiles<D, RT>(a, u);
  return true;
}

// One CTA's run of a unit: tiles [t0, t1) of it.
struct Run {
  Unit u;
  int t0, t1;
  int64_t pos;   // place of the run's first tile on the line
  bool first;    // the CTA's first run
};

struct LineStart {  // found once per CTA
  int lh, b, rt, tile;
  int64_t begin, end;  // the CTA's stretch of the line
  int64_t per_cta;
};

template <int D, int RT>
__device__ __forceinline__ bool first_run(const ChunkArgs& a, const LineStart& s, Run& r) {
  if (s.begin >= s.end) return false;
  r.u.layer = s.lh / a.lo.H;
  r.u.h = s.lh % a.lo.H;
  r.u.b = s.b;
  r.u.rt = s.rt;
  (void)valid_seq(a, s.b, &r.u.n, &r.u.T, &r.u.cu);
  unit_tiles<D, RT>(a, r.u);
  r.t0 = s.tile;
  r.pos = s.begin;
  r.t1 = (int)min((int64_t)r.u.nt, r.t0 + (s.end - r.pos));
  r.first = true;
  return true;
}
template <int D, int RT>
__device__ __forceinline__ bool next_run(const ChunkArgs& a, const LineStart& s, Run& r) {
  r.pos += r.t1 - r.t0;
  if (r.pos >= s.end) return false;
  if (!next_unit<D, RT>(a, r.u)) return false;
  r.t0 = 0;
  r.t1 = (int)min((int64_t)r.u.nt, s.end - r.pos);
  r.first = false;
  return true;
}

// ---- dequantization --------------------------------------------------------------------

// 32 codes of `bits` bits at p (2-byte aligned) as fp16 pairs, exact: signed
// codes, or the raw fields when `raw` (asymmetric blocks), or table values (TBQ4).
__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// fields at bits [0, w) of each half, as fp16 integers minus the bias: 1024 + field is exact in fp16
__device__ __forceinline__ uint32_t field_pair(uint32_t x, uint32_t mask, uint32_t bias2) {
  return hsub2u((x & mask) | 0x64006400u, bias2);
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds_half(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(at));
  return __half2float(__ushort_as_half(v));
}
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
__device__ __forceinline__ void codes32(uint32_t p, int bits, bool raw, const uint32_t* pair_table,
                                        uint32_t (&h)[16]) {
  if (bits == 4) {
    uint32_t w[4];
    load_words(p, w);
    if (pair_table) {
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = pair_table[(w[i / 4] >> (8 * (i % 4))) & 0xff];
      return;
    }
    const uint32_t bias = raw ? 0x64006400u : 0x64086408u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = w[i] >> 4;
      h[4 * i] = field_pair(__byte_perm(w[i], v, 0x0400), 0x000f000fu, bias);
      h[4 * i + 1] = field_pair(__byte_perm(w[i], v, 0x1511), 0x000f000fu, bias);
      h[4 * i + 2] = field_pair(__byte_perm(w[i], v, 0x2622), 0x000f000fu, bias);
      h[4 * i + 3] = field_pair(__byte_perm(w[i], v, 0x3733), 0x000f000fu, bias);
    }
  } else if (bits == 8) {
    uint32_t w[8];
    load_words(p, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = w[i] ^ 0x80808080u;
      h[2 * i] = hsub2u(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
      h[2 * i + 1] = hsub2u(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
    }
  } else if (bits == 3) {
    uint32_t w[3];
    load_words(p, w);
    const uint32_t g[4] = {w[0], __funnelshift_r(w[0], w[1], 24), __funnelshift_r(w[1], w[2], 16), w[2] >> 8};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t t = g[k] >> (6 * j);
        h[4 * k + j] = field_pair((t & 7u) | ((t & 0x38u) << 13), 0x00070007u, 0x64046404u);
      }
  } else {
    uint32_t w[2];
    load_words(p, w);
    const uint32_t bias = raw ? 0x64006400u : 0x64026402u;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t x = (w[i] >> (8 * b)) & 0xffu;
        const uint32_t y = x | (x << 14);  // fields 0 and 2 low; 1 and 3 at bit 16 and 20
        h[8 * i + 2 * b] = field_pair(y, 0x00030003u, bias);
        h[8 * i + 2 * b + 1] = field_pair(y >> 4, 0x00030003u, bias);
      }
  }
}

__device__ __forceinline__ float2 half2_f(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// Scale and zero of a block; a scale that is not finite (the block's values are unspecified) counts as 0.
struct BlockScale {
  float s, z;
  bool big;  // a value may leave fp16's range
};
__device__ __forceinline__ BlockScale block_scale_of_run(uint32_t blk, const FmtInfo& f) {
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
// bf16: through fp32, where the product is exact.  Values past fp16's range saturate: an
// infinity would turn a masked token's zero probability into NaN.
template <int DT>
__device__ __forceinline__ void scale32(uint32_t (&h)[16], const BlockScale& b, bool zp) {
  if constexpr (DT == KVQ_DT_F16) {
    if (!b.big) {
      const __half2 s2 = __float2half2_rn(b.s), z2 = __float2half2_rn(b.z);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __half2 c = *reinterpret_cast<const __half2*>(&h[i]);
        const __half2 v = zp ? __hfma2(c, s2, z2) : __hmul2(c, s2);
        h[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 c = half2_f(h[i]);
    float x = fmaf(c.x, b.s, b.z), y = fmaf(c.y, b.s, b.z);
    if constexpr (DT == KVQ_DT_F16) {
      x = fminf(fmaxf(x, -65504.f), 65504.f);
      y = fminf(fmaxf(y, -65504.f), 65504.f);
    }
    h[i] = pack16<DT>(x, y);
  }
}

__device__ __forceinline__ void store32(uint32_t dst, int row, int run, int rows, const uint32_t (&h)[16]) {
  const uint32_t blk = dst + (uint32_t)(run >> 1) * rows * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(blk + swz(row, (run & 1) * 4 + j)),
                 "r"(h[4 * j]), "r"(h[4 * j + 1]), "r"(h[4 * j + 2]), "r"(h[4 * j + 3])
                 : "memory");
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

// Dequantizes half of one tensor's tile (a piece: 256 runs of 32 values, one
// per dequantizing thread) from its staged packed bytes into the swizzled
// shared-memory tile at dst.  Rows of the tile are tokens (per-token blocks,
// runs along channels) or channels (per-channel blocks, runs along tokens).
template <int D, int DT>
struct Dequant {
  static constexpr int NT = chunk_tile(D);
  static constexpr int PIECE = NT / 2;  // tokens of a piece
  static constexpr int THREADS = 32 * kChunkDequantWarps;

  const ChunkArgs& a;
  const Unit& u;
  int which, warp, lane;
  uint32_t dst;
  int qe, ce;
  const uint32_t* pair_table;
  volatile uint32_t* nonfinite;
  int a0;           // the piece's first token
  uint32_t staged;  // its packed bytes: 32-token subtiles, a.sub_bytes apart
  uint32_t bad;     // copies (of a.copy_shift tokens each) whose page id is out of range

  __device__ __forceinline__ bool turned() const { return which == 0 && (a.lo.flags & KVQ_K_PRE_ROPE); }
  __device__ __forceinline__ const FmtInfo& fmt_of(int t) const {
    return t < ce ? fmt_cold(a.lo, which) : fmt_main(a.lo, which);
  }
  // block of the run (token or channel row, run) of a quantized tier and its codes
  __device__ __forceinline__ uint32_t token_block(int t, int run, const FmtInfo& f, uint32_t* codes) const {
    const int per = f.group / 32;  // runs of a block: 1 or 4
    const uint32_t blk = staged + ((t - a0) >> 5) * a.sub_bytes + (t & 31) * f.row + (per == 1 ? run : run >> 2) * f.bb;
    *codes = blk + (f.zp ? 4 : 2) + (per == 1 ? 0 : (run & 3) * 4 * f.bits);
    return blk;
  }
  __device__ __forceinline__ uint32_t channel_block(int t, int c, const FmtInfo& f, uint32_t* codes) const {
    const uint32_t blk = staged + ((t - a0) >> 5) * a.sub_bytes + c * f.bb;
    *codes = blk + (f.zp ? 4 : 2);
    return blk;
  }
  __device__ __forceinline__ bool no_page(int t) const { return (bad >> ((t - a0) >> a.copy_shift)) & 1u; }

  // 16-bit window values as they are; values that are not finite become 0 in V's tile (see fix_rows)
  __device__ __forceinline__ uint32_t clean(uint32_t w) const {
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

  __device__ __forceinline__ void raw_token_run(int t, int run, uint32_t (&h)[16]) const {
    const uint4* p = reinterpret_cast<const uint4*>(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t)) + run * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 v = p[j];
      h[4 * j] = clean(v.x);
      h[4 * j + 1] = clean(v.y);
      h[4 * j + 2] = clean(v.z);
      h[4 * j + 3] = clean(v.w);
    }
  }
  // channel c of tokens t .. t + 31, zeros from token T on
  __device__ __forceinline__ void raw_channel_run(int t, int c, uint32_t (&h)[16]) const {
    const uint16_t* p = resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t) + c;
    int left = a.lo.ring - t % a.lo.ring;  // slots until the ring wraps
    uint32_t x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      x[j] = *p;  // slots past the length exist, and count as zeros below
      --left;
      p += left == 0 ? (int64_t)a.lo.D - (int64_t)a.lo.ring * a.lo.D : (int64_t)a.lo.D;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (t + j >= u.T) x[j] = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = clean(x[2 * j] | (x[2 * j + 1] << 16));
  }

  // One run, turn aside, in the input dtype.
  __device__ __forceinline__ void token_run(int t, int run, uint32_t (&h)[16]) const {
    if (t >= u.T || no_page(t)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = 0;
    } else if (t >= qe) {
      raw_token_run(t, run, h);
    } else {
      const FmtInfo& f = fmt_of(t);
      uint32_t codes;
      const uint32_t blk = token_block(t, run, f, &codes);
      codes32(codes, f.bits, f.zp, f.codebook ? pair_table : nullptr, h);
      scale32<DT>(h, block_scale_of_run(blk, f), f.zp);
    }
  }
  __device__ __forceinline__ void channel_run(int t, int c, uint32_t (&h)[16]) const {
    if (t >= qe) {
      raw_channel_run(t, c, h);
    } else {
      const FmtInfo& f = fmt_of(t);
      uint32_t codes;
      const uint32_t blk = channel_block(t, c, f, &codes);
      codes32(codes, f.bits, f.zp, nullptr, h);
      scale32<DT>(h, block_scale_of_run(blk, f), f.zp);
    }
  }

  // Values of a run as code pairs and (scale, zero), for the turn in fp32; window values are pairs of the input dtype
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
  __device__ __forceinline__ void loose_token(int t, int run, Loose& l) const {
    l.raw = true;
    if (t >= u.T || no_page(t)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) l.h[i] = 0;
    } else if (t >= qe) {
      raw_token_run(t, run, l.h);
    } else {
      const FmtInfo& f = fmt_of(t);
      uint32_t codes;
      const uint32_t blk = token_block(t, run, f, &codes);
      codes32(codes, f.bits, f.zp, nullptr, l.h);
      const BlockScale b = block_scale_of_run(blk, f);
      l.raw = false;
      l.s = b.s;
      l.z = b.z;
    }
  }
  __device__ __forceinline__ void loose_channel(int t, int c, Loose& l) const {
    l.raw = t >= qe;
    if (l.raw) {
      raw_channel_run(t, c, l.h);
    } else {
      const FmtInfo& f = fmt_of(t);
      uint32_t codes;
      const uint32_t blk = channel_block(t, c, f, &codes);
      codes32(codes, f.bits, f.zp, nullptr, l.h);
      const BlockScale b = block_scale_of_run(blk, f);
      l.s = b.s;
      l.z = b.z;
    }
  }
  // cos and sin of a 64-bit turn fraction
  __device__ __forceinline__ static float2 cos_sin(uint64_t turn) {
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
  }
  __device__ __forceinline__ static float keep_range(float x) {
    if constexpr (DT == KVQ_DT_F16) return isinf(x) || isnan(x) ? x : fminf(fmaxf(x, -65504.f), 65504.f);
    return x;
  }

  // Keys stored pre-RoPE: the runs of channels i and i + D/2 together.
  __device__ void turned_tile(const TileTokens& tt, bool per_channel) const {
    if (per_channel) {
      constexpr int G = PIECE / 32;  // token groups of the piece
      for (int e = warp * 32 + lane; e < (D / 2) * G; e += THREADS) {
        const int c = (e & 7) | ((e / (8 * G)) << 3);
        const int t = a0 + 32 * ((e >> 3) % G), run = (t - tt.t0) >> 5;
        if (t + 32 <= tt.v0 || t >= tt.v1) continue;
        Loose x, y;
        loose_channel(t, c, x);
        loose_channel(t, c + D / 2, y);
        const uint64_t w = a.turns[c];
        // token after token the angle grows by the same step: a complex
        // product each, 31 times from an exact start (error below 31 x 2^-22)
        float2 k = cos_sin((uint64_t)t * w);
        const float2 step = cos_sin(w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 xa = x.value(i), ya = y.value(i);
          const float x0 = xa.x * k.x - ya.x * k.y, y0 = ya.x * k.x + xa.x * k.y;
          k = make_float2(k.x * step.x - k.y * step.y, k.y * step.x + k.x * step.y);
          const float x1 = xa.y * k.x - ya.y * k.y, y1 = ya.y * k.x + xa.y * k.y;
          k = make_float2(k.x * step.x - k.y * step.y, k.y * step.x + k.x * step.y);
          x.h[i] = pack16<DT>(keep_range(x0), keep_range(x1));
          y.h[i] = pack16<DT>(keep_range(y0), keep_range(y1));
        }
        store32(dst, c, run, D, x.h);
        store32(dst, c + D / 2, run, D, y.h);
      }
    } else {
      constexpr int R = D / 64;  // runs of half a row
      for (int e = warp * 32 + lane; e < PIECE * R; e += THREADS) {
        const int run = (e >> 3) % R, t = a0 + ((e & 7) | ((e / (8 * R)) << 3)), row = t - tt.t0;
        if (t < (tt.v0 & ~31) || t >= ((tt.v1 + 31) & ~31)) continue;
        Loose x, y;
        loose_token(t, run, x);
        loose_token(t, run + R, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 k0 = cos_sin((uint64_t)t * a.turns[32 * run + 2 * i]);
          const float2 k1 = cos_sin((uint64_t)t * a.turns[32 * run + 2 * i + 1]);
          const float2 xa = x.value(i), ya = y.value(i);
          x.h[i] = pack16<DT>(keep_range(xa.x * k0.x - ya.x * k0.y), keep_range(xa.y * k1.x - ya.y * k1.y));
          y.h[i] = pack16<DT>(keep_range(ya.x * k0.x + xa.x * k0.y), keep_range(ya.y * k1.x + xa.y * k1.y));
        }
        store32(dst, row, run, NT, x.h);
        store32(dst, row, run + R, NT, y.h);
      }
    }
  }

  // Window tokens of a rotated format, turned into the rotated domain: a warp per token.
  __device__ void rotated_window(const TileTokens& tt) const {
    const int t1 = min(min(u.T, a0 + PIECE), (tt.v1 + 31) & ~31);
    for (int t = max(max(qe, a0), tt.v0 & ~31) + warp; t < t1; t += kChunkDequantWarps) {
      const uint2* p = reinterpret_cast<const uint2*>(resid_row(a.lo, a.cp, which, u.layer, u.b, u.h, t));
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const uint2 w = p[32 * c + lane];
        const uint32_t w0 = clean(w.x), w1 = clean(w.y);
        float v[4] = {in_to_f32((uint16_t)w0, DT), in_to_f32((uint16_t)(w0 >> 16), DT), in_to_f32((uint16_t)w1, DT),
                      in_to_f32((uint16_t)(w1 >> 16), DT)};
        warp_rotate128(v, a.lo.d1, a.lo.d2);
        const int ch = 128 * c + 4 * lane;
        const uint32_t at = dst + (uint32_t)(ch >> 6) * NT * 128 + swz(t - tt.t0, (ch & 63) >> 3) + (ch & 4) * 2;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at),
                     "r"(pack16<DT>(keep_range(v[0]), keep_range(v[1]))), "r"(pack16<DT>(keep_range(v[2]), keep_range(v[3])))
                     : "memory");
      }
    }
  }

  __device__ void piece(const TileTokens& tt) const {
    const bool per_channel = fmt_main(a.lo, which).axis == KVQ_AXIS_CHANNEL;
    if (turned()) {
      turned_tile(tt, per_channel);
      return;
    }
    const int e = warp * 32 + lane;
    uint32_t h[16];
    if (per_channel) {
      constexpr int G = PIECE / 32;
      const int c = (e & 7) | ((e / (8 * G)) << 3), t = a0 + 32 * ((e >> 3) % G);
      if (t + 32 <= tt.v0 || t >= tt.v1) return;
      channel_run(t, c, h);
      store32(dst, c, (t - tt.t0) >> 5, D, h);
      return;
    }
    constexpr int R = D / 32;
    const bool rotated = (a.lo.flags & (which ? KVQ_ROTATE_V : KVQ_ROTATE_K)) != 0;
    const int run = (e >> 3) % R, t = a0 + ((e & 7) | ((e / (8 * R)) << 3));
    if (t >= (tt.v0 & ~31) && t < ((tt.v1 + 31) & ~31) && !(rotated && t >= qe && t < u.T)) {
      token_run(t, run, h);
      store32(dst, t - tt.t0, run, NT, h);
    }
    if (rotated) rotated_window(tt);
  }
};

// ---- staging -----------------------------------------------------------------------------

// The loader warp: the packed bytes of every piece into a ring of
// shared-memory slots, as bulk copies of 32-token subtiles (of pages, when those are smaller).
template <int D>
struct Loader {
  static constexpr int NT = chunk_tile(D), PIECE = NT / 2, SUBS = PIECE / 32;

  const ChunkArgs& a;
  int lane;

  // page id of the lane-th page of the tile (small pages)
  __device__ __forceinline__ int page_id(const Unit& u, const TileTokens& tt, int qe) const {
    const int t = tt.t0 + (lane << a.copy_shift);
    if (!a.small_pages || lane >= (NT >> a.copy_shift) || t >= qe) return -1;
    return __ldg(a.cp.block_table + (int64_t)u.b * a.lo.max_pages + t / a.lo.pt);
  }

  __device__ __forceinline__ static void copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
  }

  // One piece into the slot at `dst`; the slot's barrier completes once the bytes are there.
  __device__ __forceinline__ void piece(const Unit& u, const TileTokens& tt, int which, int half, int qe, int ce, int pid,
                                        uint32_t dst, uint32_t bar, uint32_t* bad_at) const {
    const int a0 = tt.t0 + half * PIECE;
    if (a.direct) {
      piece_direct(u, tt, which, a0, qe, dst, bar, bad_at);
      return;
    }
    const int n = PIECE >> a.copy_shift;  // copies of the piece, one per lane
    const int t = a0 + (lane << a.copy_shift), sub = t & ~31;
    bool active = lane < n && t < qe && sub + 32 > tt.v0 && sub < tt.v1, bad = false;
    const bool cold = t < ce;
    const FmtInfo& f = cold ? fmt_cold(a.lo, which) : fmt_main(a.lo, which);
    const uint8_t* src = nullptr;
    int p = 0;
    if (a.small_pages) p = __shfl_sync(0xffffffffu, pid, (lane + half * n) & 31);
    if (active) {
      if (a.small_pages) {
        bad = p < 0 || p >= a.lo.n_pages;
        const uint8_t* base = which ? a.cp.v_main : a.cp.k_main;
        src = base + (((int64_t)u.layer * a.lo.n_pages + p) * a.lo.H + u.h) * a.lo.pt * f.row;
      } else {
        src = cold ? cold_row(a.lo, a.cp, which, u.layer, u.b, u.h, t)
                   : main_row(a.lo, a.cp, which, u.layer, u.b, u.h, t, &bad);
      }
    }
    const uint32_t bytes = f.axis == KVQ_AXIS_CHANNEL ? f.row : f.row << a.copy_shift;
    active = active && !bad && span_ok(a.lo, a.cp, which + (cold ? 2 : 0), src, bytes);
    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
    const uint32_t total = __reduce_add_sync(0xffffffffu, active ? bytes : 0u);
    if (lane == 0) {
      *bad_at = bads;
      if (bads) atomicOr(a.status, KVQ_DEV_PAGE);
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(total) : "memory");
    }
    __syncwarp();
    if (active) copy(dst + ((t - a0) >> 5) * a.sub_bytes + (t & 31) * f.row, src, bytes, bar);
  }

  // Pages whose rows are no whole 16-byte words, or do not divide a subtile: 2 bytes at a time.
  __device__ __noinline__ void piece_direct(const Unit& u, const TileTokens& tt, int which, int a0, int qe, uint32_t dst,
                                            uint32_t bar, uint32_t* bad_at) const {
    const FmtInfo& f = fmt_main(a.lo, which);
    for (int i = 0; i < PIECE; ++i) {
      const int t = a0 + i;
      if (t >= qe || (t & ~31) + 32 <= tt.v0 || (t & ~31) >= tt.v1) continue;
      bool bad = false;
      const uint8_t* src = main_row(a.lo, a.cp, which, u.layer, u.b, u.h, t, &bad);
      const uint32_t to = dst + (i >> 5) * a.sub_bytes + (t & 31) * f.row;
      for (int e = 2 * lane; e < f.row; e += 64) {
        // a page out of range reads as blocks of scale 0 (and zero 0)
        const uint16_t v = bad ? (uint16_t)0 : *reinterpret_cast<const uint16_t*>(src + e);
        asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(to + e), "h"(v) : "memory");
      }
      if (bad && lane == 0) atomicOr(a.status, KVQ_DEV_PAGE);
    }
    __syncwarp();
    if (lane == 0) {
      *bad_at = 0;
      bar_arrive(bar);
    }
  }
};

// ---- the kernel ----------------------------------------------------------------------

template <int D, bool PAIRED>
struct ChunkShape {
  static constexpr int NT = chunk_tile(D);
  static constexpr int STREAMS = chunk_streams(D);
  static constexpr int QTILES = PAIRED ? 2 : 1;
  static constexpr int RT = 128 * QTILES;  // rows of a row tile
  static constexpr int SOFT_WARPS = 4 * STREAMS;
  static constexpr int WARPS = SOFT_WARPS + kChunkDequantWarps + 2;  // and the loader and product warps
  static constexpr int THREADS = 32 * WARPS;
  static constexpr uint32_t Q_BYTES = 128u * D * 2;
  static constexpr uint32_t TILE_BYTES = (uint32_t)NT * D * 2;  // 32 KiB
  static constexpr uint32_t FIXED = 1024 + QTILES * Q_BYTES + 4 * TILE_BYTES;  // the rest of the SM's is staging
  static constexpr uint32_t S_COL = 0, O_COL = D == 128 ? 256 : 256;
};

struct ChunkShared {
  uint64_t raw_full[kChunkMaxSlots], raw_empty[kChunkMaxSlots];
  uint32_t bad_pages[kChunkMaxSlots];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], s_full[2], p_full[2], o_full, pv_done, soft;
  uint32_t tmem;
  uint32_t gave_up;
  uint32_t nonfinite;
  uint32_t last;  // this CTA joins the unit's partials
  LineStart start;
  int64_t scan[32];
  uint32_t pair_table[256];  // TBQ4: centroids of a byte's two indices
};

// Sum over the block's threads of x, and the exclusive prefix.
template <int THREADS>
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* scan, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = y;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t s = scan[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + y - x;
}

// Finds this CTA's stretch of the line of tiles and the unit it starts in.
template <int D, int RT, int THREADS>
__device__ __forceinline__ void find_start(const ChunkArgs& a, ChunkShared& sh) {
  const int lane = a.by_warp ? threadIdx.x & 31 : 0, lanes = a.by_warp ? 32 : 1;
  const int group = threadIdx.x / lanes, groups = THREADS / lanes;
  const int64_t lh = (int64_t)a.n_layers * a.lo.H;
  bool bad = false;
  int64_t line = 0;
  for (int b0 = 0; b0 < a.lo.B; b0 += groups) {
    const int b = b0 + group;
    const int64_t mine = b < a.lo.B ? seq_tiles<D, RT>(a, b, lane, lanes, &bad) : 0;
    int64_t sum;
    (void)block_sum<THREADS>(mine, sh.scan, &sum);
    line += sum;
  }
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0 && __ldg(a.cu_q) != 0) bad = true;
    if (bad) atomicOr(a.status, KVQ_DEV_LENGTH);
  }
  const int64_t all = line * lh;
  // at least two tiles a run: joining costs about as much
  const int64_t per = max((all + gridDim.x - 1) / (int64_t)gridDim.x, (int64_t)2);
  const int64_t begin = min(all, per * blockIdx.x), end = min(all, begin + per);
  if (threadIdx.x == 0) {
    sh.start.begin = begin;
    sh.start.end = end;
    sh.start.per_cta = per;
  }
  if (begin >= end) return;
  const int64_t x = begin % line;  // place within one (layer, kv head)
  int64_t base = 0;
  for (int b0 = 0; b0 < a.lo.B && base <= x; b0 += groups) {
    const int b = b0 + group;
    bool ignore = false;
    int64_t mine = b < a.lo.B ? seq_tiles<D, RT>(a, b, lane, lanes, &ignore) : 0;
    int64_t sum, at = block_sum<THREADS>(mine, sh.scan, &sum);
    if (a.by_warp) {  // the sequence's tiles, seen from lane 0
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    }
    at += base;
    if (lane == 0 && b < a.lo.B && x >= at && x < at + mine) {
      Unit u;
      (void)valid_seq(a, b, &u.n, &u.T, &u.cu);
      int64_t left = x - at;
      u.rt = 0;
      for (;;) {
        unit_tiles<D, RT>(a, u);
        if (left < u.nt) break;
        left -= u.nt;
        ++u.rt;
      }
      sh.start.lh = (int)(begin / line);
      sh.start.b = b;
      sh.start.rt = u.rt;
      sh.start.tile = (int)left;
    }
    base += sum;
  }
}

// V's values that are not finite were left out of the products: every row
// that sees such a window token gets the value itself (an infinity stays one
// under any positive weight, a NaN stays NaN).  Row of query position p, 4 channels of a lane.
template <int DT>
__device__ __noinline__ void add_nonfinite(const ChunkArgs& a, const Unit& u, int p, int ch, float (&o)[4]) {
  const int qe = q_end_of(a.lo, u.T);
  for (int t = qe; t <= p; ++t) {
    if (a.window && t <= p - a.window && t >= a.sinks) continue;
    const uint16_t* v = resid_row(a.lo, a.cp, 1, u.layer, u.b, u.h, t) + ch;
    for (int e = 0; e < 4; ++e) {
      const float x = in_to_f32(v[e], DT);
      if (!(fabsf(x) <= 3.402823466e38f)) o[e] += x;
    }
  }
}

// All softmax warps meet (boundedly, like every wait): false once a warp has given up.
__device__ __forceinline__ bool soft_sync(uint32_t bar, uint32_t& phase, volatile uint32_t* gave_up) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(bar);
  const bool ok = __all_sync(0xffffffffu, bar_wait(bar, phase & 1, gave_up));
  ++phase;
  return ok;
}

// Joins the partial rows of one unit and writes its output rows; all softmax threads.
template <int D, int DT, bool PAIRED>
__device__ void join_unit(const ChunkArgs& a, const Unit& u, const LineStart& line, int64_t unit_pos, bool cut,
                          bool fix, int tid) {
  using C = ChunkShape<D, PAIRED>;
  constexpr int N = D / 128;
  constexpr int64_t PR = chunk_part_row(D), SLOT = (int64_t)chunk_slot_rows(D) * PR;
  const int lane = tid & 31, warp = tid >> 5;
  const int c0 = cut ? (int)(unit_pos / line.per_cta) : blockIdx.x;
  const int c1 = cut ? (int)((unit_pos + u.nt - 1) / line.per_cta) : blockIdx.x;
  const int copies = PAIRED ? 1 : C::STREAMS * a.rep;  // partial rows of one query row in one slot
  const int lanes_per = 128 / a.rep;
  const int parts = (c1 - c0 + 1) * copies;
  auto part = [&](int i, int r) {
    const int c = c0 + i / copies, k = i % copies;
    const int slot = !cut ? 2 : c > c0 || unit_pos == (int64_t)c * line.per_cta ? 0 : 1;
    const int row = PAIRED ? r : (k / a.rep) * 128 + (k % a.rep) * lanes_per + r;
    return a.partials + ((int64_t)c * kChunkSlots + slot) * SLOT + row * PR;
  };
  for (int r = warp; r < u.rows; r += C::SOFT_WARPS) {
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(part(i, r) + D));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, acc[N][4];
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
    for (int i0 = 0; i0 < parts; i0 += 32) {
      float w = 0.f;
      if (i0 + lane < parts) {
        const float* p = part(i0 + lane, r) + D;
        const float m = __ldcg(p), l = __ldcg(p + 1);
        // a part that saw none of the row's tokens has m = -inf and l = 0
        w = m == -INFINITY && l == 0.f ? 0.f : ex2(m - M);
        L += w == 0.f && l == 0.f ? 0.f : w * l;
      }
      const int k1 = min(32, parts - i0);
#pragma unroll 4
      for (int k = 0; k < k1; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (wk == 0.f) continue;
        const float4* o4 = reinterpret_cast<const float4*>(part(i0 + k, r));
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float4 v = __ldcg(o4 + 32 * c + lane);
          acc[c][0] = fmaf(wk, v.x, acc[c][0]);
          acc[c][1] = fmaf(wk, v.y, acc[c][1]);
          acc[c][2] = fmaf(wk, v.z, acc[c][2]);
          acc[c][3] = fmaf(wk, v.w, acc[c][3]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const int row = u.r0 + r, tok = row / a.lo.g, head = u.h * a.lo.g + row % a.lo.g;
    uint16_t* dst = a.out + (((int64_t)(u.layer - a.layer0) * a.total_q + u.cu + tok) * a.lo.Hq + head) * D;
    const float inv = 1.f / L;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      float v[4] = {acc[c][0] * inv, acc[c][1] * inv, acc[c][2] * inv, acc[c][3] * inv};
      if (a.lo.flags & KVQ_ROTATE_V) warp_unrotate128(v, a.lo.d1, a.lo.d2);
      if (fix) add_nonfinite<DT>(a, u, u.T - u.n + tok, 128 * c + 4 * lane, v);
      *reinterpret_cast<uint2*>(dst + 128 * c + 4 * lane) = make_uint2(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]));
    }
  }
}

// In-thread inverse of the 128-point transform on TMEM columns [col, col +
// 128) of this lane, in place: two 64-point halves, then the last stage.
__device__ void unrotate_columns(uint32_t col, const uint32_t* d1, const uint32_t* d2, float factor) {
  uint32_t r0[32], r1[32];
  const float f = factor * hadamard_scale();
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    tmem_ld32(col + 64 * half, r0);
    tmem_ld32(col + 64 * half + 32, r1);
    tmem_wait_ld();
    float x[64];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      x[i] = __uint_as_float(r0[i] ^ (((d2[2 * half] >> i) & 1u) << 31)) * f;
      x[32 + i] = __uint_as_float(r1[i] ^ (((d2[2 * half + 1] >> i) & 1u) << 31)) * f;
    }
#pragma unroll
    for (int h = 1; h < 64; h <<= 1)
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (!(i & h)) {
          const float u = x[i], v = x[i + h];
          x[i] = u + v;
          x[i + h] = u - v;
        }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      r0[i] = __float_as_uint(x[i]);
      r1[i] = __float_as_uint(x[32 + i]);
    }
    tmem_st32(col + 64 * half, r0);
    tmem_st32(col + 64 * half + 32, r1);
    tmem_wait_st();
  }
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    tmem_ld32(col + 32 * c, r0);
    tmem_ld32(col + 64 + 32 * c, r1);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float u = __uint_as_float(r0[i]), v = __uint_as_float(r1[i]);
      r0[i] = __float_as_uint(u + v) ^ (((d1[c] >> i) & 1u) << 31);
      r1[i] = __float_as_uint(u - v) ^ (((d1[2 + c] >> i) & 1u) << 31);
    }
    tmem_st32(col + 32 * c, r0);
    tmem_st32(col + 64 + 32 * c, r1);
    tmem_wait_st();
  }
}

template <int D, int DT, bool PAIRED>
__global__ void __launch_bounds__(ChunkShape<D, PAIRED>::THREADS, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkArgs a) {
  using C = ChunkShape<D, PAIRED>;
  constexpr int NT = C::NT, RT = C::RT;
  extern __shared__ uint8_t raw_smem[];
  __shared__ ChunkShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = smem_addr(smem), k_at = q_at + C::QTILES * C::Q_BYTES, v_at = k_at + 2 * C::TILE_BYTES;
  const uint32_t raw_at = v_at + 2 * C::TILE_BYTES;

  // set-up that needs nothing of the stream's earlier work
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sh.k_full[i]), kChunkDequantWarps);
      bar_init(smem_addr(&sh.v_full[i]), kChunkDequantWarps);
      bar_init(smem_addr(&sh.k_empty[i]), 1);
      bar_init(smem_addr(&sh.v_empty[i]), 1);
      bar_init(smem_addr(&sh.q_full[i]), 4);
      bar_init(smem_addr(&sh.s_full[i]), 1);
      bar_init(smem_addr(&sh.p_full[i]), 4);
    }
    for (int i = 0; i < a.slots; ++i) {
      bar_init(smem_addr(&sh.raw_full[i]), 1);
      bar_init(smem_addr(&sh.raw_empty[i]), kChunkDequantWarps);
    }
    bar_init(smem_addr(&sh.o_full), 1);
    bar_init(smem_addr(&sh.pv_done), 1);
    bar_init(smem_addr(&sh.soft), C::SOFT_WARPS);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    sh.gave_up = 0;
    sh.nonfinite = 0;
  }
  if (warp == C::WARPS - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  // V tiles and queries start as zeros: rows that are never written must not
  // hold infinities or NaN (a zero probability times one is NaN)
  for (uint32_t e = tid * 16; e < C::QTILES * C::Q_BYTES; e += C::THREADS * 16)
    *reinterpret_cast<uint4*>(smem + e) = make_uint4(0, 0, 0, 0);
  for (uint32_t e = tid * 16; e < 2 * C::TILE_BYTES; e += C::THREADS * 16)
    *reinterpret_cast<uint4*>(smem + C::QTILES * C::Q_BYTES + 2 * C::TILE_BYTES + e) = make_uint4(0, 0, 0, 0);
  if (a.lo.flags & (KVQ_TBQ4_K | KVQ_TBQ4_V))
    for (int i = tid; i < 256; i += C::THREADS) {
      const __half2 p = __floats2half2_rn(a.lo.cb[i & 15], a.lo.cb[i >> 4]);
      sh.pair_table[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  grid_launch_dependents();
  grid_dependency_wait();
  find_start<D, RT, C::THREADS>(a, sh);
  proxy_fence();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const LineStart line = sh.start;
  const bool k_chan = a.lo.kf.axis == KVQ_AXIS_CHANNEL, v_chan = a.lo.vf.axis == KVQ_AXIS_CHANNEL;
  Run run;
  bool more = first_run<D, RT>(a, line, run);

  if (warp == C::WARPS - 1) {
    // ---- products: one thread ----------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t F = DT == KVQ_DT_F16 ? 0 : 1;
      constexpr uint32_t base = (1u << 4) | (F << 7) | (F << 10) | ((128u >> 4) << 24);
      const uint32_t qk_desc = base | ((uint32_t)k_chan << 16) | ((uint32_t)(NT >> 3) << 17);
      const uint32_t pv_desc = base | ((uint32_t)!v_chan << 16) | ((uint32_t)(D >> 3) << 17);
      uint32_t kt = 0;             // tiles of this CTA so far
      uint32_t np[2] = {0, 0};     // steps of each S buffer so far
      uint32_t runs = 0;
      bool ok = true;
      for (; more && ok; more = next_run<D, RT>(a, line, run), ++runs) {
        const int tiles = run.t1 - run.t0, steps = PAIRED ? 2 * tiles : tiles;
        auto tile_of = [&](int s) { return kt + (PAIRED ? s >> 1 : s); };
        auto qk = [&](int s) {
          const uint32_t t = tile_of(s), st = t & 1;
          if (s < C::QTILES) ok = ok && bar_wait(smem_addr(&sh.q_full[s]), runs & 1, &sh.gave_up);
          ok = ok && bar_wait(smem_addr(&sh.k_full[st]), (t >> 1) & 1, &sh.gave_up);
          if (!ok) return;
          tc_fence_after();
          const uint32_t q0 = q_at + (PAIRED ? (s & 1) * C::Q_BYTES : 0), k0 = k_at + st * C::TILE_BYTES;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t da = operand_desc(q0 + (k >> 2) * 16384 + (k & 3) * 32, 0, 1024);
            const uint64_t db = k_chan ? operand_desc(k0 + k * 2048, D * 128, 1024)
                                       : operand_desc(k0 + (k >> 2) * (NT * 128) + (k & 3) * 32, 0, 1024);
            mma_ss(tmem + C::S_COL + (s & 1) * NT, da, db, qk_desc, k > 0);
          }
          tc_commit(smem_addr(&sh.s_full[s & 1]));
          if (!PAIRED || (s & 1)) tc_commit(smem_addr(&sh.k_empty[st]));
        };
        auto pv = [&](int s) {
          const uint32_t t = tile_of(s), st = t & 1;
          ok = ok && bar_wait(smem_addr(&sh.p_full[s & 1]), np[s & 1] & 1, &sh.gave_up);
          ++np[s & 1];
          ok = ok && bar_wait(smem_addr(&sh.v_full[st]), (t >> 1) & 1, &sh.gave_up);
          if (!ok) return;
          tc_fence_after();
          const uint32_t v0 = v_at + st * C::TILE_BYTES;
          const uint32_t o = tmem + C::O_COL + (C::STREAMS == 2 ? (s & 1) * D : 0);
          const bool fresh = C::STREAMS == 2 ? s < 2 : s == 0;
#pragma unroll
          for (int k = 0; k < NT / 16; ++k) {
            const uint64_t db = v_chan ? operand_desc(v0 + (k >> 2) * (D * 128) + (k & 3) * 32, 0, 1024)
                                       : operand_desc(v0 + k * 2048, NT * 128, 1024);
            mma_ts(o, tmem + C::S_COL + (s & 1) * NT + k * 8, db, pv_desc, !fresh || k > 0);
          }
          if (C::STREAMS == 1) tc_commit(smem_addr(&sh.pv_done));
          if (!PAIRED || (s & 1)) tc_commit(smem_addr(&sh.v_empty[st]));
        };
        qk(0);
        if (steps > 1) qk(1);
        for (int s = 0; s < steps && ok; ++s) {
          pv(s);
          if (s + 2 < steps && ok) qk(s + 2);
        }
        if (ok) tc_commit(smem_addr(&sh.o_full));
        kt += tiles;
      }
    }
    __syncwarp();
  } else if (warp >= C::SOFT_WARPS && warp < C::WARPS - 2) {
    // ---- dequantization ---------------------------------------------------------------
    const int dw = warp - C::SOFT_WARPS;
    uint32_t kt = 0, slot = 0, lap = 0;
    bool ok = true;
    for (; more && ok; more = next_run<D, RT>(a, line, run)) {
      const Unit& u = run.u;
      const int qe = q_end_of(a.lo, u.T), ce = c_end_of(a.lo, u.T);
      Unit in_cache = u;
      in_cache.layer += a.layer0;
      for (int j = run.t0; j < run.t1 && ok; ++j, ++kt) {
        const uint32_t st = kt & 1, par = ((kt >> 1) & 1) ^ 1;
        const TileTokens tt = tile_tokens<D>(u, j);
#pragma unroll 1
        for (int which = 0; which < 2 && ok; ++which) {
          ok = __all_sync(0xffffffffu, bar_wait(smem_addr(which ? &sh.v_empty[st] : &sh.k_empty[st]), par, &sh.gave_up));
#pragma unroll 1
          for (int half = 0; half < 2 && ok; ++half) {
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.raw_full[slot]), lap & 1, &sh.gave_up));
            if (!ok) break;
            const Dequant<D, DT> dq{a, in_cache, which, dw, lane, (which ? v_at : k_at) + st * C::TILE_BYTES, qe, ce,
                                    sh.pair_table, &sh.nonfinite, tt.t0 + half * (NT / 2),
                                    raw_at + slot * a.slot_bytes, *(volatile uint32_t*)&sh.bad_pages[slot]};
            dq.piece(tt);
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&sh.raw_empty[slot]));
            if (++slot == (uint32_t)a.slots) {
              slot = 0;
              ++lap;
            }
          }
          proxy_fence();
          __syncwarp();
          if (ok && lane == 0) bar_arrive(smem_addr(which ? &sh.v_full[st] : &sh.k_full[st]));
        }
      }
    }
  } else if (warp == C::WARPS - 2) {
    // ---- staging ------------------------------------------------------------------------
    const Loader<D> ld{a, lane};
    uint32_t slot = 0, lap = 0, filled = 0;
    bool ok = true;
    for (; more && ok; more = next_run<D, RT>(a, line, run)) {
      Unit u = run.u;
      u.layer += a.layer0;
      const int qe = q_end_of(a.lo, u.T), ce = c_end_of(a.lo, u.T);
      int pid = ld.page_id(u, tile_tokens<D>(u, run.t0), qe);
      for (int j = run.t0; j < run.t1 && ok; ++j) {
        const TileTokens tt = tile_tokens<D>(u, j);
        // the next tile's page ids load while this one waits for slots
        const int next_pid = j + 1 < run.t1 ? ld.page_id(u, tile_tokens<D>(u, j + 1), qe) : -1;
#pragma unroll 1
        for (int i = 0; i < 4 && ok; ++i) {
          ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sh.raw_empty[slot]), (lap & 1) ^ 1, &sh.gave_up));
          if (!ok) break;
          ld.piece(u, tt, i >> 1, i & 1, qe, ce, pid, raw_at + slot * a.slot_bytes, smem_addr(&sh.raw_full[slot]),
                   &sh.bad_pages[slot]);
          ++filled;
          if (++slot == (uint32_t)a.slots) {
            slot = 0;
            ++lap;
          }
        }
        pid = next_pid;
      }
    }
    // the copies in flight land before the CTA ends, also when another warp has given up
    for (uint32_t i = 0; i < (uint32_t)a.slots && i < filled; ++i) {
      const uint32_t back = filled - 1 - i, s = back % a.slots, n = back / a.slots;
      for (int k = 0; k < kChunkSpin && !bar_test(smem_addr(&sh.raw_full[s]), n & 1); ++k) {
      }
    }
  } else {
    // ---- softmax and outputs -----------------------------------------------------------
    const int stream = warp >> 2, quad = warp & 3;
    const int my_lane = quad * 32 + lane;  // TMEM lane: row of the 128-row tile
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const int lanes_per = 128 / a.rep;
    const int cols = NT / a.rep, col0 = (my_lane / lanes_per) * cols;  // this row's tokens of a tile
    const float sc = 1.4426950408889634f * rsqrtf((float)D);
    uint32_t ns[2] = {0, 0}, runs = 0, steps_done = 0, syncs = 0;
    bool ok = true;
    for (; more && ok; more = next_run<D, RT>(a, line, run), ++runs) {
      const Unit& u = run.u;
      const int tiles = run.t1 - run.t0, steps = PAIRED ? 2 * tiles : tiles;
      // queries: row r of this stream's tile (each repetition a copy)
      if (PAIRED || stream == 0) {
        const int first = PAIRED ? stream * 128 : 0;
        const int n = min(a.rep > 1 ? lanes_per : 128, u.rows - first);
        const uint32_t q0 = q_at + (PAIRED ? stream * C::Q_BYTES : 0);
        for (int r = quad; r < n; r += 4) {
          const int row = u.r0 + first + r, tok = row / a.lo.g, head = u.h * a.lo.g + row % a.lo.g;
          const uint16_t* src = a.q + (((int64_t)u.layer * a.total_q + u.cu + tok) * a.lo.Hq + head) * D;
#pragma unroll
          for (int c = 0; c < D / 128; ++c) {
            uint2 w = __ldg(reinterpret_cast<const uint2*>(src) + 32 * c + lane);
            if (a.lo.flags & KVQ_ROTATE_K) {
              float v[4] = {in_to_f32((uint16_t)w.x, DT), in_to_f32((uint16_t)(w.x >> 16), DT),
                            in_to_f32((uint16_t)w.y, DT), in_to_f32((uint16_t)(w.y >> 16), DT)};
              warp_rotate128(v, a.lo.d1, a.lo.d2);
              w = make_uint2(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]));
            }
            const int ch = 128 * c + 4 * lane;
            for (int k = 0; k < a.rep; ++k) {
              const uint32_t at = q0 + (uint32_t)(ch >> 6) * 16384 + swz(r + k * lanes_per, (ch & 63) >> 3) + (ch & 4) * 2;
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(at), "r"(w.x), "r"(w.y) : "memory");
            }
          }
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.q_full[PAIRED ? stream : 0]));
      }
      const int my_row = (PAIRED ? stream * 128 : 0) + my_lane % lanes_per;  // query row of the row tile
      const int pos = u.T - u.n + (u.r0 + my_row) / a.lo.g;
      const int win_lo = a.window ? max(0, pos - a.window + 1) : 0;  // visible: [win_lo, pos] and [0, sinks)
      float m = -INFINITY, l = 0.f;
      int first_step = 1;
      for (int s = C::STREAMS == 2 ? stream : 0; s < steps && ok; s += C::STREAMS) {
        const int b = s & 1;
        ok = bar_wait(smem_addr(&sh.s_full[b]), ns[b] & 1, &sh.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++ns[b];
        tc_fence_after();
        const int j = run.t0 + (PAIRED ? s >> 1 : s);
        const int t0 = (j < u.st ? j : u.lo_tile + (j - u.st)) * NT;
        const bool masked = t0 + NT - 1 > u.p_lo || (a.window && t0 <= u.p_hi - a.window && t0 + NT > a.sinks);
        const uint32_t s_col = lane_base + C::S_COL + b * NT;
        uint32_t x[32];
        auto mask32 = [&](int c) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int t = t0 + c + i;
            if (t > pos || (t < win_lo && t >= a.sinks)) x[i] = 0xff800000u;
          }
        };
        float mt = -INFINITY;
        for (int c = col0; c < col0 + cols; c += 32) {
          tmem_ld32(s_col + c, x);
          tmem_wait_ld();
          if (masked) mask32(c);
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            m0 = fmaxf(m0, __uint_as_float(x[i]));
            m1 = fmaxf(m1, __uint_as_float(x[i + 1]));
          }
          mt = fmaxf(mt, fmaxf(m0, m1));
        }
        mt *= sc;
        // the reference maximum follows only when it falls behind by 2^8: P
        // stays below 2^8 and the accumulator is rescaled rarely
        const bool grow = mt > m + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
          const float nm = grow ? mt : m;
          const float f = m == -INFINITY ? 0.f : ex2(m - nm);
          l = l == 0.f ? 0.f : l * f;
          if (!first_step) {
            if (C::STREAMS == 1) {
              // the products of the step before must have left the accumulator
              ok = bar_wait(smem_addr(&sh.pv_done), (steps_done - 1) & 1, &sh.gave_up);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t o_col = lane_base + C::O_COL + (C::STREAMS == 2 ? stream * D : 0);
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
          m = nm;
        }
        first_step = 0;
        const float mneg = m == -INFINITY ? 0.f : -m;
        float l0 = 0.f, l1 = 0.f;
        for (int c = col0; c < col0 + cols; c += 32) {
          tmem_ld32(s_col + c, x);
          tmem_wait_ld();
          if (masked) mask32(c);
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float e0 = ex2(fmaf(__uint_as_float(x[2 * i]), sc, mneg));
            const float e1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), sc, mneg));
            l0 += e0;
            l1 += e1;
            p[i] = pack16<DT>(e0, e1);
          }
          tmem_st16(s_col + c / 2, p);
        }
        l += l0 + l1;
        if (a.rep > 1) {  // the other repetitions' tokens count nothing in this row
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0;
          for (int c = 0; c < NT; c += 32)
            if (c < col0 || c >= col0 + cols) tmem_st16(s_col + c / 2, z);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sh.p_full[b]));
        ++steps_done;
      }
      // ---- the run's outputs -----------------------------------------------------------
      if (!ok) break;
      ok = bar_wait(smem_addr(&sh.o_full), runs & 1, &sh.gave_up);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool cut = run.t0 > 0 || run.t1 < u.nt;
      const uint32_t o_col = lane_base + C::O_COL + (C::STREAMS == 2 ? stream * D : 0);
      Unit in_cache = u;
      in_cache.layer += a.layer0;
      const bool direct = !cut && (PAIRED || (C::STREAMS == 1 && a.rep == 1));
      if (direct) {
        const bool mine = my_row < u.rows;
        const float inv = 1.f / l;
        if (a.lo.flags & KVQ_ROTATE_V) {
#pragma unroll 1
          for (int c = 0; c < D; c += 128) unrotate_columns(o_col + c, a.lo.d1, a.lo.d2, inv);
        }
        const int row = u.r0 + my_row, tok = row / a.lo.g, head = u.h * a.lo.g + row % a.lo.g;
        uint16_t* dst = a.out + (((int64_t)u.layer * a.total_q + u.cu + tok) * a.lo.Hq + head) * D;
        const float f = a.lo.flags & KVQ_ROTATE_V ? 1.f : inv;
        const bool fix = *(volatile uint32_t*)&sh.nonfinite != 0;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          tmem_ld32(o_col + c, x);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(x[i + e]) * f;
            if (fix) {
              float v0[4] = {v[0], v[1], v[2], v[3]}, v1[4] = {v[4], v[5], v[6], v[7]};
              add_nonfinite<DT>(a, in_cache, pos, c + i, v0);
              add_nonfinite<DT>(a, in_cache, pos, c + i + 4, v1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = v0[e];
                v[4 + e] = v1[e];
              }
            }
            *reinterpret_cast<uint4*>(dst + c + i) =
                make_uint4(pack16<DT>(v[0], v[1]), pack16<DT>(v[2], v[3]), pack16<DT>(v[4], v[5]), pack16<DT>(v[6], v[7]));
          }
          }
          __syncwarp();
        }
        tc_fence_before();
      } else {
        const int64_t unit_pos = run.pos - run.t0;
        // a unit's ticket belongs to its first CTA: entry 0 when the unit
        // starts with that CTA's stretch, else 1
        const int c0 = (int)(unit_pos / line.per_cta);
        const int slot = !cut ? 2 : run.first ? 0 : 1;
        float* part = a.partials + (((int64_t)blockIdx.x * kChunkSlots + slot) * chunk_slot_rows(D) + stream * 128 + my_lane) *
                                       chunk_part_row(D);
        const bool mine = my_row < u.rows;
        // a stream without a step of this run has no accumulator
        const bool none = C::STREAMS == 2 && stream >= steps;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          tmem_ld32(o_col + c, x);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(part + c + i) =
                  none ? make_uint4(0, 0, 0, 0) : make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
          __syncwarp();
        }
        if (mine) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
        tc_fence_before();
        const int64_t tick = (int64_t)c0 * kChunkTickets + (unit_pos == (int64_t)c0 * line.per_cta ? 0 : 1);
        const uint32_t soft = smem_addr(&sh.soft);
        if (cut) {
          __threadfence();
          if (!(ok = soft_sync(soft, syncs, &sh.gave_up))) break;
          if (tid == 0) {
            if (*(volatile uint32_t*)&sh.nonfinite) atomicOr(a.nonfinite + tick, 1u);
            __threadfence();
            const int c1 = (int)((unit_pos + u.nt - 1) / line.per_cta);
            sh.last = atomicAdd(a.tickets + tick, 1u) == (uint32_t)(c1 - c0);
          }
          if (!(ok = soft_sync(soft, syncs, &sh.gave_up))) break;
          if (*(volatile uint32_t*)&sh.last) {
            __threadfence();
            const bool fix = __ldcg(a.nonfinite + tick) != 0;
            join_unit<D, DT, PAIRED>(a, in_cache, line, unit_pos, true, fix, tid);
            if (!(ok = soft_sync(soft, syncs, &sh.gave_up))) break;
            if (tid == 0) {
              a.tickets[tick] = 0;
              a.nonfinite[tick] = 0;
            }
          }
        } else {
          if (!(ok = soft_sync(soft, syncs, &sh.gave_up))) break;
          join_unit<D, DT, PAIRED>(a, in_cache, line, unit_pos, false, *(volatile uint32_t*)&sh.nonfinite != 0, tid);
        }
        if (!(ok = soft_sync(soft, syncs, &sh.gave_up))) break;
      }
    }
  }
  // every role ends here, also after a wait that gave up
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.gave_up) atomicOr(a.status, KVQ_DEV_STALL);
  if (warp == C::WARPS - 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

template <int D, int DT, bool PAIRED>
cudaError_t launch_chunk(ChunkArgs a, int grid, cudaStream_t s) {
  using C = ChunkShape<D, PAIRED>;
  // all of the SM's shared memory that the tiles leave is staging
  const uint32_t all = 227 * 1024 - (uint32_t)sizeof(ChunkShared);
  const uint32_t left = all - C::FIXED - 16;
  a.slots = (int)(left / a.slot_bytes);
  if (a.slots > kChunkMaxSlots) a.slots = kChunkMaxSlots;
  if (a.slots < 1) return cudaErrorInvalidConfiguration;
  const uint32_t smem = C::FIXED + 16 + a.slots * a.slot_bytes;
  // set on every call: the attribute belongs to the current device
  cudaError_t e = cudaFuncSetAttribute(chunk_attention_kernel<D, DT, PAIRED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_attention_kernel<D, DT, PAIRED>, dim3(grid), dim3(C::THREADS), smem, s, a);
}

}  // namespace
}  // namespace kvq
