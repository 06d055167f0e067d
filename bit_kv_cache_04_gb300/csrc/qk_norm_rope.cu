// kvq_qk_norm_rope: RMS norm of every query and key head and the rotary turn
// of its channel pairs, in one pass over the projection's output.
//
// Bound by HBM: 2 bytes in and 2 bytes out per value, and a few fp32
// operations.  A row (one token's head) belongs to D / 8 lanes of 8 channels
// (one 16-byte load and store each), so the mean square is a shuffle sum and
// the partner of a half-split pair sits in another lane of the same row.  A
// warp works out a token's cosines and sines once, in registers, for all the heads it takes.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "kvq_host.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

enum TurnMode { kTurnInterleaved = 0, kTurnHalf8 = 1, kTurnHalfAny = 2 };

struct NormRopeArgs {
  const uint16_t* x[2];  // queries, keys (nullptr: left out)
  uint16_t* y[2];
  const uint16_t* w[2];
  int64_t st[2], sh[2];  // strides between tokens and heads, in elements
  int heads[2];
  int vec[2];            // 16-byte loads and stores fit
  int w_vec[2];
  const int32_t* positions;
  int n_tokens, shares, rows_per_share;  // warps of a token, and heads of each
  float eps, scale;
  int rot_dim;
  uint64_t turns[128];
};

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (DT == KVQ_DT_F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == KVQ_DT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (Not with non-coherent loads: a call in place writes what it has read, and the stream's next call may begin before this one ends.)
__device__ __forceinline__ uint4 load8(const uint16_t* p, bool vec) {
  if (vec) return __ldcg(reinterpret_cast<const uint4*>(p));
  uint4 v;
  v.x = p[0] | ((uint32_t)p[1] << 16);
  v.y = p[2] | ((uint32_t)p[3] << 16);
  v.z = p[4] | ((uint32_t)p[5] << 16);
  v.w = p[6] | ((uint32_t)p[7] << 16);
  return v;
}

__device__ __forceinline__ void store8(uint16_t* p, uint4 v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p[2 * j] = (uint16_t)w[j];
    p[2 * j + 1] = (uint16_t)(w[j] >> 16);
  }
}

template <int DT>
__device__ __forceinline__ void to_f32(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = unpack2<DT>(w[j]);
    f[2 * j] = a.x;
    f[2 * j + 1] = a.y;
  }
}

// Where pair i's frequency sits in shared memory: lanes read pairs 8 (or 4)
// apart, which this order puts next to each other.
template <int MODE>
__device__ __forceinline__ int turn_slot(int i) {
  return MODE == kTurnInterleaved ? (i & 3) * 32 + (i >> 2) : (i & 7) * 16 + (i >> 3);
}

// Cosine and sine of a lane's channel pairs at one position: 4 adjacent pairs
// (interleaved), or one for each of its 8 channels (half split).
template <int MODE>
__device__ __forceinline__ void angles(const NormRopeArgs& a, const uint64_t* turns, int64_t pos, int c, float2 (&cs)[8]) {
  const int half = a.rot_dim / 2;
#pragma unroll
  for (int j = 0; j < (MODE == kTurnInterleaved ? 4 : 8); ++j) {
    const int ch = MODE == kTurnInterleaved ? 8 * c + 2 * j : 8 * c + j;
    const int i = MODE == kTurnInterleaved ? 4 * c + j : ch < half ? ch : ch - half;
    cs[j] = make_float2(1.f, 0.f);
    if (ch < a.rot_dim) {
      // the angle in turns as a 64-bit fraction: exact for every position, so
      // only its top 32 bits, as a signed number of half turns, see fp32
      float s, co;
      sincospif((float)(int32_t)((uint64_t)pos * turns[turn_slot<MODE>(i)] >> 32) * 0x1p-31f, &s, &co);
      cs[j] = make_float2(co * a.scale, s * a.scale);
    }
  }
}

// One row in f (this lane's 8 channels from 8c): norm (with the weights w) and turn.
template <int DT, int D, int MODE>
__device__ __forceinline__ void row_result(float (&f)[8], bool norm, uint4 w, float eps, int rot,
                                           const float2 (&cs)[8], float* buf, int c) {
  constexpr int LPR = D / 8;
  if (norm) {  // of the whole warp: its rows are of one tensor
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
    float wf[8];
    to_f32<DT>(w, wf);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * r * wf[j];
  }
  if constexpr (MODE == kTurnInterleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (8 * c + 2 * j < rot) {
        const float x = f[2 * j], y = f[2 * j + 1];
        f[2 * j] = x * cs[j].x - y * cs[j].y;
        f[2 * j + 1] = y * cs[j].x + x * cs[j].y;
      }
    }
  } else {
    const int half = rot / 2;
    float o[8];
    if constexpr (MODE == kTurnHalf8) {
      // rot / 2 is a multiple of 8: the partner channels are another lane's 8
      const int hl = half / 8, src = (threadIdx.x & 31 & ~(LPR - 1)) + (8 * c >= rot ? c : c < hl ? c + hl : c - hl);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, f[j], src);
    } else {
      // any even rot: through the row's buffer in shared memory
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) buf[8 * c + j] = f[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 8 * c + j;
        o[j] = buf[i < half ? i + half : i < rot ? i - half : i];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 8 * c + j;
      if (i < rot) f[j] = i < half ? f[j] * cs[j].x - o[j] * cs[j].y : f[j] * cs[j].x + o[j] * cs[j].y;
    }
  }
}

// A warp per (token, share of its heads): the angles once, in registers, then
// row after row.  8192 tokens of 40 heads of 128, bf16: 47 us, 53 % of the copy rate, bound by issue slots (64 %
// full: 219 instructions for a lane's 8 values); with a block per token and the angles in shared memory 93 us.
// Three blocks an SM and two rows in flight: of eight shapes tried the best on 1777 tokens of 28 heads of 256
// (9.9 us; 128 threads 11.1, four blocks 12.0, one row in flight 11.8).
template <int DT, int D, int MODE>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 2;  // lanes a row, rows a pass, passes a turn (the next turn's loads in flight)
  __shared__ float buf[MODE == kTurnHalfAny ? kThreads / 32 * RPW * D : 1];
  __shared__ uint64_t turns[128];  // a lane's own word of the parameters would be a serialized load, every time
  if (threadIdx.x < 128) turns[turn_slot<MODE>(threadIdx.x)] = a.turns[threadIdx.x];
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  const int64_t tok = w / a.shares;
  if (tok >= a.n_tokens) return;
  const int H = a.heads[0] + a.heads[1];
  const int r0 = (int)(w - tok * a.shares) * a.rows_per_share, r1 = min(H, r0 + a.rows_per_share);
  const int c = lane & (LPR - 1), sub = lane / LPR;
  float2 cs[8];
  bool have = false;
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    // this share's heads of tensor t
    const int h0 = max(0, r0 - (t ? a.heads[0] : 0)), h1 = min(a.heads[t], r1 - (t ? a.heads[0] : 0));
    if (h0 >= h1) continue;
    const uint16_t* src = a.x[t] + tok * a.st[t] + 8 * c;
    uint16_t* dst = a.y[t] + tok * (int64_t)a.heads[t] * D + 8 * c;
    const int64_t sh = a.sh[t];
    const bool vec = a.vec[t] != 0, norm = a.w[t] != nullptr;
    uint4 wt = make_uint4(0, 0, 0, 0);
    if (norm) wt = load8(a.w[t] + 8 * c, a.w_vec[t]);
    auto load = [&](uint4 (&raw)[U], int h) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (h + u * RPW < h1) raw[u] = load8(src + (h + u * RPW) * sh, vec);
      }
    };
    uint4 raw[U], next[U];
    load(raw, h0 + sub);
    if (!have) {  // while the first rows load
      angles<MODE>(a, turns, a.rot_dim ? a.positions[tok] : 0, c, cs);
      have = true;
    }
#pragma unroll 1
    for (int h = h0 + sub; h - sub < h1; h += RPW * U) {
      load(next, h + RPW * U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[8];
        to_f32<DT>(raw[u], f);
        // rows past the end take part in the shuffles only
        row_result<DT, D, MODE>(f, norm, wt, a.eps, a.rot_dim, cs, MODE == kTurnHalfAny ? buf + (warp * RPW + sub) * D : buf, c);
        if (h + u * RPW < h1) {
          uint4 v;
          v.x = pack2<DT>(f[0], f[1]);
          v.y = pack2<DT>(f[2], f[3]);
          v.z = pack2<DT>(f[4], f[5]);
          v.w = pack2<DT>(f[6], f[7]);
          store8(dst + (int64_t)(h + u * RPW) * D, v, vec);
        }
        raw[u] = next[u];
      }
    }
  }
}

}  // namespace

template <int DT, int D>
static cudaError_t launch_mode(const NormRopeArgs& a, int mode, dim3 grid, size_t smem, cudaStream_t s) {
  if (mode == kTurnInterleaved)
    return launch_dependent(norm_rope_kernel<DT, D, kTurnInterleaved>, grid, dim3(kThreads), smem, s, a);
  if (mode == kTurnHalf8) return launch_dependent(norm_rope_kernel<DT, D, kTurnHalf8>, grid, dim3(kThreads), smem, s, a);
  return launch_dependent(norm_rope_kernel<DT, D, kTurnHalfAny>, grid, dim3(kThreads), smem, s, a);
}

}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_rope_plan_init(const kvq_rope_params* p, kvq_rope_plan* plan) {
  if (!p || !plan) return fail(KVQ_ERR_ARG, "params / plan is NULL");
  if (p->reserved != 0) return fail(KVQ_ERR_ARG, "reserved must be 0");
  if (p->D != 128 && p->D != 256) return fail(KVQ_ERR_UNSUPPORTED, "D=%d not in {128,256}", p->D);
  if (p->rot_dim < 2 || p->rot_dim > p->D || p->rot_dim % 2)
    return fail(KVQ_ERR_ARG, "rot_dim=%d not an even number in [2, %d]", p->rot_dim, p->D);
  if (p->interleaved != 0 && p->interleaved != 1) return fail(KVQ_ERR_ARG, "interleaved=%d", p->interleaved);
  if (!(p->theta > 1.0) || !std::isfinite(p->theta)) return fail(KVQ_ERR_ARG, "theta must be finite and > 1");
  if (p->scaling < KVQ_ROPE_NONE || p->scaling > KVQ_ROPE_BANDS) return fail(KVQ_ERR_ARG, "scaling=%d", p->scaling);
  if (!(p->attn_factor >= 0.0) || !std::isfinite(p->attn_factor)) return fail(KVQ_ERR_ARG, "attn_factor");
  if (p->scaling != KVQ_ROPE_NONE && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
    return fail(KVQ_ERR_ARG, "factor must be finite and >= 1");
  const bool bands = p->scaling == KVQ_ROPE_YARN || p->scaling == KVQ_ROPE_BANDS;
  if (bands && (p->original_len < 1 || !(p->low > 0.0) || !(p->high > p->low) || !std::isfinite(p->high)))
    return fail(KVQ_ERR_ARG, "original_len >= 1 and 0 < low < high are needed");
  const double two_pi = 6.283185307179586476925286766559;
  const double d = p->rot_dim, f = p->factor;
  double theta = p->theta, m = p->attn_factor;
  if (p->scaling == KVQ_ROPE_NTK && p->rot_dim > 2) theta *= std::pow(f, d / (d - 2));
  if (!std::isfinite(theta)) return fail(KVQ_ERR_ARG, "theta times the factor's power is not finite");
  double a = 0, z = 0;
  if (p->scaling == KVQ_ROPE_YARN) {
    auto at = [&](double x) { return d * std::log(p->original_len / (x * two_pi)) / (2 * std::log(theta)); };
    a = std::max(0.0, std::floor(at(p->high)));
    z = std::min(d - 1, std::ceil(at(p->low)));
    if (m == 0.0) m = 0.1 * std::log(f) + 1.0;
  }
  if (m == 0.0) m = 1.0;
  std::memset(plan, 0, sizeof(*plan));
  plan->D = p->D;
  plan->rot_dim = p->rot_dim;
  plan->interleaved = p->interleaved;
  plan->scale = (float)m;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    const double plain = std::pow(theta, -2.0 * i / d);
    double w = plain;
    if (p->scaling == KVQ_ROPE_LINEAR) w = plain / f;
    if (p->scaling == KVQ_ROPE_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - a) / std::max(z - a, 0.001)));
      w = r * plain / f + (1 - r) * plain;
    }
    if (p->scaling == KVQ_ROPE_BANDS) {
      const double b = std::min(1.0, std::max(0.0, (p->original_len * plain / two_pi - p->low) / (p->high - p->low)));
      w = b * plain + (1 - b) * plain / f;
    }
    // w <= 1 radian a position, so the fraction stays below 2^62
    plan->turns[i] = (uint64_t)std::ldexp(w / two_pi, 64);
  }
  return ok();
}

kvq_status kvq_qk_norm_rope(const kvq_config* cfg, const kvq_rope_plan* plan, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                            int32_t n_tokens, void* q_out, void* k_out, void* stream) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return fail(KVQ_ERR_ARG, "an input and its output are given together or not at all");
  if (!q && !k) return fail(KVQ_ERR_ARG, "q and k are both NULL");
  if ((!q && q_weight) || (!k && k_weight)) return fail(KVQ_ERR_ARG, "a weight without its tensor");
  if (n_tokens < 0) return fail(KVQ_ERR_ARG, "n_tokens < 0");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(KVQ_ERR_ARG, "eps must be finite and >= 0");
  if (plan) {
    if (plan->D != cfg->D || plan->rot_dim < 2 || plan->rot_dim > cfg->D || plan->rot_dim % 2 || plan->reserved != 0 ||
        (plan->interleaved & ~1))
      return fail(KVQ_ERR_ARG, "the plan is not one of kvq_rope_plan_init for D=%d", cfg->D);
    if (!positions) return fail(KVQ_ERR_ARG, "positions is NULL");
    if (((uintptr_t)positions) & 3u) return fail(KVQ_ERR_ARG, "positions must be 4-byte aligned");
  }
  const uintptr_t any = (uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)q_weight |
                        (uintptr_t)k_weight;
  if (any & 1u) return fail(KVQ_ERR_ARG, "tensors must be aligned to their elements");
  if (q_token_stride < 0 || q_head_stride < 0 || k_token_stride < 0 || k_head_stride < 0)
    return fail(KVQ_ERR_ARG, "negative stride");
  // the stride of a dimension of one element says nothing
  auto contiguous = [&](int64_t token_stride, int64_t head_stride, int64_t heads) {
    return (heads == 1 || head_stride == cfg->D) && (n_tokens <= 1 || token_stride == heads * cfg->D);
  };
  if (q && q == q_out && !contiguous(q_token_stride, q_head_stride, cfg->H_q))
    return fail(KVQ_ERR_ARG, "q in place must be contiguous");
  if (k && k == k_out && !contiguous(k_token_stride, k_head_stride, cfg->H_kv))
    return fail(KVQ_ERR_ARG, "k in place must be contiguous");
  if (n_tokens == 0) return ok();
  NormRopeArgs a{};
  const void* xs[2] = {q, k};
  void* ys[2] = {q_out, k_out};
  const void* ws[2] = {q_weight, k_weight};
  const int64_t sts[2] = {q_token_stride, k_token_stride}, shs[2] = {q_head_stride, k_head_stride};
  const int heads[2] = {cfg->H_q, cfg->H_kv};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = (const uint16_t*)xs[i];
    a.y[i] = (uint16_t*)ys[i];
    a.w[i] = (const uint16_t*)ws[i];
    a.st[i] = sts[i];
    a.sh[i] = shs[i];
    a.heads[i] = xs[i] ? heads[i] : 0;
    a.vec[i] = ((((uintptr_t)xs[i] | (uintptr_t)ys[i]) & 15u) == 0 && ((sts[i] | shs[i]) & 7) == 0) ? 1 : 0;
    a.w_vec[i] = (((uintptr_t)ws[i]) & 15u) == 0 ? 1 : 0;
  }
  a.positions = positions;
  a.n_tokens = n_tokens;
  a.eps = eps;
  int mode = kTurnInterleaved;
  if (plan) {
    a.scale = plan->scale;
    a.rot_dim = plan->rot_dim;
    std::memcpy(a.turns, plan->turns, sizeof(a.turns));
    if (!plan->interleaved) mode = plan->rot_dim % 16 == 0 ? kTurnHalf8 : kTurnHalfAny;
  }
  // Shares of a token's heads: one warp takes them all once every SM has its
  // fill of warps (the angles are worked out once), fewer passes while warps are scarce.
  const int H = a.heads[0] + a.heads[1], rpw = 32 / (cfg->D / 8);
  const int64_t warps = (int64_t)sm_count() * 24;
  int64_t shares = std::max<int64_t>(1, warps / n_tokens);
  shares = std::min<int64_t>(shares, (H + rpw - 1) / rpw);
  a.rows_per_share = (int)(((H + shares - 1) / shares + rpw - 1) / rpw * rpw);
  a.shares = (H + a.rows_per_share - 1) / a.rows_per_share;
  const int64_t blocks = ((int64_t)n_tokens * a.shares + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return fail(KVQ_ERR_UNSUPPORTED, "%d tokens of %d heads", n_tokens, H);
  const dim3 grid((unsigned)blocks);
  const size_t smem = 0;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (cfg->in_dtype == KVQ_DT_F16)
    e = cfg->D == 128 ? launch_mode<KVQ_DT_F16, 128>(a, mode, grid, smem, s) : launch_mode<KVQ_DT_F16, 256>(a, mode, grid, smem, s);
  else
    e = cfg->D == 128 ? launch_mode<KVQ_DT_BF16, 128>(a, mode, grid, smem, s) : launch_mode<KVQ_DT_BF16, 256>(a, mode, grid, smem, s);
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotary kernel");
  return ok();
}

}  // extern "C"
