// kvq_chunk_attention: the last tokens of every sequence attend to the packed
// cache, causally, over a sliding window plus the first tokens.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "block_codec.cuh"
#include "kvq_host.cuh"

namespace kvq {
namespace {

struct ChunkArgs {
  Layout lo;
  CachePtrs cp;
  int layer0, n_layers;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int total_q, max_q, window, sinks;
  uint32_t* status;
  uint64_t turns[128];  // pre-RoPE keys: turns per position of every pair, 64-bit fractions
};

__device__ __forceinline__ float chunk_value(const Layout& lo, const CachePtrs& cp, int which, int layer, int seq,
                                             int h, int t, int qe, int ce, int d, bool* bad) {
  if (t >= qe) return in_to_f32(resid_row(lo, cp, which, layer, seq, h, t)[d], lo.dtype);
  const bool cold = t < ce;
  const FmtInfo& f = cold ? fmt_cold(lo, which) : fmt_main(lo, which);
  const uint8_t* row = cold ? cold_row(lo, cp, which, layer, seq, h, t) : main_row(lo, cp, which, layer, seq, h, t, bad);
  if (!row) return 0.f;
  if (f.axis == KVQ_AXIS_CHANNEL) return block_value(row + (int64_t)d * f.bb, f.bits, 0, f.zp, lo.cb, t % f.group);
  return block_value(row + (int64_t)(d / f.group) * f.bb, f.bits, f.codebook, f.zp, lo.cb, d % f.group);
}

// One warp per (layer, query row): the definition, key by key.
template <int D>
__global__ void chunk_simple_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int N = D / 32;  // channels per lane: 128 c + 4 lane + e
  const Layout& lo = a.lo;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < lo.B; b += blockDim.x) {
      const int n = a.cu_q[b + 1] - a.cu_q[b], T = a.seq_lens[b];
      if (n < 0 || n > a.max_q || T < n || T > lo.max_T || a.cu_q[b] < 0 || a.cu_q[b + 1] > a.total_q)
        atomicOr(a.status, KVQ_DEV_LENGTH);
    }
  if (w >= (int64_t)a.n_layers * a.total_q * lo.Hq) return;
  const int hq = (int)(w % lo.Hq), row = (int)(w / lo.Hq % a.total_q), layer = a.layer0 + (int)(w / lo.Hq / a.total_q);
  if (row >= a.cu_q[lo.B]) return;
  int lob = 0, hib = lo.B;  // the last b with cu_q[b] <= row
  while (hib - lob > 1) {
    const int mid = (lob + hib) / 2;
    if (a.cu_q[mid] <= row)
      lob = mid;
    else
      hib = mid;
  }
  const int b = lob, n = a.cu_q[b + 1] - a.cu_q[b], T = a.seq_lens[b], h = hq / lo.g;
  if (n < 1 || n > a.max_q || T < n || T > lo.max_T || a.cu_q[b] < 0) {
    if (lane == 0) atomicOr(a.status, KVQ_DEV_LENGTH);
    return;
  }
  const int qe = q_end_of(lo, T), ce = c_end_of(lo, T);
  const int p = T - n + row - a.cu_q[b];
  const uint16_t* qp = a.q + w * D;
  float q[N], qr[N], acc[N], accr[N];
  for (int c = 0; c < N; ++c) {
    const int d = 128 * (c / 4) + 4 * lane + c % 4;
    q[c] = qr[c] = in_to_f32(qp[d], lo.dtype);
    acc[c] = accr[c] = 0.f;
  }
  if (lo.flags & KVQ_ROTATE_K)
    for (int c = 0; c < N; c += 4) warp_rotate128(qr + c, lo.d1, lo.d2);
  const float scale = 1.0f / sqrtf((float)D);
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int j = 0; j <= p; ++j) {
    if (a.window && j <= p - a.window && j >= a.sinks) {
      j = p - a.window;  // to the window's first token
      continue;
    }
    float s = 0.f;
    for (int c = 0; c < N; ++c) {
      const int d = 128 * (c / 4) + 4 * lane + c % 4;
      float k = chunk_value(lo, a.cp, 0, layer, b, h, j, qe, ce, d, &bad);
      if (lo.flags & KVQ_K_PRE_ROPE) {
        const int i = d % (D / 2);
        const float o = chunk_value(lo, a.cp, 0, layer, b, h, j, qe, ce, d < D / 2 ? d + D / 2 : d - D / 2, &bad);
        float sn, cs;
        sincospif((float)(int32_t)((j * a.turns[i]) >> 32) * 0x1p-31f, &sn, &cs);
        k = d < D / 2 ? k * cs - o * sn : k * cs + o * sn;
      }
      s += k * (j >= qe ? q[c] : qr[c]);
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= scale;
    const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
    l = l * f + e;
    m = mn;
    for (int c = 0; c < N; ++c) {
      const int d = 128 * (c / 4) + 4 * lane + c % 4;
      const float v = chunk_value(lo, a.cp, 1, layer, b, h, j, qe, ce, d, &bad);
      acc[c] = acc[c] * f + (j >= qe ? e * v : 0.f);
      accr[c] = accr[c] * f + (j < qe ? e * v : 0.f);
    }
  }
  if (bad) atomicOr(a.status, KVQ_DEV_PAGE);
  if (lo.flags & KVQ_ROTATE_V)
    for (int c = 0; c < N; c += 4) warp_unrotate128(accr + c, lo.d1, lo.d2);
  for (int c = 0; c < N; ++c) {
    const int d = 128 * (c / 4) + 4 * lane + c % 4;
    const float o = (acc[c] + accr[c]) / l;
    a.out[w * D + d] = lo.dtype == KVQ_DT_F16 ? __half_as_ushort(__float2half_rn(o)) : __bfloat16_as_ushort(__float2bfloat16_rn(o));
  }
}

size_t chunk_ws_bytes(const kvq_config*) { return kWsAlign; }

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_chunk_workspace_bytes(const kvq_config* cfg, size_t* bytes) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  *bytes = chunk_ws_bytes(cfg);
  return ok();
}

static kvq_status check_chunk_ws(const kvq_config* cfg, void* workspace, size_t ws_bytes) {
  if (!workspace) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  if (ws_bytes < chunk_ws_bytes(cfg))
    return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", ws_bytes, chunk_ws_bytes(cfg));
  if (((uintptr_t)workspace) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return KVQ_OK;
}

kvq_status kvq_chunk_workspace_init(const kvq_config* cfg, void* workspace, size_t ws_bytes, void* stream) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if ((st = check_chunk_ws(cfg, workspace, ws_bytes)) != KVQ_OK) return st;
  cudaError_t e = cudaMemsetAsync(workspace, 0, kWsAlign, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return ok();
}

kvq_status kvq_chunk_attention(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0, int32_t n_layers,
                               const void* q, const int32_t* cu_q, int32_t total_q, int32_t max_q,
                               const int32_t* seq_lens, int32_t window, int32_t sinks, void* out, void* workspace,
                               size_t ws_bytes, void* stream) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (layer0 < 0 || n_layers < 1 || n_layers > cfg->L - layer0)
    return fail(KVQ_ERR_ARG, "layers [%d, +%d) outside [0, %d)", layer0, n_layers, cfg->L);
  if (total_q < 0 || max_q < 0 || max_q > total_q) return fail(KVQ_ERR_ARG, "total_q=%d, max_q=%d", total_q, max_q);
  if (max_q > cfg->max_T) return fail(KVQ_ERR_CAPACITY, "max_q=%d > max_T=%d", max_q, cfg->max_T);
  if (window < 0 || sinks < 0) return fail(KVQ_ERR_ARG, "window=%d, sinks=%d", window, sinks);
  if (!cu_q || !seq_lens || (total_q > 0 && (!q || !out))) return fail(KVQ_ERR_ARG, "q / cu_q / seq_lens / out is NULL");
  if (((uintptr_t)q | (uintptr_t)out) & 15u) return fail(KVQ_ERR_ARG, "q / out must be 16-byte aligned");
  if (((uintptr_t)cu_q | (uintptr_t)seq_lens) & 3u) return fail(KVQ_ERR_ARG, "cu_q / seq_lens must be 4-byte aligned");
  ChunkArgs a{};
  if ((st = cache_ptrs(cfg, cache, &a.cp)) != KVQ_OK) return st;
  if ((st = check_chunk_ws(cfg, workspace, ws_bytes)) != KVQ_OK) return st;
  if (total_q == 0 || max_q == 0) return ok();
  a.lo = make_layout(cfg);
  a.layer0 = layer0;
  a.n_layers = n_layers;
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.cu_q = cu_q;
  a.seq_lens = seq_lens;
  a.total_q = total_q;
  a.max_q = max_q;
  a.window = window;
  a.sinks = sinks;
  a.status = (uint32_t*)workspace;
  a.cp.status = a.status;
  if (cfg->flags & KVQ_K_PRE_ROPE)
    for (int i = 0; i < cfg->D / 2; ++i)
      a.turns[i] = (uint64_t)std::ldexp(std::pow((double)cfg->rope_theta, -2.0 * i / cfg->D) / 6.283185307179586476925286766559, 64);
  const int64_t warps = (int64_t)n_layers * total_q * cfg->H_q;
  const int64_t blocks = (warps + 7) / 8;
  if (cfg->D == 128)
    chunk_simple_kernel<128><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  else
    chunk_simple_kernel<256><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "chunk attention kernel");
  return ok();
}

}  // extern "C"
