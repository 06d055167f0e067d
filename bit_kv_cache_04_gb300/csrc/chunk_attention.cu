// kvq_chunk_attention: the last tokens of every sequence attend to the packed
// cache, causally, over a sliding window plus the first tokens.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "chunk_attention.cuh"
#include "kvq_host.cuh"

namespace kvq {
namespace {

// Workspace: status word and the count of finished CTAs, tickets and flags (these zero between calls, also after one
// that stalled), partial rows.
struct ChunkWs {
  size_t tickets, nonfinite, partials, total;
  int grid;
};

ChunkWs chunk_ws(const kvq_config* c) {
  ChunkWs w{};
  w.grid = sm_count();  // one CTA per SM
  w.tickets = kWsAlign;
  const size_t words = align_up(sizeof(uint32_t) * (size_t)w.grid * kChunkTickets);
  w.nonfinite = w.tickets + words;
  w.partials = w.nonfinite + words;
  w.total = w.partials +
            align_up(sizeof(float) * (size_t)w.grid * kChunkSlots * chunk_slot_rows(c->D) * chunk_part_row(c->D));
  return w;
}

}  // namespace

size_t chunk_workspace_bytes(const kvq_config* cfg, size_t* zeroed) {
  const ChunkWs w = chunk_ws(cfg);
  if (zeroed) *zeroed = w.partials;
  return w.total;
}

int chunk_workspace(const kvq_config* cfg, void* workspace, ChunkArgs* a) {
  const ChunkWs w = chunk_ws(cfg);
  a->status = (uint32_t*)workspace;
  a->cp.status = a->status;
  a->left = a->status + 1;
  a->tickets = (uint32_t*)((char*)workspace + w.tickets);
  a->nonfinite = (uint32_t*)((char*)workspace + w.nonfinite);
  a->partials = (float*)((char*)workspace + w.partials);
  return w.grid;
}

int chunk_form(const kvq_config* cfg, int64_t rows) {
  return cfg->D != 128 ? kChunkShared : rows <= kFewRows ? kChunkFew : rows > 128 ? kChunkPaired : kChunkShared;
}

kvq_status chunk_common(const kvq_config* cfg, ChunkArgs* args, int most, int64_t owners, int* form) {
  ChunkArgs& a = *args;
  a.stall_polls = stall_polls();
  const bool wide = a.lo.kf.bits == 8 || (a.lo.tiered && a.lo.kc.bits == 8);
  const int shift = cfg->in_dtype == KVQ_DT_F16 ? 0 : wide ? 8 : 4;  // the largest code's bits: code times scale stays in fp16's range
  a.k_pre = std::ldexp(1.f, -shift);
  a.q_pre = cfg->flags & KVQ_ROTATE_K ? 0.0625f : 1.f;
  a.score_scale = (float)(1.4426950408889634 / std::sqrt((double)cfg->D)) / (a.k_pre * a.q_pre);
  a.k_one = ((25u - shift) << 10) * 0x10001u;
  if (cfg->flags & KVQ_K_PRE_ROPE)
    for (int i = 0; i < cfg->D / 2; ++i)
      a.turns[i] = (uint64_t)std::ldexp(std::pow((double)cfg->rope_theta, -2.0 * i / cfg->D) / 6.283185307179586476925286766559, 64);
  const int64_t rows = (int64_t)most * a.lo.g;
  if (rows > (int64_t)1 << 28) return fail(KVQ_ERR_UNSUPPORTED, "%d tokens x %d heads", most, a.lo.g);
  const int mode = chunk_form(cfg, rows);
  const int tile = chunk_tile(cfg->D), row_tile = mode == kChunkPaired ? 256 : 128;
  // the kernel counts its tiles in 32 bits
  const int64_t units = ((int64_t)a.total_q * a.lo.g / row_tile + owners) * a.n_layers * cfg->H_kv;
  if (units * (cfg->max_T / tile + 2) > 0x7fffffff - 2 * sm_count())
    return fail(KVQ_ERR_UNSUPPORTED, "too many tiles for one call: pass fewer layers or rows");
  a.g_magic = (uint32_t)((1ull << 32) / a.lo.g + 1);
  a.turn_here = (cfg->flags & KVQ_ROTATE_K) && rows <= 64 ? 1 : 0;
  a.cols = rows <= 16 ? 16 : kFewRows;
  a.by_warp = rows > 4 * row_tile;
  // Staging: 32-token subtiles as single bulk copies; pages of fewer tokens
  // as copies of their own when their bytes are whole 16-byte words and a
  // tile has at most one page per lane; other pages by plain loads.
  int sub = 0;
  for (const FmtInfo* f : {&a.lo.kf, &a.lo.vf, &a.lo.kc, &a.lo.vc})
    sub = std::max(sub, f->axis == KVQ_AXIS_CHANNEL ? f->row : 32 * f->row);
  a.sub_bytes = (sub + 15) & ~15;
  a.slot_bytes = a.sub_bytes * (chunk_tile(cfg->D) / 64);
  a.copy_shift = 5;
  if (a.lo.paged && a.lo.pt % 32 != 0) {
    const bool fits = 32 % a.lo.pt == 0 && chunk_tile(cfg->D) / a.lo.pt <= 32 &&
                      (a.lo.pt * a.lo.kf.row) % 16 == 0 && (a.lo.pt * a.lo.vf.row) % 16 == 0;
    if (fits) {
      a.small_pages = 1;
      while ((1 << a.copy_shift) > a.lo.pt) --a.copy_shift;
    } else {
      a.direct = 1;
    }
  }
  *form = mode;
  return KVQ_OK;
}

}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_chunk_workspace_bytes(const kvq_config* cfg, size_t* bytes) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if (!bytes) return fail(KVQ_ERR_ARG, "bytes is NULL");
  *bytes = chunk_ws(cfg).total;
  return ok();
}

static kvq_status check_chunk_ws(const kvq_config* cfg, void* workspace, size_t ws_bytes) {
  if (!workspace) return fail(KVQ_ERR_WORKSPACE, "workspace is NULL");
  if (ws_bytes < chunk_ws(cfg).total)
    return fail(KVQ_ERR_WORKSPACE, "workspace %zu B < %zu B needed", ws_bytes, chunk_ws(cfg).total);
  if (((uintptr_t)workspace) % kWsAlign) return fail(KVQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return KVQ_OK;
}

kvq_status kvq_chunk_workspace_init(const kvq_config* cfg, void* workspace, size_t ws_bytes, void* stream) {
  kvq_status st = check_config(cfg, false);
  if (st != KVQ_OK) return st;
  if ((st = check_chunk_ws(cfg, workspace, ws_bytes)) != KVQ_OK) return st;
  cudaError_t e = cudaMemsetAsync(workspace, 0, chunk_ws(cfg).partials, (cudaStream_t)stream);
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
  {
    const uintptr_t bytes = (uintptr_t)2 * n_layers * total_q * cfg->H_q * cfg->D, x = (uintptr_t)q, y = (uintptr_t)out;
    if (total_q > 0 && x < y + bytes && y < x + bytes) return fail(KVQ_ERR_ARG, "q and out overlap");
  }
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
  const int grid = chunk_workspace(cfg, workspace, &a);
  int mode;
  if ((st = chunk_common(cfg, &a, max_q, cfg->batch, &mode)) != KVQ_OK) return st;
  cudaError_t e = mode == kChunkFew ? launch_chunk_few(a, grid, (cudaStream_t)stream)
                  : cfg->D == 128   ? launch_chunk_d128(a, mode, grid, (cudaStream_t)stream)
                                    : launch_chunk_d256(a, grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "chunk attention kernel");
  return ok();
}

}  // extern "C"
