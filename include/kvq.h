/*
 * kvq.h - C ABI of libkvq: a quantized KV cache for decode attention on
 * NVIDIA GB300 (sm_103a).
 *
 * The operations follow five web pages on KV-cache quantization:
 *  - troisinh.com "KV Cache Quantization - Nen cache INT4/INT3" (sections
 *    "Tai sao Key va Value lai khac nhau?", "Mixed Precision", "Tai sao no
 *    hoat dong": per-channel keys, per-token values, Hadamard rotation,
 *    pre-RoPE keys rotated on the fly, hot 4-bit / cold 2-bit tokens);
 *  - nalar.dev "Kuantisasi KV Cache dengan Error Budget yang Eksplisit"
 *    (sections "Ukuran cache...", "Error pada key...", "Error pada value...",
 *    "Granularitas...", "Evaluasi...": the size law 2*L*T*H_kv*D, the scores
 *    s_i = q.k_i/sqrt(D), the output sum_i p_i v_i, a recent window kept at
 *    higher precision);
 *  - trefon.com "Matematyka cache KV" (sections "Bajty na token", the format
 *    table of "Przyklad: model 27B przy 262K", "Jak 4-bitowemu cache to
 *    uchodzi: najpierw obrot": block layouts Q8_0 34 B/32, Q4_0 18 B/32,
 *    66 B/128, 50 B/128; the randomized Walsh-Hadamard transform; attention
 *    in the rotated domain);
 *  - lehuy.net "NexusQuant" (section "Cac mo hinh duoc ho tro": split-half
 *    RoPE).
 *
 * Conventions shared by every entry point:
 *  - Ownership: the library never allocates device memory.  The caller owns
 *    every buffer and passes raw device pointers and a cudaStream_t (as
 *    void*; NULL means the legacy default stream).
 *  - Asynchrony: every call only enqueues work on the given stream, except
 *    kvq_read_device_status, which synchronizes that stream.
 *  - Errors: a kvq_status return.  Bad arguments are rejected on the host
 *    before anything is launched, with a message in kvq_last_error().  Bad
 *    runtime data found by a kernel (a length beyond capacity, a page id out
 *    of range) sets a bit of the device status word in the workspace and
 *    skips that piece of work; nothing traps.  The only waits are bounded
 *    waits of a CTA for its own copies into shared memory and, in
 *    kvq_chunk_attention, of its roles for one another (KVQ_DEV_STALL when
 *    one runs out).
 *  - Head mapping: query head h reads kv head h / (H_q / H_kv).
 *  - Softmax scale: fixed at 1/sqrt(D).
 *
 * Cache representation (per sequence of T tokens, per layer and kv head):
 *  - tokens [q_end, T) stay unquantized in a 16-bit window (raw bits of the
 *    input dtype), q_end = max(0, floor((T - R)/Gamma)) * Gamma, where R is
 *    residual_window and Gamma is the token group of a per-channel format (1
 *    when both formats are per-token);
 *  - with hot_window W > 0: tokens [c_end, q_end) are in the hot formats
 *    (k_fmt, v_fmt) and [0, c_end) in the cold formats (k_cold, v_cold),
 *    c_end = max(0, floor((q_end - W)/Gamma)) * Gamma; a group that leaves
 *    the hot tier is requantized from its dequantized hot values;
 *  - with W = 0: tokens [0, q_end) are in k_fmt / v_fmt.
 *
 * Block: fp16 scale (little endian) then G*b/8 bytes of codes.  Absmax
 * scaling in fp32: amax = max|x|, scale = fp16_rn(min(amax/qmax, 65504)),
 * code = clamp(rint(x / float(scale)), -qmax, qmax), qmax = 2^(b-1) - 1,
 * all codes 0 when the scale is 0.  Packing: 8-bit two's complement;
 * 4-bit code+8, element 2i in the low nibble of byte i; 3-bit code+4,
 * eight values per 24-bit little-endian word, value j at bits [3j, 3j+3);
 * 2-bit code+2, value j of a byte at bits [2j, 2j+2).
 *
 * Buffer layouts (byte arrays; "row" = one storage row):
 *  - per-token row: the D/G blocks of one token and kv head;
 *  - per-channel row: D blocks (channel-ascending), each one channel over
 *    the G tokens of one token group;
 *  - main tier, contiguous: [L][batch][H_kv][capacity][row], capacity =
 *    max_T rounded up to a multiple of 32 tokens (per-token rows) or
 *    ceil(max_T/G) groups (per-channel rows);
 *  - main tier, paged (page_tokens > 0, per-token formats, W = 0):
 *    [L][n_pages][H_kv][page_tokens][row]; block_table is
 *    [batch][max_pages_per_seq] int32 (device), page of token t =
 *    block_table[seq][t / page_tokens];
 *  - hot tier when W > 0: a ring of W/G + 1 group rows (per-channel) or
 *    W + Gamma token rows (per-token); slot = index mod ring length;
 *  - cold tier: [L][batch][H_kv][capacity][row] (capacity as above);
 *  - window: [L][batch][H_kv][R + Gamma][D] 16-bit values, slot = t mod
 *    (R + Gamma).
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_ARG = 1,          /* invalid argument; nothing launched */
  KVQ_ERR_UNSUPPORTED = 2,  /* valid but not implemented combination */
  KVQ_ERR_CUDA = 3,         /* a CUDA runtime call failed */
  KVQ_ERR_CAPACITY = 4,     /* a host-visible size exceeds capacity */
  KVQ_ERR_WORKSPACE = 5     /* workspace missing or too small */
} kvq_status;

typedef enum { KVQ_DT_F16 = 0, KVQ_DT_BF16 = 1, KVQ_DT_F32 = 2 /* logits only */ } kvq_dtype;

/* A block spans G consecutive channels of one token (TOKEN) or one channel
 * over G consecutive tokens (CHANNEL). */
typedef enum { KVQ_AXIS_TOKEN = 0, KVQ_AXIS_CHANNEL = 1 } kvq_axis;

/* bits in {8, 4, 3, 2} (16 is accepted by the size functions only, meaning
 * plain 16-bit storage); group in {32, 128}, dividing D for TOKEN; group 32
 * for CHANNEL. */
typedef struct {
  int32_t bits;
  int32_t group;
  int32_t axis;
} kvq_fmt;

/* flags */
enum {
  KVQ_ROTATE_K = 1u << 0,  /* randomized Hadamard-128 on K before quantizing (TOKEN formats) */
  KVQ_ROTATE_V = 1u << 1,  /* the same on V */
  KVQ_K_PRE_ROPE = 1u << 2, /* K is stored pre-RoPE; decode applies split-half RoPE at position t */
  /* TBQ4 (trefon.com, "Jak 4-bitowemu cache to uchodzi: najpierw obrot"): a rotated
   * 4-bit 128-value block holds the block's L2 norm (fp16) and, per value, the index
   * of the nearest of the 16 Lloyd-Max centroids of N(0, 1/128) (see
   * kvq_tbq4_codebook).  Needs the tensor's rotation flag, 4 bits, group 128,
   * per-token blocks, one tier.  Same 66 B per 128 values.  The append kernels
   * find an index with one lookup in bins of 1/8 octave of |u|; validation
   * answers KVQ_ERR_UNSUPPORTED if two nonzero thresholds ever shared a bin
   * (the built-in table's never do). */
  KVQ_TBQ4_K = 1u << 3,
  KVQ_TBQ4_V = 1u << 4,
  /* Asymmetric blocks ("scale and zero point", nalar.dev, "Granularitas
   * kuantisasi..."): every block of that tensor (both tiers) is the fp16 scale
   * s, the fp16 zero z (the block minimum), then codes c in [0, 2^b - 1] in the
   * usual bit fields, x = c s + z: 2 more bytes per block (20 B / 32 values
   * at 4 bits, 12 B / 32 at 2 bits).  Needs 4- or 2-bit
   * blocks of 32 values, no rotation.  The tensor-core decode reads them when
   * both tensors are asymmetric (the zero adds one term per block to the
   * scores or the output); other mixes take the generic decode kernel. */
  KVQ_ZP_K = 1u << 5,
  KVQ_ZP_V = 1u << 6
};

/* Device status bits (workspace word 0), OR-ed by kernels. */
enum {
  KVQ_DEV_CAPACITY = 1u << 0, /* an append would exceed max_T, or more new tokens than max_new */
  KVQ_DEV_PAGE = 1u << 1,     /* a block_table entry outside [0, n_pages) */
  KVQ_DEV_RANGE = 1u << 2,    /* kvq_dequantize range outside [0, T) */
  KVQ_DEV_LENGTH = 1u << 3,   /* a sequence length < 0 or > max_T, or cu_new not ascending */
  KVQ_DEV_STALL = 1u << 4,    /* a bounded wait ran out: of a decode kernel for its own bulk copy into shared
                                 memory, or of a chunk attention role for another one of its CTA; that call's
                                 outputs are undefined, and the next call on the workspace is whole again */
  KVQ_DEV_BOUNDS = 1u << 5,   /* bounds-checked build only (libkvq_checked.so): a computed cache address
                                 fell outside its buffer segment; the access was skipped */
  KVQ_DEV_SEQ = 1u << 6       /* a sequence index of a page call outside [0, batch), listed twice where that is
                                 not allowed, or a fork target that is not empty */
};

typedef struct {
  int32_t L;        /* layers held by the buffers */
  int32_t H_kv;     /* kv heads */
  int32_t H_q;      /* query heads, a multiple of H_kv, H_q/H_kv <= 8 */
  int32_t D;        /* head dim: 128 or 256 */
  int32_t batch;    /* sequences */
  int32_t max_T;    /* capacity in tokens per sequence */
  int32_t in_dtype; /* kvq_dtype of k, v, q inputs and of the window */
  kvq_fmt k_fmt, v_fmt;   /* the only tier (W = 0) or the hot tier */
  kvq_fmt k_cold, v_cold; /* cold tier when hot_window > 0 (same axis and group, fewer bits) */
  int32_t hot_window;      /* W: tokens kept in the hot tier (multiple of Gamma), 0 = one tier */
  int32_t residual_window; /* R: tokens kept in the 16-bit window, 0 allowed */
  uint32_t flags;          /* OR of KVQ_ROTATE_K, KVQ_ROTATE_V, KVQ_K_PRE_ROPE, KVQ_TBQ4_K,
                              KVQ_TBQ4_V, KVQ_ZP_K, KVQ_ZP_V (see the flags above) */
  float rope_theta;        /* RoPE base (KVQ_K_PRE_ROPE), e.g. 10000 */
  uint64_t sign_seed;      /* 0: plain Sylvester transform; else SplitMix64 sign vectors */
  int32_t page_tokens;     /* 0 = contiguous; 16 = paged main tier */
  int32_t n_pages;         /* pages in the pool (paged) */
  int32_t max_pages_per_seq; /* block_table row length (paged) */
  int32_t reserved;        /* must be 0 */
} kvq_config;

/* Every buffer is 16-byte aligned (KVQ_ERR_ARG otherwise). */
typedef struct {
  void* k_main;  /* main / hot tier of K */
  void* v_main;  /* main / hot tier of V */
  void* k_cold;  /* cold tier of K (hot_window > 0), else NULL */
  void* v_cold;  /* cold tier of V (hot_window > 0), else NULL */
  void* k_resid; /* 16-bit window of K (when R + Gamma > 1), else NULL */
  void* v_resid; /* 16-bit window of V */
  const int32_t* block_table; /* [batch][max_pages_per_seq] device (paged), else NULL */
} kvq_cache;

/* Version string of the library. */
KVQ_API const char* kvq_version(void);

/* Message of the last error returned on this thread ("" if none). */
KVQ_API const char* kvq_last_error(void);

/* Checks a configuration (the same checks every entry point makes). */
KVQ_API kvq_status kvq_validate_config(const kvq_config* cfg);

/* Bytes of one block: 2 + group*bits/8 (2*group for bits = 16)
 * (trefon.com, format table). */
KVQ_API kvq_status kvq_block_bytes(int32_t bits, int32_t group, int32_t* bytes);

/* Steady-state bytes per token over all L layers, K and V, in the format
 * that holds most of a long sequence (cold when hot_window > 0).  Scales
 * count (nalar.dev, section "Ukuran cache...": compare actual bytes per
 * token; trefon.com, section "Bajty na token"). */
KVQ_API kvq_status kvq_bytes_per_token(const kvq_config* cfg, int64_t* bytes);

/* Exact bytes the representation keeps for one sequence of T tokens over
 * all layers: cold + hot/main tiers + 16-bit window, K and V. */
KVQ_API kvq_status kvq_cache_bytes(const kvq_config* cfg, int64_t T, int64_t* bytes);

/* Bytes to allocate for the six kvq_cache buffers, in the order k_main,
 * v_main, k_cold, v_cold, k_resid, v_resid (0 = buffer not used). */
KVQ_API kvq_status kvq_buffer_sizes(const kvq_config* cfg, size_t sizes[6]);

/* Bytes of the workspace every launching call takes (status word, split
 * tickets, RoPE tables, split partials); 256-byte aligned. */
KVQ_API kvq_status kvq_workspace_bytes(const kvq_config* cfg, size_t* bytes);

/* Prepares a workspace of at least kvq_workspace_bytes: zeroes the status
 * word and tickets and fills the RoPE tables.  Call once after allocating
 * it; later calls keep the tickets at zero themselves. */
KVQ_API kvq_status kvq_workspace_init(const kvq_config* cfg, void* workspace, size_t ws_bytes, void* stream);

/* Quantize-on-append for layers [layer0, layer0 + n_layers): every new
 * token is rotated (flags), scaled per block and coded into the layout above
 * (trefon.com, format table of "Przyklad: model 27B przy 262K"; per-channel
 * keys and per-token values as troisinh.com "Tai sao Key va Value lai khac
 * nhau?"; the recent window kept unquantized as nalar.dev "Evaluasi harus
 * memisahkan...").
 *  k, v:     [n_layers][total_new][H_kv][D] in_dtype, device, 16-byte
 *            aligned (KVQ_ERR_ARG otherwise); sequences back
 *            to back in batch order (post-RoPE keys, or pre-RoPE with
 *            KVQ_K_PRE_ROPE).
 *  cu_new:   [batch + 1] int32 device, cu_new[0] = 0, cu_new[batch] =
 *            total_new; sequence b appends cu_new[b+1] - cu_new[b] tokens.
 *  seq_lens: [batch] int32 device, lengths BEFORE this append (the caller
 *            advances them after all layers, e.g. with kvq_commit_lengths).
 *  total_new, max_new: host copies of cu_new[batch] and of the largest
 *            per-sequence count (they size the grids).
 * Window tokens move into the quantized tiers by whole groups; bulk append
 * and token-by-token append give the same cache.  Inputs are finite or
 * infinite numbers; a block holding a NaN gets unspecified codes (and a NaN
 * or unspecified scale), and no other block is affected. */
KVQ_API kvq_status kvq_append(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0, int32_t n_layers,
                      const void* k, const void* v, const int32_t* cu_new, const int32_t* seq_lens,
                      int32_t total_new, int32_t max_new, void* workspace, size_t ws_bytes, void* stream);

/* seq_lens[b] += cu_new[b+1] - cu_new[b] on the device. */
KVQ_API kvq_status kvq_commit_lengths(const kvq_config* cfg, const int32_t* cu_new, int32_t* seq_lens, void* stream);

/* Decode attention of one query token per sequence, for layers
 * [layer0, layer0 + n_layers) (independent per-layer queries; n_layers > 1
 * only saves launches), read straight from the packed blocks: scores
 * s_t = q.k_t / sqrt(D) and output sum_t p_t v_t as nalar.dev "Error pada
 * key mengubah input softmax" and "Error pada value masuk setelah attention
 * probability" define them; rotated blocks are read in the rotated domain
 * (trefon.com, "Jak 4-bitowemu cache to uchodzi: najpierw obrot").
 *  q:        [n_layers][batch][H_q][D] in_dtype, device, post-RoPE.
 *  seq_lens: [batch] int32 device, tokens currently cached.
 *  out:      [n_layers][batch][H_q][D] fp32, device:
 *            out = sum_t softmax_t(q.k_t/sqrt(D)) v_t over the dequantized
 *            cache (keys RoPE-rotated at position t when stored pre-RoPE);
 *            0 for an empty sequence.
 *  num_splits: blocks per (layer, seq, kv head), 1..256; 0 picks the
 *            count (kvq_decode_splits).  With more than one, the tensor-core
 *            decode plans on the device from all lengths: when its grid is
 *            at most two waves of resident blocks, each unit of n tiles
 *            (32 tokens) is cut into ceil(n / C) nearly equal chunks for the
 *            smallest C that fits the budget, so long sequences get more
 *            blocks and short ones fewer (with a count passed here, no unit
 *            gets more than num_splits).  With 0, the budget is one whole
 *            wave of resident blocks per call where that exceeds batch x
 *            kvq_decode_splits blocks per (layer, kv head), and the grid
 *            grows to hold it (blocks past the last chunk exit at once;
 *            without room in the workspace the plain budget stays).  The
 *            result does not depend on the
 *            split beyond the order of fp32 sums.  KVQ_ERR_WORKSPACE when the
 *            workspace's partial rows cannot hold the blocks. */
KVQ_API kvq_status kvq_decode_attention(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0,
                                int32_t n_layers, const void* q, const int32_t* seq_lens, float* out,
                                int32_t num_splits, void* workspace, size_t ws_bytes, void* stream);

/* One decode step: appends one token to every sequence, then decode
 * attention over the cache including it (nalar.dev, "Pertumbuhan cache
 * dinamis mengubah persoalan kalibrasi": the cache grows by one entry per
 * generated token and is written online).  Equivalent to kvq_append of
 * k_new / v_new with one token per sequence followed by
 * kvq_decode_attention over seq_lens[b] + 1 tokens: the same cache bytes
 * and the same outputs.
 *  k_new, v_new: [n_layers][batch][H_kv][D] in_dtype, device, 16-byte
 *            aligned: the new token of every (layer, sequence).
 *  q, out, num_splits: as kvq_decode_attention.
 *  seq_lens: [batch] int32 device, lengths BEFORE the step; the new token
 *            is at position seq_lens[b].  Not advanced here: the caller
 *            advances them after all layers (kvq_commit_lengths with
 *            cu_new = 0, 1, ..., batch).
 * When the tensor-core decode handles the formats the step is one launch:
 * the blocks that own the (at most three) tiles the token changes -- its
 * window slot, the unit leaving the window, the group leaving the hot tier
 * -- write them and then decode them; no block waits for another.  Other
 * formats run the append and decode launches in turn. */
KVQ_API kvq_status kvq_decode_step(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0, int32_t n_layers,
                                   const void* k_new, const void* v_new, const void* q, const int32_t* seq_lens,
                                   float* out, int32_t num_splits, void* workspace, size_t ws_bytes, void* stream);

/* Kernel launches one kvq_decode_step call makes (1 when fused). */
KVQ_API kvq_status kvq_step_launches(const kvq_config* cfg, int32_t* launches);

/* The split count per (layer, seq, kv head) kvq_decode_attention takes for
 * num_splits = 0: the count with the best fill of whole waves of resident
 * blocks (the device's SM count), each block keeping at least 8 tiles of the
 * longest possible sequence (48 for rotated formats).  A call whose chunks
 * are planned on the device may widen it to give the plan one whole wave
 * (kvq_decode_attention). */
KVQ_API kvq_status kvq_decode_splits(const kvq_config* cfg, int32_t n_layers, int32_t* splits);

/* Dequantizes tokens [t0, t1) of (layer, seq) to fp32 k_out, v_out
 * [t1 - t0][H_kv][D] (device) in the original domain: x = code * scale
 * (+ zero) per block (trefon.com, format table), rotation undone, keys as
 * stored (pre-RoPE when flagged).  k_out and v_out hold at least
 * (t1 - t0) * H_kv * D floats each; the caller owns them.  seq_lens as for decode; a range beyond
 * the current length sets KVQ_DEV_RANGE and writes nothing. */
KVQ_API kvq_status kvq_dequantize(const kvq_config* cfg, const kvq_cache* cache, int32_t layer, int32_t seq,
                          int32_t t0, int32_t t1, const int32_t* seq_lens, float* k_out, float* v_out,
                          void* workspace, size_t ws_bytes, void* stream);

/* Size of the library's built-in device scratch used by
 * kvq_decode_attention_static (32 MiB on every GPU that loads the library,
 * held until the process exits). */
#define KVQ_STATIC_SCRATCH_BYTES (32u << 20)

/* Decode attention that allocates nothing and takes no workspace.
 *
 * There is no counterpart on the pages: this is an addition of this library
 * for callers that cannot hand it device memory.  Examples are code whose
 * device memory all belongs to another runtime's pool that it may not
 * allocate from, and plugins that are given inputs and outputs but no
 * scratch buffer.  kvq_decode_attention needs the caller to allocate a
 * workspace; this variant keeps the same scratch (split partials, tickets,
 * status word, RoPE tables) in a fixed device array inside the library.
 *
 * Arguments and results are those of kvq_decode_attention without the
 * workspace.  The call needs 256 B + 4 B per (layer, sequence, kv head)
 * unit + the RoPE tables (KVQ_K_PRE_ROPE) + the split partials; a call that
 * needs more than KVQ_STATIC_SCRATCH_BYTES returns KVQ_ERR_WORKSPACE and
 * launches nothing (pass a smaller n_layers or num_splits).  It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *
 * The first call on each device looks up the array's device address with
 * that device current, so make that first call before any stream capture.
 * Every call on a device uses the same array and leaves its contents
 * behind; each call clears the parts that must start at zero (tickets and
 * status word) on `stream`, so calls that overlap on the GPU (two streams,
 * or two threads) race and must be serialized by the caller.  Device status
 * bits of these calls are not reported. */
KVQ_API kvq_status kvq_decode_attention_static(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0,
                                               int32_t n_layers, const void* q, const int32_t* seq_lens,
                                               float* out, int32_t num_splits, void* stream);

/* Kernel launches one kvq_append call (with new tokens) and one
 * kvq_decode_attention call make for this configuration, e.g. to budget
 * launches per decode step.  No pages counterpart: library bookkeeping. */
KVQ_API kvq_status kvq_launch_counts(const kvq_config* cfg, int32_t* append_launches, int32_t* decode_launches);

/* The TBQ4 tables the library uses: the 16 Lloyd-Max centroids of
 * N(0, sigma^2), sigma = 1/sqrt(128), ascending, from Lloyd's algorithm run
 * on the host in fp64 and rounded once to fp16 (the lookup table), and the
 * 15 decision thresholds, the exact midpoints of neighbouring entries.  A
 * value u = y / norm (fp32, y the rotated value) takes the index of the
 * number of thresholds strictly below u; it decodes as centroid[index] *
 * norm.  The norm is fp16(min(sqrt(S), 65504)) with S = (p0 + p1) + (p2 + p3)
 * in fp32, p_k the sum of y_i^2 over the k-th run of 32 values in index
 * order.  No device work; the tables are computed once per process. */
KVQ_API kvq_status kvq_tbq4_codebook(float centroids[16], float thresholds[15]);

/* Testing hook of the failure-detection path; no counterpart on the pages.
 * While polls > 0, every tensor-core decode launch (kvq_decode_attention,
 * kvq_decode_step, kvq_decode_attention_static) makes its warps' first copy
 * wait on a shared-memory barrier that nothing ever completes, bounded by
 * `polls` polls: the wait runs out, KVQ_DEV_STALL is set, the warp waits
 * (with the normal bound) for its bulk copies still in flight and the
 * kernel finishes; that call's outputs are undefined.  In every second CTA
 * of kvq_chunk_attention one of the roles (products, loads, dequantization,
 * softmax, in turn) does the same and leaves; the others give up in turn, and the CTAs between
 * finish their runs.  polls = 0 (the
 * default) turns it off.  Process-wide; polls outside [0, 2^20] give
 * KVQ_ERR_ARG.  Not for production use. */
KVQ_API kvq_status kvq_test_force_stall(int32_t polls);

/* Testing hook of the bounds-checked build (libkvq_checked.so, compiled
 * with KVQ_BOUNDS_CHECK); no counterpart on the pages.  Later calls treat
 * the last `rows` rows (or page rows) of every cache segment as outside the
 * buffer, so accesses there set KVQ_DEV_BOUNDS and are skipped: a test that
 * the checks fire without any real out-of-bounds access.  0 (the default)
 * turns it off.  The normal build answers KVQ_ERR_UNSUPPORTED for rows > 0. */
KVQ_API kvq_status kvq_test_shrink_bounds(int32_t rows);

/* Synchronizes `stream` and reads the device status word (KVQ_DEV_* bits). */
KVQ_API kvq_status kvq_read_device_status(const void* workspace, uint32_t* bits, void* stream);

/* Clears the device status word. */
KVQ_API kvq_status kvq_clear_device_status(void* workspace, void* stream);

/* ==== serving operators around the cache =====================================
 * Queries and keys made ready (norm + rotary turn), pages of a paged cache
 * shared, moved and freed, and attention of many new tokens over the packed
 * cache.  These are additions of this library next to the pages' method; the
 * formulas are stated with each entry. */

/* ---- norm and rotary turn of queries and keys -------------------------------- */

/* How the turn frequencies f_i = theta^(-2i / rot_dim), i in [0, rot_dim / 2),
 * are scaled for contexts longer than the original one:
 *  NONE    f_i
 *  LINEAR  f_i / factor
 *  NTK     theta replaced by theta * factor^(rot_dim / (rot_dim - 2)) (theta kept when rot_dim = 2)
 *  YARN    r_i f_i / factor + (1 - r_i) f_i, r_i = clamp((i - a) / max(z - a, 0.001), 0, 1) with
 *          a = max(0, floor(p(high))), z = min(rot_dim - 1, ceil(p(low))),
 *          p(x) = rot_dim ln(original_len / (2 pi x)) / (2 ln theta); cos and sin times
 *          attn_factor (0 means 0.1 ln(factor) + 1)
 *  BANDS   b_i f_i + (1 - b_i) f_i / factor, b_i = clamp((n_i - low) / (high - low), 0, 1), n_i =
 *          original_len f_i / (2 pi), the turns within the original context */
typedef enum {
  KVQ_ROPE_NONE = 0,
  KVQ_ROPE_LINEAR = 1,
  KVQ_ROPE_NTK = 2,
  KVQ_ROPE_YARN = 3,
  KVQ_ROPE_BANDS = 4
} kvq_rope_scaling;

typedef struct {
  int32_t D;            /* head dim: 128 or 256 */
  int32_t rot_dim;      /* channels [0, rot_dim) turn, the others pass: even, 2..D */
  int32_t interleaved;  /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1) */
  int32_t scaling;      /* kvq_rope_scaling */
  double theta;         /* base, > 1 */
  double factor;        /* >= 1 (LINEAR, NTK, YARN, BANDS) */
  double low, high;     /* YARN, BANDS: turns within original_len, 0 < low < high */
  int32_t original_len; /* YARN, BANDS: >= 1 */
  int32_t reserved;     /* must be 0 */
  double attn_factor;   /* factor on cos and sin; 0: the scaling's own (1, or YARN's) */
} kvq_rope_params;

/* A prepared turn: plain host data that the caller keeps and passes by
 * pointer; made by kvq_rope_plan_init and not changed by any call.
 * turns[i] = frequency i in turns per position, as a 64-bit binary fraction
 * (f_i / (2 pi) * 2^64): position * turns[i] mod 2^64 is the angle, exact to
 * the fraction's last bits at any 32-bit position. */
typedef struct {
  int32_t D, rot_dim, interleaved, reserved;
  float scale;  /* factor on cos and sin */
  float unused;
  uint64_t turns[128];
} kvq_rope_plan;

KVQ_API kvq_status kvq_rope_plan_init(const kvq_rope_params* params, kvq_rope_plan* plan);

/* Per-head RMS norm and rotary turn of queries and keys in one pass:
 *   y = x / sqrt(mean(x^2) + eps) * w   (only with a weight; over the D channels of one head)
 *   (y_a, y_b) -> m (y_a cos - y_b sin, y_b cos + y_a sin)  for every pair (a, b) of the plan,
 * angle = position * f_i, all in fp32 and rounded once to in_dtype.
 *  plan:   NULL leaves out the turn (then positions may be NULL).
 *  q, k:   [n_tokens][H_q or H_kv][D] in_dtype, device; strides in elements
 *          between tokens and between heads (channels contiguous), so heads
 *          of a fused projection are read in place.  Either may be NULL with its output.
 *  q_weight, k_weight: [D] in_dtype, device, or NULL (no norm of that tensor).
 *  positions: [n_tokens] int32, device (any value; negative ones turn backwards).
 *  q_out, k_out: [n_tokens][H][D] in_dtype, contiguous: the layout kvq_append
 *          and the attention entries take.  May be the input itself when that is
 *          contiguous; any other overlap is not allowed.
 * cfg gives H_q, H_kv, D and in_dtype. */
KVQ_API kvq_status kvq_qk_norm_rope(const kvq_config* cfg, const kvq_rope_plan* plan, const void* q,
                                    int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                    int64_t k_token_stride, int64_t k_head_stride, const void* q_weight,
                                    const void* k_weight, float eps, const int32_t* positions, int32_t n_tokens,
                                    void* q_out, void* k_out, void* stream);

/* ---- pages of a paged cache ------------------------------------------------------
 * The block table [batch][max_pages_per_seq] holds page ids, -1 where there
 * is none.  refs [n_pages] counts, per page, the table entries that hold it;
 * a page with refs 0 is free.  Both belong to the caller, like the lengths;
 * these calls keep them consistent, all on the device, in stream order:
 * they read no length on the host and can be captured.
 *
 * A sequence's pages hold its quantized tokens [0, q_end); the 16-bit window
 * (residual_window > 0) is per sequence.  A page that several sequences hold
 * is read by all of them and written by none: before tokens are appended,
 * kvq_pages_reserve gives the sequence its own copy of a partly filled page.
 *
 * All need a paged config (page_tokens > 0) with batch <= 32768 and
 * batch * (max_pages_per_seq + 1) < 2^31.  The
 * workspace is of kvq_pages_workspace_bytes, 256-byte aligned, prepared by
 * kvq_pages_init; its first word is the device status word
 * (kvq_read_device_status).  Lists (seqs, src, dst, n_new) are int32 on the
 * device, n of them known to the host. */
KVQ_API kvq_status kvq_pages_workspace_bytes(const kvq_config* cfg, size_t* bytes);

/* Prepares the workspace and counts refs from the block table (all -1: every
 * page is free).  An entry outside [-1, n_pages) sets KVQ_DEV_PAGE and is not counted. */
KVQ_API kvq_status kvq_pages_init(const kvq_config* cfg, const int32_t* block_table, int32_t* refs, void* workspace,
                                  size_t ws_bytes, void* stream);

/* Frees sequences: their table rows become -1, each page loses one reader
 * (free when that was the last), their lengths become 0.  An index outside
 * [0, batch) sets KVQ_DEV_SEQ and is passed over; one listed twice is freed
 * once.  An entry outside the pool, or a page with no readers, sets KVQ_DEV_PAGE. */
KVQ_API kvq_status kvq_pages_release(const kvq_config* cfg, int32_t* block_table, int32_t* refs, int32_t* seq_lens,
                                     const int32_t* seqs, int32_t n, void* workspace, size_t ws_bytes, void* stream);

/* Sequence dst[i] becomes a copy of src[i]: it shares the pages that hold
 * quantized tokens (each gets one more reader), gets a copy of the 16-bit
 * window of every layer, and the length.  Pairs that are passed over, with
 * KVQ_DEV_SEQ set: an index outside [0, batch); a dst that is not empty
 * (length 0 and no pages) or that an earlier pair has too; a sequence listed both
 * as a src and as a dst (every pair that has it).
 * A page of src outside the pool (KVQ_DEV_PAGE) or a bad length (KVQ_DEV_LENGTH) passes the
 * pair over too. */
KVQ_API kvq_status kvq_pages_fork(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table, int32_t* refs,
                                  int32_t* seq_lens, const int32_t* src, const int32_t* dst, int32_t n,
                                  void* workspace, size_t ws_bytes, void* stream);

/* Makes room for n_new[i] more tokens of sequence seqs[i] (lengths as before
 * the append, and not advanced): its table row gets pages for tokens [0,
 * length + n_new[i]), and if the page that the next quantized token goes to
 * is partly filled and has other readers, a copy of it (all layers, K and V).  New pages
 * are the free pages with the lowest ids, given out in list order and, within a sequence, in
 * row order.  Where several listed sequences share such a page they are
 * served in list order: the last reader left keeps the page itself.
 * All or nothing: with too few free pages or a length beyond max_T
 * (KVQ_DEV_CAPACITY), a bad or repeated index (KVQ_DEV_SEQ), a bad length or
 * count (KVQ_DEV_LENGTH), or a table that breaks the rules above
 * (KVQ_DEV_PAGE), nothing changes.
 * One block does the bookkeeping, so the time grows with the list: some 10 us
 * for 64 sequences, 0.3 to 0.5 ms for 4096, 3 to 13 ms for 32768. */
KVQ_API kvq_status kvq_pages_reserve(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table,
                                     int32_t* refs, const int32_t* seq_lens, const int32_t* seqs,
                                     const int32_t* n_new, int32_t n, void* workspace, size_t ws_bytes,
                                     void* stream);

/* Moves the used pages together: with U pages in use, those with ids >= U go,
 * in ascending order, to the free ids below U, in ascending order; the new
 * table and counts are written to table_out and refs_out (which may be the
 * inputs).  The bytes of the pages left behind stay as they were.  A
 * table entry outside the pool or of a free page sets KVQ_DEV_PAGE and becomes -1. */
KVQ_API kvq_status kvq_pages_compact(const kvq_config* cfg, const kvq_cache* cache, const int32_t* block_table,
                                     const int32_t* refs, int32_t* table_out, int32_t* refs_out, void* workspace,
                                     size_t ws_bytes, void* stream);

/* Reorders the sequences of a beam search: the batch is groups of `group`
 * consecutive slots (1..32, dividing batch), and slot b of a group becomes what slot
 * parents[b] of the same group was before the call: its pages that hold quantized tokens, length and 16-bit
 * window (all layers).  Pages that are reserved behind those stay one sequence's own: the slot's that keeps
 * it (parents[b] = b), else its lowest child's; without a child they are freed, and the other children have -1 there.
 * parents [batch] int32, device, counted from the group's
 * first slot, as kvq_beam_select writes them.  refs follow the table: a page that no slot
 * holds any more is free, one that several hold is copied by kvq_pages_reserve before
 * it is written.  No page moves.  A group with a parent outside [0, group) (KVQ_DEV_SEQ) or a bad length (KVQ_DEV_LENGTH)
 * stays as it was; a table entry outside the pool sets KVQ_DEV_PAGE, moves along and is not counted. */
KVQ_API kvq_status kvq_pages_reorder(const kvq_config* cfg, const kvq_cache* cache, int32_t* block_table,
                                     int32_t* refs, int32_t* seq_lens, const int32_t* parents, int32_t group,
                                     void* workspace, size_t ws_bytes, void* stream);

/* ---- selection of a beam search ----------------------------------------------------
 * The `beams` best continuations of every group's beams over the whole vocabulary.  With x the logits of beam b and s its
 * score, the candidate (b, v) scores
 *   c = s + x_v - log sum_u e^(x_u);
 * a finished beam has one candidate, the end token with c = s.  The group's candidates in descending order, ties to the
 * lower beam and then the lower token:
 *   scores_out[i] = c, tokens[i] = v, parents[i] = b, done_out[i] = the beam was finished, or v is the end token.
 * Maxima are taken of the logits as they are, sums in fp32 a thread and in 64 bits across threads' pieces, scores are compared
 * in 64 bits and rounded once.  Logits may lie anywhere: rows far from zero, or masked by large finite numbers, keep their log-sum.
 *  logits: [n_groups][beams][vocab] of dtype (KVQ_DT_F16, BF16 or F32), device; strides in elements between groups and beams, tokens
 *          contiguous.  -inf: the token may not follow.  NaN counts as -inf, +inf as the largest finite fp32 number.
 *  scores: [n_groups][beams] fp32 (-inf: an empty beam, e.g. all but the first of a new search; NaN counts as -inf).
 *  done:   [n_groups][beams] int32, not 0: finished; or NULL (none is).  Needs an end token.
 *  eos:    the end token, or -1 for none.
 *  scores_out, tokens, parents, done_out: [n_groups][beams]; scores_out may be scores and done_out may be done,
 *          nothing else may overlap (KVQ_ERR_ARG); done_out may be NULL.
 * With fewer candidates above -inf than beams the rest have -inf, the lowest beams and tokens first.
 * beams in 1..32, vocab below 2^26, n_groups * beams at most 2^24.
 *  workspace: kvq_beam_workspace_bytes bytes, 256-byte aligned, prepared once by kvq_beam_workspace_init for
 *          these sizes; calls that may run at the same time (captured ones that are replayed side by side, too) need one each. */
KVQ_API kvq_status kvq_beam_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, size_t* bytes);
KVQ_API kvq_status kvq_beam_workspace_init(int32_t n_groups, int32_t beams, int32_t vocab, void* workspace, size_t ws_bytes,
                                           void* stream);
KVQ_API kvq_status kvq_beam_select(const void* logits, int32_t dtype, int64_t group_stride, int64_t beam_stride,
                                   int32_t n_groups, int32_t beams, int32_t vocab, const float* scores, const int32_t* done,
                                   int32_t eos, float* scores_out, int32_t* tokens, int32_t* parents, int32_t* done_out,
                                   void* workspace, size_t ws_bytes, void* stream);

/* ---- attention of a chunk of new tokens over the packed cache ---------------------
 * The last n_b = cu_q[b+1] - cu_q[b] cached tokens of sequence b attend to
 * the cache, causally, optionally through a sliding window that always keeps
 * the first `sinks` tokens visible:
 *   out_i = sum_j softmax_j(q_i.k_j / sqrt(D)) v_j  over cached tokens j with
 *   j <= p_i and (window = 0 or j > p_i - window or j < sinks),
 * p_i = seq_lens[b] - n_b + i.  One call covers a decode step (n_b = 1), the
 * verification of a draft (a few) and prefill chunks (thousands), over every
 * format, tier and page layout of the cache as kvq_append left it.
 *  q, out:   [n_layers][total_q][H_q][D] in_dtype, device, 16-byte aligned, not
 *            overlapping; the rows of a sequence back to back in batch order; q post-RoPE.
 *            (A sequence's rows of out may hold intermediate values while the call runs.)
 *  cu_q:     [batch + 1] int32, device, cu_q[0] = 0.  Rows from cu_q[batch]
 *            to total_q are left as they are; a sequence may have no rows.
 *  total_q, max_q: host values: rows of q, and a bound on every n_b (at most total_q and max_T; with
 *            either 0 there is nothing to do, and the device values are not looked at).
 *  seq_lens: [batch] int32, device, cached tokens INCLUDING the chunk (the
 *            chunk was appended and the lengths advanced before this call).
 *  window:   0 = every earlier token; else tokens in the sliding window, the
 *            query's own among them.  sinks: >= 0 (no effect when window = 0).
 * Products run on the tensor cores with fp32 sums: keys and queries in fp16 (queries turned into a
 * rotated format's domain are rounded to it), values and probabilities in in_dtype; softmax statistics
 * and outputs are held in fp32 and rounded once.  What passes fp16's range counts as its end: queries
 * beyond 65504 (2^20 after the turn of a rotated format); in a bf16 cache keys beyond 2^20 (2^24 with 8-bit key
 * formats), which is more than its quantized tokens can hold; in an fp16 cache keys and values beyond 65504, as
 * dequantized or, in rotated formats, as turned.
 * A sequence with cu_q not ascending, n_b > max_q, a length outside [0,
 * max_T] or n_b > length sets KVQ_DEV_LENGTH and its rows are left as they are; a page
 * id out of range sets KVQ_DEV_PAGE and that page's tokens count as zeros.
 * A NaN or infinity in a 16-bit window token reaches only the queries that see the token.
 *  workspace: kvq_chunk_workspace_bytes bytes, 256-byte aligned, prepared once
 *            by kvq_chunk_workspace_init; calls that may run at the same time
 *            need workspaces of their own.  Its first word is the device
 *            status word (kvq_read_device_status). */
KVQ_API kvq_status kvq_chunk_workspace_bytes(const kvq_config* cfg, size_t* bytes);
KVQ_API kvq_status kvq_chunk_workspace_init(const kvq_config* cfg, void* workspace, size_t ws_bytes, void* stream);
KVQ_API kvq_status kvq_chunk_attention(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0,
                                       int32_t n_layers, const void* q, const int32_t* cu_q, int32_t total_q,
                                       int32_t max_q, const int32_t* seq_lens, int32_t window, int32_t sinks,
                                       void* out, void* workspace, size_t ws_bytes, void* stream);

/* ---- attention of groups of sequences that share a prefix -------------------------------
 * kvq_chunk_attention without a window, for paged caches where groups of consecutive sequences hold the same pages for a common
 * prefix (beams and samples of one prompt, chats behind one system prompt; kvq_pages_fork makes them): the prefix is
 * read and dequantized once for all of a group's rows.  The same rows in and out as kvq_chunk_attention, up to rounding.
 *
 * kvq_prefix_plan works out, on the device, what the groups share: the pages that all sequences of the group with
 * new tokens hold in the same places of their table rows, as far as they are quantized and before the new tokens of all of them, in
 * whole tiles of 128 tokens (64 with D = 256).  A group that shares less, has one sequence with new tokens, or has so many rows a
 * sequence that row tiles across sequences save nothing is attended to sequence by sequence.
 * One plan serves the calls of all layers; it holds until the lengths, the table or the rows change.
 * With one new token a sequence kvq_decode_attention gives the same rows, in fp32 and more exactly (2-norm errors of 2.7e-5; here 4.0e-4 with fp16,
 * 2.9e-3 with bf16, the output's rounding included).  It reads every sequence by itself, and layer by layer it is the faster one for few
 * sequences behind short prompts (4 to 16 over 4096 tokens; 4 over 32768 take the same time either way).  Sharing is faster beyond, where one
 * call takes several layers, and for 16-bit windows of rotated or bf16 caches.
 *  cu_groups: [n_groups + 1] int32, device, ascending from 0 to batch: group i is sequences [cu_groups[i], cu_groups[i + 1])
 *             (else KVQ_DEV_SEQ, and no rows are written).
 *  cu_q, total_q, max_q, seq_lens: as for kvq_chunk_attention (lengths INCLUDING the new tokens; pages for them are
 *             reserved; the tokens themselves may be appended later, before the attention of their layer).
 *  max_group_q: a host bound on the new tokens of any group, max_q <= max_group_q <= total_q (the larger it is, the more rows the
 *             kernel expects at a time).  A group with more sets KVQ_DEV_LENGTH and goes without its common prefix, as does a group with
 *             a sequence whose rows or length are out of order (KVQ_DEV_LENGTH; that sequence's rows are left as they are).
 * kvq_prefix_attention takes n_groups, total_q, max_q and max_group_q as the plan did (else KVQ_DEV_SEQ, and no rows are
 * written); q, out, roundings, values out of range and pages out of range as kvq_chunk_attention.
 *  workspace: kvq_prefix_workspace_bytes for `rows` = the largest total_q, 256-byte aligned,
 *             prepared once by kvq_prefix_workspace_init for the same n_groups and rows; holds the plan; calls that may run at the same
 *             time need one each.  Its first word is the device status word. */
KVQ_API kvq_status kvq_prefix_workspace_bytes(const kvq_config* cfg, int32_t n_groups, int32_t rows, size_t* bytes);
KVQ_API kvq_status kvq_prefix_workspace_init(const kvq_config* cfg, int32_t n_groups, int32_t rows, void* workspace,
                                             size_t ws_bytes, void* stream);
KVQ_API kvq_status kvq_prefix_plan(const kvq_config* cfg, const int32_t* block_table, const int32_t* cu_groups, int32_t n_groups,
                                   const int32_t* cu_q, int32_t total_q, int32_t max_q, int32_t max_group_q,
                                   const int32_t* seq_lens, void* workspace, size_t ws_bytes, void* stream);
KVQ_API kvq_status kvq_prefix_attention(const kvq_config* cfg, const kvq_cache* cache, int32_t layer0, int32_t n_layers,
                                        int32_t n_groups, const void* q, int32_t total_q, int32_t max_q, int32_t max_group_q,
                                        void* out, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
