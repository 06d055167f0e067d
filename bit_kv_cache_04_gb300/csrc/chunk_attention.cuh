// Attention of many new tokens over the packed cache (kvq_chunk_attention):
// shared definitions and the kernel.
//
// For one (layer, sequence, kv head) the query rows are its new tokens times
// the g query heads of the kv head, row r = token r / g, head r % g.  With S = Q K^T / sqrt(D),
//   m = max_j S_j, P_j = 2^(log2e (S_j - m)), l = sum_j P_j, out = P V / l,
// tile by tile of cached tokens with running m and l.  Both products run on
// the 5th-generation tensor cores (tcgen05.mma, accumulators in TMEM); keys
// and values are dequantized on the way from their packed blocks to the swizzled
// shared-memory tiles that the products read, so packed bytes are all that HBM delivers.
//
// One CTA per SM, specialized warps, joined by mbarriers:
//   softmax warps   one TMEM lane (query row) per thread: row maximum, exponentials, P back to
//                   TMEM in the input dtype, the accumulator's rescaling, outputs
//   loader warps    packed bytes of half tiles ("pieces") into a ring of slots, bulk copies
//   dequant warps   packed blocks -> K and V tiles in shared memory (2 stages each)
//   product warp    one thread issues every tcgen05.mma
// D = 128: tiles of 128 tokens and two streams of softmax warps, each with
// its own S and output accumulator, so that one stream's exponentials run
// under the other's products.  PAIRED (more than 128 rows a sequence): both
// streams take the same tokens and different rows (256 rows a CTA, a tile is
// dequantized once for both: two chunks of 2048 tokens over a 4096-token window 395 us, 695 TFLOP/s, twice
// as long unpaired).  Not PAIRED: the streams share the rows and take alternate tiles.
// D = 256: tiles of 64 tokens, 128 rows, one output accumulator and one group
// of softmax warps over two S buffers (TMEM holds no more).
// FEW (D = 128, at most 32 rows a sequence): rows are the products' columns, see the kernel.
// Otherwise rows are lanes, however few.  (Repeating few rows over the lanes, each copy with its share of a tile's tokens,
// gained nothing: 48 rows of 128 channels 301 us both ways, 48 rows of 256 channels 207 us against 165 us.)
//
// Roundings: values and P go to the input's 16-bit type, keys and turned queries to fp16 whatever that is: the
// tensor cores multiply nothing wider at this rate, and a key's rounding weighs most.  (Keys in bf16: 2-norm
// errors of 3.7e-3 with rotated keys and 5.3e-3 with per-channel ones that have outlier channels, where the output's own rounding is 1.7e-3.)
// Scores, row sums and outputs are fp32 until the last store.
//
// The tiles of all (layer, kv head, sequence, row tile) units form one line
// that is cut into equal runs, one per CTA, whatever the lengths; a unit cut
// by run ends leaves partial rows (O, m, l) in the workspace, and the CTA that
// takes the unit's last ticket joins them.  No CTA waits for another.
#pragma once

#include "block_codec.cuh"

namespace kvq {

// what a launch's rows ask of the kernel: at most 32 a sequence (D = 128); more than 128 (D = 128); else
constexpr int kChunkShared = 0, kChunkPaired = 1, kChunkFew = 2;
constexpr int kFewRows = 32;
constexpr uint32_t kFewBytes = kFewRows * 128 * 2;  // of a few queries, or of their P over a tile
constexpr int kChunkSlots = 3;       // partial slots per CTA: first cut unit, last cut unit, whole units
constexpr int kChunkTickets = 2;     // per CTA: units whose first run is the CTA's first or last one
constexpr int kChunkMaxSlots = 16;   // staging ring, in pieces
constexpr int kChunkBars = 8;        // barriers of one kind of piece: more tiles than the ring can span
constexpr int kChunkSpin = 1 << 20;  // polls after which a wait gives up (KVQ_DEV_STALL)
constexpr uint32_t kChunkPollNs = 2000;  // a poll's own wait, at most

KVQ_HD constexpr int chunk_tile(int D) { return D == 128 ? 128 : 64; }
KVQ_HD constexpr int chunk_streams(int D) { return D == 128 ? 2 : 1; }
KVQ_HD constexpr int chunk_slot_rows(int D) { return 128 * chunk_streams(D); }
KVQ_HD constexpr int chunk_part_row(int D) { return D + 4; }  // O, m, l, two pads

struct ChunkArgs {
  Layout lo;
  CachePtrs cp;
  int layer0, n_layers;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int total_q, max_q, window, sinks;
  int turn_here;  // rotated formats: the kernel turns the (few) queries itself; else a pass before it does
  int cols;     // few rows: columns of the products, 16 or 32
  uint32_t g_magic;  // floor(2^32 / g) + 1
  int by_warp;  // row tiles per sequence are many: count them with a warp per sequence
  int direct;       // 1: pages cannot be staged by bulk copies
  int small_pages;  // 1: pages of fewer than 32 tokens
  int copy_shift;   // log2 of the tokens of one copy: 5, less for small pages
  int sub_bytes;    // staged bytes of a 32-token subtile, the largest of the formats
  int slot_bytes;   // of a staged piece (half a tile of one tensor)
  int slots;        // pieces in the ring
  int stall_polls;  // > 0: failure-detection test mode (kvq_test_force_stall)
  uint32_t* status;
  uint32_t* left;       // CTAs that have finished, and in the upper half those that gave up; zero between calls
  uint32_t* tickets;    // [grid][kChunkTickets]
  uint32_t* nonfinite;  // [grid][kChunkTickets]: a 16-bit window value of the unit is not finite
  float* partials;      // [grid][kChunkSlots][slot rows][part row]
  float k_pre, q_pre;  // factors (powers of two) on a bf16 cache's keys and on turned queries
  float score_scale;   // log2(e) / sqrt(D), both factors undone
  uint32_t k_one;       // the fp16 number whose last bit counts k_pre, twice
  uint64_t turns[128];  // pre-RoPE keys: turns per position of every pair, 64-bit fractions
};

cudaError_t launch_chunk_d128(const ChunkArgs& a, int mode, int grid, cudaStream_t s);
cudaError_t launch_chunk_few(const ChunkArgs& a, int grid, cudaStream_t s);
cudaError_t launch_chunk_d256(const ChunkArgs& a, int grid, cudaStream_t s);

}  // namespace kvq
