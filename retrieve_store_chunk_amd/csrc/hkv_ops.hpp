// Kernel argument blocks and host-side launches of the operators that read
// and update the pool in place (MLA attention, eviction, the KDA step).
// Shared by the host checks (hkv_ops.cpp) and the kernels (plain structs, no
// HIP types).
#pragma once

#include <cstdint>

#include "hkv_device_tables.hpp"

namespace hkv {

// ---------------------------------------------------------------- attention
constexpr uint32_t kAttendTile = 32;        // cached tokens per step of a workgroup
constexpr uint32_t kAttendMaxWidth = 576;   // values per cached row
constexpr uint32_t kAttendMaxValues = 512;  // of them, values that are summed
constexpr uint32_t kAttendMaxWorkers = 256; // one workgroup per CU
// Rows of a call whose tables can hold more than the last-level cache are read
// past the caches (nontemporal): they cannot be there from the call before, and
// should not evict what is (1 sequence of 10^6 tokens, 32 heads: 191 us, 213
// without; 64 of up to 14001: 128, 140; 64 of up to 4000, 418 MB of tables: 53,
// 56).  Smaller calls are no slower, or faster, through the caches, with seven
// layers read in turn as in a decode loop (16 of up to 9000, 32 heads: 38.7 us,
// 38.2 past the caches; 16 of up to 2400, 64 heads: 27.6, 29.7; 4 of up to 9000,
// 32 heads: 23.6, 25.2; one layer again and again gains 3 us more).  With two
// head tiles both ways meet at the limit (16 of up to 20000, 64 heads, 383 MB:
// 73.9 us, 73.5; 64 of up to 4000: 70.5, 72.2).
constexpr uint64_t kAttendStreamBytes = uint64_t(256) << 20;

// One call's geometry as the host plans it and the kernels follow it.
struct AttendArgs {
  const uint8_t* pages;  // the layer's page of block 0
  uint64_t stride;       // bytes between block ids
  const void* q;         // [n_seqs][n_heads][width]
  int64_t q_seq_stride, q_head_stride;  // elements
  const int32_t* table;  // [n_seqs][max_blocks]
  int64_t table_stride;
  const int32_t* lens;   // [n_seqs]
  void* out;             // [n_seqs][n_heads][values]
  int64_t out_seq_stride, out_head_stride;
  float* lse;            // [n_seqs][n_heads], natural log, or nullptr
  float* weights;        // [n_seqs][weights_stride], or nullptr
  int64_t weights_stride;
  // workspace
  float* part_o;         // [workers][head tiles][2][head tile][values]
  float* part_ml;        // [workers][head tiles][2][head tile][2]: maximum, sum
  int32_t* spans;        // [n_seqs][4]: first worker, last worker, slot of the first
  float* norm;           // [n_seqs][n_heads] the lse that weights subtract (weights only)
  float* logits;         // [n_seqs][max_tiles][n_heads][kAttendTile] (weights only)
  float scale;           // softmax scale x cache scale
  float cache_scale;
  uint32_t num_blocks, block_tokens, row_bytes, width, values;
  uint32_t n_seqs, n_heads, head_tile, head_tiles, max_blocks, workers;
  uint32_t streams;      // rows are read past the caches
  uint32_t join_shift;   // lanes a joining group has (log2)
  uint32_t max_tiles;    // tiles of the longest sequence the table can hold
};

// Heads one workgroup takes.  `units`: the tiles that the tables can hold, times
// the groups of 16 heads, which is as much as the host knows of a call's size.
// More heads to a workgroup read a row from L2 and from LDS for fewer
// workgroups, but make its rounds longer and the partial results of a short
// call more: with 16 heads, 32 and 64 to a workgroup
//   1 sequence of 1000 tokens, 64 heads: 14.4, 15.5, 19.3 us
//   16 of up to 2400: 28.1, 29.1, 37.6 (7600 units)
//   16 of up to 4800: 37.6, 34.0, 43.9 (11000)
//   16 of up to 20000: 101.7, 75.8, 82.7 (42000); 40000: 182.8, 128.0, 125.5
// An e4m3 cache has half the bytes to wait for in a round and turns earlier
// (16 of up to 9600: 58.4, 45.5, 47.1 at 20000 units; 14000: 76.5, 56.7, 55.0 at
// 29000; 20000: 102.7, 70.3, 65.5).
inline constexpr uint32_t attend_head_tile(uint32_t n_heads, uint64_t units, bool fp8) {
  const uint32_t most = units <= 8192 ? 16u : units <= (fp8 ? 24576u : 49152u) ? 32u : 64u;
  const uint32_t need = n_heads <= 16 ? 16u : n_heads <= 32 ? 32u : 64u;
  return need < most ? need : most;
}

// Tiles per worker: an even share of all tiles, down to one, but three instead
// of two: a worker's start and the joining of its result cost about as much as
// a tile, so that a third fewer of them outweigh one more tile each (1 sequence
// of 16000 tokens: 18.9 us for 20.0 with 16 heads, 28.3 for 30.3 with 64; 24 of
// 700: 18.7 for 20.0).  More than that is no gain where the tiles are few (4
// sequences of 2300 tokens, 16 heads: 16.5 us with one tile each, 17.7 with
// three, 19.4 with four).
inline constexpr uint64_t attend_share(uint64_t tiles, uint64_t workers) {
  const uint64_t s = (tiles + workers - 1) / workers;
  return s == 2 ? 3 : s;
}

// Workspace sections, each on a 256-byte boundary.
struct AttendWorkspace {
  uint64_t part_o, part_ml, spans, norm, logits, total;
};
inline AttendWorkspace attend_workspace(uint64_t workers, uint64_t head_tiles, uint64_t head_tile,
                                        uint64_t values, uint64_t n_seqs, uint64_t n_heads,
                                        uint64_t max_tiles, bool weights) {
  AttendWorkspace w{};
  const uint64_t slots = workers * head_tiles * 2 * head_tile;
  w.part_o = 0;
  w.part_ml = w.part_o + align256(slots * values * sizeof(float));
  w.spans = w.part_ml + align256(slots * 2 * sizeof(float));
  w.norm = w.spans + align256(n_seqs * 4 * sizeof(int32_t));
  w.logits = w.norm + (weights ? align256(n_seqs * n_heads * sizeof(float)) : 0);
  w.total = w.logits +
            (weights ? align256(n_seqs * max_tiles * n_heads * kAttendTile * sizeof(float)) : 0);
  return w;
}

// Enqueues the attention of one call on `stream` (a hipStream_t).  dtype and
// cache_dtype: HKV_BF16, HKV_FP16, HKV_E4M3.  Returns the hipError_t.
int launch_attend(const AttendArgs& a, int32_t dtype, int32_t cache_dtype, void* stream);

// ---------------------------------------------------------------- eviction
constexpr uint32_t kEvictMaxLayers = 64;
constexpr uint32_t kEvictSelectSlots = 16384;  // a row's slots that one workgroup takes
constexpr uint32_t kEvictChunkSlots = 8192;    // slots of a longer row per workgroup
// Block ids are checked pair by pair, by every workgroup for its sequence, up to
// this many of one sequence and this many pairs for it; beyond by counting in the
// workspace, a launch of one workgroup (16 sequences of 128 blocks of 16 tokens:
// 18 us for the call, 32 when counted; at the limit, 4 of 512: 37 and 40, 1 of
// 1024: 38 and 45; pairs grow with the square).
constexpr uint32_t kEvictPairBlocks = 1024;
constexpr uint64_t kEvictPairs = uint64_t(1) << 20;

struct EvictArgs {
  uint8_t* pool;
  uint64_t page_of[kEvictMaxLayers];  // each layer's page of block 0, from the pool's start
  uint64_t stride;       // bytes between block ids
  const int32_t* table;  // [n_seqs][max_blocks]
  int64_t table_stride;
  const int32_t* lens;   // [n_seqs]
  const int32_t* next;   // [n_seqs]
  const float* weights;  // [n_layers][n_seqs][slots], these four
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int64_t layer_stride, seq_stride;  // elements
  int32_t* new_lens;     // [n_seqs] or nullptr
  // workspace
  int32_t* claims;       // [num_blocks] uses of a block by the call's sequences
  int32_t* ok;           // [n_seqs] 1: the sequence can be evicted from
  uint32_t* moves;       // [rows]: slots that move
  uint32_t* lists;       // [rows][2 * max_moves]: freed slots, then the slots that fill them
  uint32_t* hist;        // long rows: [rows][3][2048] keys by digit
  uint32_t* totals;      // long rows: [rows][chunks][2] keys above the least kept, ties with it
  uint32_t* least;       // long rows: [rows][3][2] after each digit: the least kept key so far,
                         // how many keys that match it stay
  uint32_t num_blocks, block_tokens, row_bytes;
  uint32_t n_layers, n_seqs, max_blocks, budget, sinks, recent;
  uint32_t max_moves;    // min(budget, max_blocks * block_tokens - budget)
  uint32_t chunks;       // of a long row's slots; 0: rows are short
  uint32_t by_pairs;     // how the block ids are checked
};

struct EvictWorkspace {
  uint64_t claims, ok, moves, lists, hist, totals, least, total;
};
inline EvictWorkspace evict_workspace(uint64_t num_blocks, uint64_t n_seqs, uint64_t rows,
                                      uint64_t max_moves, uint64_t chunks, bool by_pairs) {
  EvictWorkspace w{};
  w.claims = 0;
  w.ok = w.claims + (by_pairs ? 0 : align256(num_blocks * 4));
  w.moves = w.ok + align256(n_seqs * 4);
  w.lists = w.moves + align256(rows * 4);
  w.hist = w.lists + align256(rows * 2 * max_moves * 4);
  w.totals = w.hist + (chunks ? align256(rows * 3 * 2048 * 4) : 0);
  w.least = w.totals + align256(rows * chunks * 2 * 4);
  w.total = w.least + (chunks ? align256(rows * 3 * 2 * 4) : 0);
  return w;
}

int launch_evict(const EvictArgs& a, void* stream);

// ---------------------------------------------------------------- KDA step
constexpr uint32_t kKdaMaxKernel = 8;   // conv taps
constexpr uint32_t kKdaMaxSeqs = 4096;  // every workgroup looks through the call's block ids

struct KdaArgs {
  uint8_t* pages;        // the layer's page of block 0
  uint64_t stride;       // bytes between block ids
  uint64_t conv_bytes;   // the recurrent state's offset in a page
  const void* x;         // [n_seqs][conv_dim]
  int64_t x_stride;      // elements, as the other strides
  const void* conv_weight;  // [conv_dim][taps]
  const float* log_decay;   // [n_seqs][heads * d]
  int64_t decay_stride;
  const float* beta;        // [n_seqs][heads]
  int64_t beta_stride;
  const int32_t* src;       // [n_seqs]
  const int32_t* dst;
  void* out;                // [n_seqs][heads * d]
  int64_t out_stride;
  float scale, eps;
  uint32_t num_blocks, n_seqs, heads, head_dim, taps;
};

int launch_kda(const KdaArgs& a, int32_t dtype, void* stream);

// ---------------------------------------------------------------- append
constexpr uint32_t kAppendMaxWidth = 1024;          // a wave holds a row: 16 values a lane
constexpr int32_t kPromptMaxTokens = 1 << 20;       // rows of a call

struct AppendArgs {
  uint8_t* pages;        // the layer's page of block 0
  uint64_t stride;       // bytes between block ids
  const void* kv;        // [n_tokens][width]
  int64_t kv_stride;     // elements, as the other strides
  const void* norm;      // [latent] or nullptr
  const float* cos_sin;  // [n_positions][rotary]
  const int32_t* positions;  // [n_tokens]
  const int32_t* starts;     // [n_seqs + 1] or nullptr
  const int32_t* lens;       // [n_seqs]
  const int32_t* table;      // [n_seqs][max_blocks]
  int64_t table_stride;
  const void* q_in;          // [n_tokens][n_heads][rotary]
  int64_t q_in_token, q_in_head;
  void* q_out;
  int64_t q_out_token, q_out_head;
  float eps, cache_scale;
  uint32_t num_blocks, block_tokens, max_blocks, n_seqs, n_tokens, n_positions;
  uint32_t n_heads, width, latent, rotary, halves, cache_bytes;
};

int launch_append(const AppendArgs& a, int32_t dtype, void* stream);

// ---------------------------------------------------------------- KDA prefill
constexpr uint32_t kPrefillChunk = 64;       // tokens
constexpr uint32_t kPrefillChunkDim = 128;   // the head dim that is computed in chunks
constexpr uint32_t kPrefillRecord = 3 * 32768 + 12288 + 32768 + 1024;  // bytes of a chunk and head

// Calls whose longest run has up to so many tokens go token by token (us, token by token
// and in chunks: 61 runs of up to 16 tokens, 6 heads 45, 67; 24 62, 68; 32 79, 73; 61 runs
// of 32 heads, which fill the card either way, 24 167, 290; 48 305, 297; 16 runs of 6 heads
// 24 38, 38; 32 49, 38; of 32 heads 24 58, 71; 32 73, 72; 4 runs, 6 or 32 heads 16 27, 30
// and 38; 24 37, 30 and 38; one run of 12 21, 27; 16 26, 26; 24 37, 27).  In others, runs
// of up to kPrefillShort do, in a launch of their own (24 runs of one token beside 4 prompts of up to 1400, 32 heads: 256
// us; 331 with all in chunks; 61 runs of up to 12, all in chunks but those: 73 with 2, 74 with
// 4, 65 with 8; of up to 16 66, 72 and 69; of up to 32 73, 72 and 83).  A call of one sequence has no such launch.
constexpr uint32_t kPrefillTokens = 24, kPrefillTokensOne = 16;
constexpr uint32_t kPrefillShort = 2;
// Runs are cut into parts where that makes at least 4 with one workgroup a CU, from so many
// tokens of the longest on (us in all, one part and cut: 1500 tokens, 6 heads 64, 60; 16384
// 488, 279 to 291; with 16 heads, which leave room for 3 parts, 1887 tokens 83, 80, and 90 in 4).  8 at most.
// The room counts all sequences of the call, short ones too, since the host does not know
// which are: beside single tokens a long run is not cut (16384 tokens, 6 heads 285 alone,
// 504 beside one token, 638 beside 8, 648 beside 30).
constexpr uint32_t kPrefillPartTokens = 1200;

// Up to so many sequences are looked through by every workgroup of the token-by-token
// kernel itself, a launch less (us with and without: 61 of one token, 6 heads 12.8, 16.5;
// 256 42.4, 43.0; 256 of 16 heads 128.6, 125.7; 512 of 16 heads 240, 232; 1000 of 6 196, 183).
constexpr uint32_t kPrefillLookThrough = 256;

// Block ids are compared pair by pair up to so many whole blocks in the call's rows
// (n_tokens / N), by counting in the workspace beyond: two launches more, but pairs grow
// with the square, up to 2^30 for one thread (us in all, N = 16, one head of 128, counted and
// compared: 2 runs of 8 blocks each 44, 46; of 16 59, 77; of 128 313, 1632; 8 runs of 2 36,
// 32; of 4 41, 36; of 8 49, 49; one of 16 54, 51; of 64 148, 149).
constexpr uint32_t kPrefillPairBlocks = 24;

struct PrefillChunk {
  int32_t seq, row, len, off;  // its first token: row of the call, token of the sequence
  int32_t dst;                 // the block that its last token's state goes to, or none
  int32_t pad[3];
};

struct PrefillArgs {
  uint8_t* pages;        // the layer's page of block 0
  uint64_t stride;       // bytes between block ids
  uint64_t conv_bytes;   // the recurrent state's offset in a page
  const void* x;         // [n_tokens][conv_dim]
  int64_t x_stride;      // elements, as the other strides
  const void* conv_weight;  // [conv_dim][taps]
  const float* log_decay;   // [n_tokens][heads * d]
  int64_t decay_stride;
  const float* beta;        // [n_tokens][heads]
  int64_t beta_stride;
  const int32_t* starts;    // [n_seqs + 1]
  const int32_t* positions; // [n_seqs]
  const int32_t* src;       // [n_seqs]
  const int32_t* table;     // [n_seqs][max_blocks]
  int64_t table_stride;
  void* out;                // [n_tokens][heads * d]
  int64_t out_stride;
  float scale, eps;
  uint32_t num_blocks, block_tokens, max_blocks, n_seqs, n_tokens, max_seq_tokens;
  uint32_t heads, head_dim, taps;
  uint32_t counted;         // the uses of blocks are counted, not compared
  uint32_t planned;         // a launch of its own looks the sequences through
  uint32_t chunked;         // sequences of more than short_tokens are computed in chunks
  uint32_t short_tokens;
  uint32_t max_chunks;
  uint32_t column_tiles;    // of 16 columns a scanning workgroup, 1 or 2
  uint32_t parts;           // that a sequence's chunks are cut into: 1, or 4 to 8
  // workspace
  int32_t* status;          // [n_seqs]: kPrefill* below
  uint32_t* uses;           // [num_blocks][2]: entries and sources that name a block, if counted
  int32_t* first_chunk;     // [2][n_seqs], [1]: each sequence's first, how many; all of them
  PrefillChunk* chunks;     // [max_chunks]
  uint8_t* records;         // [max_chunks][heads][kPrefillRecord]
  float* made;              // [n_seqs][heads][parts - 1][2][128][128], where there are parts
};

// What becomes of a sequence.
constexpr int32_t kPrefillRuns = 0;
constexpr int32_t kPrefillRefused = 1;  // NaN in its rows, no page
constexpr int32_t kPrefillNoRows = 2;   // nothing to do, or its rows are not known

struct PrefillWorkspace {
  uint64_t status, uses, first_chunk, chunks, records, made, total;
};
// `counted_blocks`: the pool's, where their uses are counted, else 0.
inline PrefillWorkspace prefill_workspace(uint64_t n_seqs, uint64_t max_chunks, uint64_t heads,
                                          uint64_t parts, uint64_t counted_blocks) {
  PrefillWorkspace w{};
  w.uses = w.status + align256(n_seqs * 4);
  w.first_chunk = w.uses + align256(counted_blocks * 8);
  w.chunks = w.first_chunk + (max_chunks ? align256((2 * n_seqs + 1) * 4) : 0);
  w.records = w.chunks + align256(max_chunks * sizeof(PrefillChunk));
  w.made = w.records + max_chunks * heads * kPrefillRecord;
  w.total = w.made + n_seqs * heads * (parts > 1 ? (parts - 1) * 2 : 0) * kPrefillChunkDim *
                         kPrefillChunkDim * 4;
  return w;
}

int launch_prefill(const PrefillArgs& a, int32_t dtype, void* stream);

}  // namespace hkv
