// MLA attention of one new token per sequence over the paged latent cache
// (gfx950).
//
// For a sequence's cached rows k_t (width values each; the first `values` of
// them are also v_t) and a head's query q_h:
//   s_ht = scale * cache_scale * q_h . k_t
//   o_h  = cache_scale * sum_t exp(s_ht - m) v_t / sum_t exp(s_ht - m)
// in one pass over the rows: the running maximum m and sum l of each head are
// kept in fp32, and a new maximum rescales what was summed before.
//
// All heads share the rows, so a tile of 32 rows staged in LDS serves both
// products for every head of the workgroup:
//   S = K Q^T   (rows = tokens, columns = heads; Q stays in registers)
//   O^T += V^T P^T   (V^T read from the same LDS rows by transposing loads)
// with 16x16x32 matrix instructions and fp32 accumulators.  P is split into
// two 16-bit terms (p = hi + lo, about 16 significant bits for bf16), because
// one rounding of P to 16 bits would be as large as the rounding of the
// output itself.  An e4m3 cache's rows are widened to the query's type as they
// are staged, which is exact.  (For a bf16 query fp16 products with one term of
// P took 103 us for 113 on the e4m3 case below, but P then has 11 bits, and a
// query scaled by a power of two to fit fp16 loses what is 2^31 below its
// largest value.)
//
// Bound: reading the cache once (row_bytes per token).  The waves have roles,
// so that loads, both products and the softmax of different tiles overlap:
// scorers (one for 16 heads) turn a tile into P, 8 carriers load rows and sum
// values.  In the round between two barriers tile i + 1 goes to LDS, tile i is
// scored, tile i - 1 is summed (three row buffers), and the rows of tiles i + 2
// and i + 3 are on their way in the carriers' registers.  (1 sequence of 10^6
// tokens, 32 heads: 273 us when all waves loaded, scored and summed in turn, 220
// with roles; a round is 1.5 us now.)  LDS rows are padded to an odd multiple
// of 32 bytes, so that eight rows at the same column, and four rows of the
// transposing loads, start in different banks; counters still show a quarter of
// the LDS's active cycles lost to conflicts, a third with e4m3 rows.
//
// The batch's tiles, all sequences after one another, are cut into equal
// runs, one per worker (workgroup): a million-token sequence and a ragged batch
// both fill the card, and no length is needed on the host.  Null blocks count in
// the cut and are skipped only then, so that runs over dropped blocks end early
// and the others carry the call (24 sequences of up to 40000, 64 heads, e4m3: 161
// us whole, 93 with two blocks of every three null, 128 with the oldest two
// thirds null).  A worker whose run covers part of a sequence leaves a partial
// result (m, l, unnormalised O) that hkv_mla_attend_join adds up.
//
// Measured: 64 ragged sequences of up to 14001 tokens, 32 heads, bf16 (648 MB)
// 126 us, 5.1 TB/s; 1 of 10^6 tokens (1.15 GB) 192 us, 6.0 TB/s, what a torch
// sum of 4 GiB reaches (the best reading kernel here 7.4); 24 of up to 40000, 64
// heads, e4m3, a third of the blocks null (229 MB, 55 GFLOP) 113 us, where no unit
// is full (LDS active 54% of the time, matrix units 40%) and a round waits for its
// chain of widening, score, softmax and sum; 1 of 333 tokens 12 us, two launches
// and one round.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))
#define HKV_LDS __attribute__((address_space(3)))
#define HKV_CONST __attribute__((address_space(4)))

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr uint32_t kTile = hkv::kAttendTile;
constexpr uint32_t kWidthSteps = hkv::kAttendMaxWidth / 32;   // k steps of S
constexpr uint32_t kValueTiles = hkv::kAttendMaxValues / 16;  // 16-column tiles of O
constexpr uint32_t kPitch = hkv::kAttendMaxWidth * 2 + 32;  // bytes of a row in LDS
constexpr uint32_t kPPitch = kTile * 2 + 16;  // bytes of a P row (padded: 16-byte reads of
                                              // eight rows fall into different banks)
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

// exp(x) of a difference of logits: the difference is taken first, so that the
// rounding of the conversion to powers of two is relative to it and not to
// the logits.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

struct Bf16 {
  static __device__ __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const v2b r = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ float low(uint32_t u) {
    return __builtin_bit_cast(float, u << 16);
  }
  static __device__ __forceinline__ float high(uint32_t u) {
    return __builtin_bit_cast(float, u & 0xFFFF0000u);
  }
  template <bool kHigh>
  static __device__ __forceinline__ uint32_t widen(uint32_t u) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.0f, kHigh));
  }
};

struct Fp16 {
  static __device__ __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const v2h r = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ float low(uint32_t u) {
    return (float)__builtin_bit_cast(v2h, u)[0];
  }
  static __device__ __forceinline__ float high(uint32_t u) {
    return (float)__builtin_bit_cast(v2h, u)[1];
  }
  template <bool kHigh>
  static __device__ __forceinline__ uint32_t widen(uint32_t u) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, kHigh));
  }
};

__device__ __forceinline__ uint32_t uniform(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
}

__device__ __forceinline__ float lane_xor(float x, int mask) {
  return __shfl_xor(x, mask, 64);
}

// The same value, but unknown to the compiler: what is computed from it inside
// a loop stays there.  Used for addresses that a sequence needs once, which
// would otherwise be kept in registers throughout the loop over the tiles.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Orders LDS accesses across the workgroup; global loads may stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// lse = ln of the sum of exp(logits); -inf where nothing is live.  The weights
// kernel subtracts norm: +inf there, so that exp(-inf - norm) is 0.
__device__ __forceinline__ void write_lse(const hkv::AttendArgs& a, uint32_t s, uint32_t h,
                                          float top, float sum) {
  const float lse = sum == 0.0f ? -INFINITY : top + __builtin_amdgcn_logf(sum) * kLn2;
  if (a.lse) a.lse[(uint64_t)s * a.n_heads + h] = lse;
  if (a.norm) a.norm[(uint64_t)s * a.n_heads + h] = sum == 0.0f ? INFINITY : lse;
}

// A sequence's length if it can be served, else 0 (the join writes NaN for a
// length outside [0, max_blocks * block_tokens]).
__device__ __forceinline__ uint32_t served_len(const hkv::AttendArgs& a, uint32_t s) {
  const int32_t len = a.lens[s];
  return len < 0 || (uint64_t)len > (uint64_t)a.max_blocks * a.block_tokens ? 0u : (uint32_t)len;
}

__device__ __forceinline__ uint32_t tiles_of(uint32_t len) { return (len + kTile - 1) / kTile; }

// A tile has two groups of 16 rows.  A block is a multiple of 16 tokens, so a
// group lies in one page.
enum RowState : uint32_t {
  kPresent = 0,
  kAbsent = 1,  // a null block, or past the sequence's end
  kBad = 2      // a block id outside the pool
};

// The states of a tile's two groups in one word.
constexpr uint32_t kBothAbsent = kAbsent | kAbsent << 2;
__device__ __forceinline__ uint32_t state_of(uint32_t st, uint32_t group) {
  return st >> (2 * group) & 3;
}

// Where the two row groups of a tile are: their entries of the block table,
// their first token's place in the block, and the blocks' ids (asked for a
// tile early).
struct Cursor {
  uint32_t j[2], off[2];
  int32_t id[2];
};

// Largest value over the lanes that hold one column of a 16x16 result (lane,
// lane ^ 16, lane ^ 32, lane ^ 48), and their sum.  The swaps exchange half the
// rows of 16 (32) lanes of one register with the other half of a second: given
// two copies of a value they leave both partners' values, without LDS.  (The
// builtins' second result comes out equal to the first with this compiler.)
__device__ __forceinline__ float column_max(float m) {
  float x = m, y = m;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  m = fmaxf(x, y);
  x = m;
  y = m;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return fmaxf(x, y);
}
__device__ __forceinline__ float column_sum(float m) {
  m += lane_xor(m, 16);
  return m + lane_xor(m, 32);
}

// The waves' roles: one scorer per 16 heads takes their logits and
// probabilities, kCarriers bring rows into LDS and add up the values.
constexpr uint32_t kCarriers = 8;
constexpr uint32_t attend_threads(uint32_t heads) { return (heads / 16 + kCarriers) * 64; }

// T: the type of q, of out and of both products' operands (it holds every e4m3
// value exactly).
template <class T, bool kFp8, uint32_t kHeads>
struct Attend {
  // P in fp16 is taken 2^15 times as large (P <= 1), and O with it: beside a
  // weight of 1, fp16 would round those below 2^-14 ever more coarsely and lose
  // those below 2^-25, which a long sequence holds many of.
  static constexpr float kUp = std::is_same_v<T, Fp16> ? 32768.0f : 1.0f;
  static constexpr uint32_t kHeadTiles = kHeads / 16;
  static constexpr uint32_t kScorers = kHeadTiles;
  static constexpr uint32_t kWaves = kScorers + kCarriers;
  static constexpr uint32_t kThreads = attend_threads(kHeads);
  static_assert(kThreads == kWaves * 64, "the launch has a wave for every role");
  static constexpr uint32_t kOTiles = kValueTiles / kCarriers;  // column tiles per carrier
  // A carrier loads half of 8 of a tile's rows, 8 lanes to a row, 16 bytes to a
  // lane and load.
  static constexpr uint32_t kLoads = (hkv::kAttendMaxWidth * (kFp8 ? 1 : 2) / 16 + 15) / 16;
  static_assert(kCarriers / 2 * 8 == kTile, "8 rows to two carriers");
  static constexpr uint32_t kAhead = 5;    // k steps a scorer reads ahead
  static constexpr uint32_t kBuffers = 3;  // a tile is loaded, scored and summed in turn
  static constexpr uint32_t kTileSlots = 4;

  // A tile on its way: this lane's pieces, which tile, its groups' states.
  struct Stage {
    v4u x[kLoads];
    uint32_t t, st;
  };

  // The small arrays come first: the LDS instructions' 16-bit offsets reach
  // them, and the first row buffer, from one register.
  struct Lds {
    uint32_t tile[kTileSlots][2];  // which tile the i-th is, its groups' states
    uint8_t p_hi[2][kHeads * kPPitch];
    uint8_t p_lo[2][kHeads * kPPitch];
    float alpha[2][kHeads];
    float m[kHeads], l[kHeads];
    uint32_t sums[kWaves];
    uint32_t start[2];
    __align__(16) uint8_t k[kBuffers][kTile * kPitch];
  };

  // Asks for the ids of a tile's blocks (scalar loads: they are not in the
  // way of the row loads, which are waited for in order).
  static __device__ __forceinline__ void fetch_ids(const HKV_CONST int32_t* table, uint32_t t,
                                                   uint32_t end, Cursor* c) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
      c->id[i] = table[t * kTile + i * 16 < end ? c->j[i] : 0];
  }
  static __device__ __forceinline__ void place(const hkv::AttendArgs& a, uint32_t t, Cursor* c) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      c->j[i] = (t * kTile + i * 16) / a.block_tokens;
      c->off[i] = (t * kTile + i * 16) - c->j[i] * a.block_tokens;
    }
  }
  // The states of tile t's groups.
  static __device__ __forceinline__ uint32_t states(const hkv::AttendArgs& a, uint32_t t,
                                                    uint32_t end, const Cursor& c) {
    uint32_t st = 0;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t id = (uint32_t)c.id[i];
      const uint32_t x = t * kTile + i * 16 >= end || id == (uint32_t)HKV_NULL_BLOCK ? kAbsent
                         : id < a.num_blocks                                         ? kPresent
                                                                                     : kBad;
      st |= x << (2 * i);
    }
    return st;
  }
  // From tile t (its ids fetched) to the first tile that holds anything, or to
  // t1: a null block costs one look at the table, not a tile's work for each
  // of its tiles.
  static __device__ __forceinline__ uint32_t find_tile(const hkv::AttendArgs& a,
                                                       const HKV_CONST int32_t* table,
                                                       uint32_t t, uint32_t t1, uint32_t end,
                                                       Cursor* c, uint32_t* st) {
    uint32_t now = states(a, t, end, *c);
    while (now == kBothAbsent && t < t1) {
      const uint64_t next = (uint64_t)(c->j[1] + 1) * a.block_tokens / kTile;
      t = next < t1 ? (uint32_t)next : t1;
      place(a, t, c);
      fetch_ids(table, t, end, c);
      now = states(a, t, end, *c);
    }
    *st = now;
    return t;
  }

  // Where this wave's rows of tile t are.  What is absent reads the pool's first
  // bytes instead and is put to zero in stage_tile, so that the loads need no
  // branch and 0 x anything the memory holds never reaches a sum.
  static __device__ __forceinline__ const uint8_t* rows_of(const hkv::AttendArgs& a,
                                                           const Cursor& c, uint32_t st,
                                                           uint32_t carrier) {
    const uint32_t g = carrier >> 1 & 1;
    const uint32_t id = (uint32_t)(g ? c.id[1] : c.id[0]), off = g ? c.off[1] : c.off[0];
    const uint8_t* base = a.pages;
    if (state_of(st, g) == kPresent)
      base += (uint64_t)id * a.stride + (uint64_t)off * a.row_bytes;
    return base;
  }

  template <bool kStream>
  static __device__ __forceinline__ void load_rows(const hkv::AttendArgs& a, const uint8_t* base,
                                                   uint32_t carrier, uint32_t lane, v4u* x) {
    const uint32_t row = (carrier & 1) * 8 + lane / 8, pieces = a.row_bytes / 16;
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      const uint32_t k = ((carrier >> 2) + i * 2) * 8 + (lane & 7);
      const HKV_GLOBAL v4u* from =
          (const HKV_GLOBAL v4u*)((const HKV_GLOBAL uint8_t*)base +
                                  (k < pieces ? row * a.row_bytes + k * 16 : 0));
      x[i] = kStream ? __builtin_nontemporal_load(from) : *from;
    }
  }

  // Writes the loaded pieces to LDS, widening e4m3.
  static __device__ __forceinline__ void stage_tile(const hkv::AttendArgs& a, uint32_t end,
                                                    uint32_t carrier, uint32_t lane, uint32_t t,
                                                    uint32_t st, const v4u* x,
                                                    HKV_LDS uint8_t* lds) {
    const uint32_t row = (carrier & 3) * 8 + lane / 8, pieces = a.row_bytes / 16;
    const bool live =
        state_of(st, carrier >> 1 & 1) == kPresent && t * kTile + row < end;
    const bool all_live = __all(live);
    HKV_LDS uint8_t* d = lds + row * kPitch;
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      const uint32_t k = ((carrier >> 2) + i * 2) * 8 + (lane & 7);
      v4u v = x[i];
      if (!all_live) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = live ? v[e] : 0u;
      }
      if (k >= pieces) continue;
      if constexpr (kFp8) {
        const v4u lo = {T::template widen<false>(v[0]), T::template widen<true>(v[0]),
                        T::template widen<false>(v[1]), T::template widen<true>(v[1])};
        const v4u hi = {T::template widen<false>(v[2]), T::template widen<true>(v[2]),
                        T::template widen<false>(v[3]), T::template widen<true>(v[3])};
        HKV_LDS v4u* to = (HKV_LDS v4u*)(d + k * 32);
        to[0] = lo;
        to[1] = hi;
      } else {
        *(HKV_LDS v4u*)(d + k * 16) = v;
      }
    }
  }

  // The first sequence and the first tile of it that this worker's run holds,
  // and every worker's share: a scan of the batch's tile counts.
  static __device__ __forceinline__ void find_run(const hkv::AttendArgs& a, Lds& lds,
                                                  uint32_t worker, uint64_t* first,
                                                  uint64_t* share, uint64_t* total, uint32_t* seq,
                                                  uint64_t* seq_start) {
    const uint32_t t = threadIdx.x, per = (a.n_seqs + kThreads - 1) / kThreads;
    const uint32_t lo = t * per < a.n_seqs ? t * per : a.n_seqs;
    const uint32_t hi = lo + per < a.n_seqs ? lo + per : a.n_seqs;
    uint32_t mine = 0;
    for (uint32_t s = lo; s < hi; ++s) mine += tiles_of(served_len(a, s));
    uint32_t scan = mine;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = __shfl_up(scan, d, 64);
      if ((t & 63) >= (uint32_t)d) scan += up;
    }
    if ((t & 63) == 63) lds.sums[t >> 6] = scan;
    __syncthreads();
    uint32_t before = scan - mine, all = 0;
    for (uint32_t w = 0; w < kWaves; ++w) {
      if (w < (t >> 6)) before += lds.sums[w];
      all += lds.sums[w];
    }
    *total = all;
    *share = hkv::attend_share(all, a.workers);
    *first = *share * worker;
    if (*first >= before && *first < (uint64_t)before + mine) {
      uint32_t s = lo, at = before;
      for (;; ++s) {
        const uint32_t n = tiles_of(served_len(a, s));
        if (*first < (uint64_t)at + n) break;
        at += n;
      }
      lds.start[0] = s;
      lds.start[1] = at;
    }
    __syncthreads();
    *seq = uniform(lds.start[0]);
    *seq_start = uniform(lds.start[1]);
  }

  // The roles' parts of one run of tiles [t0, t1) of a sequence.  Round i (the
  // time between two barriers): the carriers write tile i + 1 to its buffer and
  // add tile i - 1, the scorers make P of tile i.  "Tile i" counts tiles that
  // hold anything; the carriers say in lds.tile which one it is, a round before
  // it is scored, and rounds go in pairs.

  // Adds a tile: O^T of this wave's value columns (those past `values` are not
  // written out) x all heads.  Transposing loads: in each group of 16 lanes,
  // lane x supplies four columns of token x / 4 and receives column x of four
  // tokens.
  static __device__ __forceinline__ void add_tile(Lds& lds, uint32_t buf, uint32_t half,
                                                  uint32_t carrier, uint32_t lane,
                                                  v4f (&acc)[kHeadTiles][kOTiles]) {
    const uint32_t col = lane & 15, quad = lane >> 4;
    const HKV_LDS uint8_t* vb = (const HKV_LDS uint8_t*)lds.k[buf] +
                                (quad * 8 + (col >> 2)) * kPitch + (col & 3) * 8 + carrier * 32;
    // Everything is read before anything is used: one wait instead of one for
    // each read.
    const HKV_LDS uint8_t* hi = (const HKV_LDS uint8_t*)lds.p_hi[half] + col * kPPitch + quad * 16;
    const HKV_LDS uint8_t* lo = (const HKV_LDS uint8_t*)lds.p_lo[half] + col * kPPitch + quad * 16;
    float alpha[kHeadTiles];
    bool moved = false;
    v4u v[kOTiles], p[kHeadTiles];
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i) alpha[i] = lds.alpha[half][i * 16 + col];
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i) p[i] = *(const HKV_LDS v4u*)(hi + i * 16 * kPPitch);
#pragma unroll
    for (uint32_t j = 0; j < kOTiles; ++j) {
      const HKV_LDS uint8_t* from = vb + j * kCarriers * 32;
      const v2u x = __builtin_bit_cast(
          v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((HKV_LDS v4s*)from));
      const v2u y = __builtin_bit_cast(
          v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((HKV_LDS v4s*)(from + 4 * kPitch)));
      v[j] = v4u{x[0], x[1], y[0], y[1]};
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i) moved |= alpha[i] != 1.0f;
    if (__any(moved)) {  // rare once the maxima have settled
#pragma unroll
      for (uint32_t i = 0; i < kHeadTiles; ++i)
#pragma unroll
        for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] *= alpha[i];
    }
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i) {
#pragma unroll
      for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] = T::mma(v[j], p[i], acc[i][j]);
      p[i] = *(const HKV_LDS v4u*)(lo + i * 16 * kPPitch);
    }
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i)
#pragma unroll
      for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] = T::mma(v[j], p[i], acc[i][j]);
  }

  template <bool kStream>
  static __device__ __forceinline__ void carry(const hkv::AttendArgs& a, Lds& lds,
                                               uint32_t carrier, uint32_t lane,
                                               const HKV_CONST int32_t* table, uint32_t t0,
                                               uint32_t t1, uint32_t end,
                                               v4f (&acc)[kHeadTiles][kOTiles]) {
#pragma unroll
    for (uint32_t i = 0; i < kHeadTiles; ++i)
#pragma unroll
      for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    Cursor cur;
    place(a, t0, &cur);
    fetch_ids(table, t0, end, &cur);
    uint32_t next = t0, slot = 0;
    // Finds the next tile that holds anything (x->t >= t1: there is none) and
    // asks for the ids of the one after it.
    auto find = [&](Stage* x) {
      x->t = find_tile(a, table, next, t1, end, &cur, &x->st);
      const uint8_t* base = rows_of(a, cur, x->st, carrier);
      next = x->t + 1;
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        cur.off[i] += kTile;
        while (cur.off[i] >= a.block_tokens) {
          cur.off[i] -= a.block_tokens;
          ++cur.j[i];
        }
      }
      fetch_ids(table, next, end, &cur);
      return base;
    };
    auto announce = [&](const Stage& x) {
      if (carrier == 0 && lane == 0)
        *(HKV_LDS v2u*)lds.tile[slot] = v2u{x.t, x.st};
      slot = (slot + 1) % kTileSlots;
    };
    // Writes a loaded tile to its buffer and starts the loads of another (found
    // first: the scalar loads' wait would include the writes).
    auto stage = [&](Stage* x, uint32_t buf) {
      const uint32_t t_now = x->t, st_now = x->st;
      const uint8_t* base = find(x);
      stage_tile(a, end, carrier, lane, t_now, st_now, x->x, (HKV_LDS uint8_t*)lds.k[buf]);
      load_rows<kStream>(a, base, carrier, lane, x->x);
    };
    auto after = [](uint32_t buf) { return buf + 1 == kBuffers ? 0 : buf + 1; };
    Stage xa, xb;
    load_rows<kStream>(a, find(&xa), carrier, lane, xa.x);
    load_rows<kStream>(a, find(&xb), carrier, lane, xb.x);
    announce(xa);
    announce(xb);
    uint32_t t = xa.t;
    stage(&xa, 0);
    lds_barrier();
    // Two rounds a turn and one exit: xa and xb stay in their registers, and the
    // waits for the loads know which of them is older.  A tile past the last is
    // staged as zeros and not looked at.
    bool left = false;      // whether a tile waits to be added
    uint32_t b0 = 0;        // the buffer of the round's scored tile
    uint32_t b_last = 0;    // and of the tile before it
    while (t < t1) {
      const uint32_t b1 = after(b0), b2 = after(b1);
      announce(xa);
      left = xb.t < t1;     // of the tile scored in the second round
      stage(&xb, b1);
      if (b_last != b0) add_tile(lds, b_last, 1, carrier, lane, acc);
      lds_barrier();
      t = xa.t;
      announce(xb);
      stage(&xa, b2);
      add_tile(lds, b0, 0, carrier, lane, acc);
      lds_barrier();
      b_last = b1;
      b0 = b2;
    }
    if (left) add_tile(lds, b_last, 1, carrier, lane, acc);
    lds_barrier();
  }

  static __device__ __forceinline__ void score(const hkv::AttendArgs& a, Lds& lds,
                                               uint32_t scorer, uint32_t lane, uint32_t s,
                                               uint32_t ht, uint32_t t1, uint32_t len) {
    const uint32_t col = lane & 15, quad = lane >> 4;
    const uint32_t hl = scorer * 16 + col, h = ht * kHeads + hl, steps = a.width / 32;
    v4u q[kWidthSteps];  // the queries, as the column operand
    {
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)s * a.q_seq_stride +
                            (int64_t)h * a.q_head_stride + quad * 8;
#pragma unroll
      for (uint32_t i = 0; i < kWidthSteps; ++i) {
        v4u v = {0u, 0u, 0u, 0u};
        if (h < a.n_heads && i < steps) v = *(const HKV_GLOBAL v4u*)(src + i * 32);
        q[i] = v;
      }
    }
    float m = -INFINITY, l = 0.0f;
    uint32_t buf = 0, half = 0, slot = 0;
    __builtin_amdgcn_s_setprio(2);  // the carriers wait for P, with more waves to fill the time
    lds_barrier();
    v2u info = *(const HKV_LDS v2u*)lds.tile[0];
    for (;;) {
      const uint32_t t = uniform(info[0]);
      if (t >= t1) break;
      const uint32_t st = uniform(info[1]);
      slot = (slot + 1) % kTileSlots;
      info = *(const HKV_LDS v2u*)lds.tile[slot];  // the next tile's
      // S of 32 tokens (two 16-row results) x 16 heads.
      const HKV_LDS uint8_t* row = (const HKV_LDS uint8_t*)lds.k[buf] + col * kPitch + quad * 16;
      v4f sc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      __builtin_amdgcn_sched_barrier(0);
      v4u k[kAhead + 1][2];  // rows are read kAhead steps before they are multiplied
#pragma unroll
      for (uint32_t i = 0; i < kWidthSteps + kAhead; ++i) {
        if (i < kWidthSteps)
#pragma unroll
          for (uint32_t r = 0; r < 2; ++r)
            k[i % (kAhead + 1)][r] = *(const HKV_LDS v4u*)(row + r * 16 * kPitch + i * 64);
        if (i >= kAhead)
#pragma unroll
          for (uint32_t r = 0; r < 2; ++r)
            sc[r] = T::mma(k[(i - kAhead) % (kAhead + 1)][r], q[i - kAhead], sc[r]);
      }
      // The order just written, which the compiler would otherwise shorten to
      // one read ahead: 2 kAhead LDS reads, then two products and two reads in
      // turn (1450 -> 1000 cycles a tile).
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 0);
#pragma unroll
      for (uint32_t i = 0; i < kWidthSteps - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 2 * kAhead, 0);
      __builtin_amdgcn_sched_barrier(0);
      sc[0] *= a.scale;
      sc[1] *= a.scale;
      if (st != 0 || t * kTile + kTile > len) {  // not all present
#pragma unroll
        for (uint32_t r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (state_of(st, r) == kAbsent || t * kTile + r * 16 + quad * 4 + i >= len)
              sc[r][i] = -INFINITY;
            else if (state_of(st, r) == kBad)
              sc[r][i] = NAN;
          }
      }
      float top = -INFINITY;
#pragma unroll
      for (uint32_t r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[r][i]);
      if (a.logits && h < a.n_heads) {
        float* to = a.logits + (((uint64_t)s * a.max_tiles + t) * a.n_heads + h) * kTile + quad * 4;
        *(HKV_GLOBAL v4f*)to = sc[0];
        *(HKV_GLOBAL v4f*)(to + 16) = sc[1];
      }
      top = fmaxf(m, column_max(top));
      const float base = top == -INFINITY ? 0.0f : top;
      const float alpha = exp_of(m - base);
      m = top;
      l *= alpha;
      HKV_LDS uint8_t* hi = (HKV_LDS uint8_t*)lds.p_hi[half] + hl * kPPitch + quad * 8;
      HKV_LDS uint8_t* lo = (HKV_LDS uint8_t*)lds.p_lo[half] + hl * kPPitch + quad * 8;
#pragma unroll
      for (uint32_t r = 0; r < 2; ++r) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = exp_of(sc[r][i] - base);
          l += p[i];
          p[i] *= kUp;
        }
        const uint32_t h01 = T::pack(p[0], p[1]), h23 = T::pack(p[2], p[3]);
        *(HKV_LDS v2u*)(hi + r * 32) = v2u{h01, h23};
        *(HKV_LDS v2u*)(lo + r * 32) = v2u{T::pack(p[0] - T::low(h01), p[1] - T::high(h01)),
                                          T::pack(p[2] - T::low(h23), p[3] - T::high(h23))};
      }
      if (quad == 0) lds.alpha[half][hl] = alpha;
      buf = buf + 1 == kBuffers ? 0 : buf + 1;
      half ^= 1;
      lds_barrier();
    }
    __builtin_amdgcn_s_setprio(0);
    l = column_sum(l);
    if (quad == 0) {
      lds.m[hl] = m;
      lds.l[hl] = l;
    }
    if (half) lds_barrier();
    lds_barrier();
  }

  static __device__ __forceinline__ void run(const hkv::AttendArgs& a, Lds& lds) {
    const uint32_t worker = blockIdx.x, ht = blockIdx.y;
    const uint32_t wave = uniform(threadIdx.x >> 6);
    uint64_t first, share, total, seq_start;
    uint32_t s = 0;
    find_run(a, lds, worker, &first, &share, &total, &s, &seq_start);
    if (first >= total) return;
    const uint64_t last = first + share < total ? first + share : total;
    // Narrower rows leave the rest of the buffers' columns at zero, so that the
    // products need no bounds.
    if (a.width < hkv::kAttendMaxWidth)
      for (uint32_t i = threadIdx.x; i < sizeof(lds.k) / 16; i += kThreads)
        ((HKV_LDS v4u*)lds.k)[i] = v4u{0u, 0u, 0u, 0u};
    lds_barrier();

    for (uint64_t at = first; at < last && s < a.n_seqs;) {
      const uint32_t len = uniform(served_len(a, s));
      const uint32_t n_tiles = tiles_of(len);
      if (n_tiles == 0) {  // an empty sequence owns no tiles
        ++s;
        continue;
      }
      const uint32_t t0 = (uint32_t)(at - seq_start);
      const uint32_t t1 = last - seq_start < n_tiles ? (uint32_t)(last - seq_start) : n_tiles;
      if (t0 == 0 && ht == 0 && threadIdx.x == 0) {
        a.spans[s * 4 + 0] = (int32_t)worker;
        a.spans[s * 4 + 1] = (int32_t)((seq_start + n_tiles - 1) / share);
        a.spans[s * 4 + 2] = at == first ? 0 : 1;
      }
      const uint32_t lane = opaque(threadIdx.x & 63);
      if (wave < kScorers) {
        score(a, lds, wave, lane, s, ht, t1, len);
      } else {
        const uint32_t carrier = wave - kScorers;
        const uint32_t end = t1 * kTile < len ? t1 * kTile : len;  // of what this worker loads
        v4f acc[kHeadTiles][kOTiles];
        const HKV_CONST int32_t* table =
            (const HKV_CONST int32_t*)(a.table + (int64_t)s * a.table_stride);
        if (a.streams)
          carry<true>(a, lds, carrier, lane, table, t0, t1, end, acc);
        else
          carry<false>(a, lds, carrier, lane, table, t0, t1, end, acc);
        const uint32_t out_lane = opaque(lane), col = out_lane & 15, quad = out_lane >> 4;
        const bool whole = t0 == 0 && t1 == n_tiles;
        const uint64_t slot = ((uint64_t)worker * a.head_tiles + ht) * 2 + (at == first ? 0 : 1);
#pragma unroll
        for (uint32_t i = 0; i < kHeadTiles; ++i) {
          const uint32_t hl = i * 16 + col, h = ht * kHeads + hl;
          const float l = lds.l[hl], top = lds.m[hl];
          if (h >= a.n_heads) continue;
          const float inv =
              (whole ? (l == 0.0f ? 0.0f : a.cache_scale / l) : 1.0f) * (1.0f / kUp);
#pragma unroll
          for (uint32_t j = 0; j < kOTiles; ++j) {
            const uint32_t v = (j * kCarriers + carrier) * 16 + quad * 4;
            if (v >= a.values) continue;
            const v4f o = acc[i][j] * inv;
            if (whole) {
              uint16_t* to = static_cast<uint16_t*>(a.out) + (int64_t)s * a.out_seq_stride +
                             (int64_t)h * a.out_head_stride + v;
              *(HKV_GLOBAL v2u*)to = v2u{T::pack(o[0], o[1]), T::pack(o[2], o[3])};
            } else {
              *(HKV_GLOBAL v4f*)(a.part_o + (slot * kHeads + hl) * a.values + v) = o;
            }
          }
          if (carrier == i && quad == 0) {
            if (whole) {
              write_lse(a, s, h, top, l);
            } else {
              a.part_ml[(slot * kHeads + hl) * 2 + 0] = top;
              a.part_ml[(slot * kHeads + hl) * 2 + 1] = l;
            }
          }
        }
      }
      at = seq_start + t1;
      seq_start += n_tiles;
      ++s;
      lds_barrier();  // the next sequence reuses the LDS
    }
  }
};

// Adds up the partial results of a sequence's workers for one head and
// 4 << a.join_shift value columns: the workgroup's threads are groups of
// 1 << join_shift lanes, each taking every so many partial results.  Few
// (sequence, head) pairs are spread over more workgroups by taking fewer
// columns in each.  Also writes the rows of sequences that own no tile (zeros
// for an empty one, NaN for a length the table cannot hold).
constexpr uint32_t kJoinThreads = hkv::kAttendMaxWorkers;  // one partial result a thread

template <class T>
__device__ __forceinline__ void join(const hkv::AttendArgs& a) {
  __shared__ v4f part[kJoinThreads];
  __shared__ float scale[kJoinThreads];
  __shared__ float red[2][kJoinThreads / 64];
  const uint32_t s = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
  const uint32_t t = threadIdx.x, lanes = 1u << a.join_shift;
  const uint32_t lane = t & (lanes - 1), grp = t >> a.join_shift, groups = kJoinThreads / lanes;
  const uint32_t v = (blockIdx.y * lanes + lane) * 4;
  uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)s * a.out_seq_stride +
                  (int64_t)h * a.out_head_stride + v;
  const int32_t len = a.lens[s];
  if (served_len(a, s) == 0) {
    const float x = len == 0 ? 0.0f : NAN;
    if (grp == 0 && v < a.values) *(HKV_GLOBAL v2u*)out = v2u{T::pack(x, x), T::pack(x, x)};
    if (t == 0 && blockIdx.y == 0) write_lse(a, s, h, x, x);
    return;
  }
  const uint32_t w0 = (uint32_t)a.spans[s * 4], w1 = (uint32_t)a.spans[s * 4 + 1];
  const uint32_t slot0 = (uint32_t)a.spans[s * 4 + 2];
  if (w0 == w1) return;
  const uint32_t ht = h / a.head_tile, hl = h % a.head_tile, n = w1 - w0 + 1;
  auto row = [&](uint32_t i) {  // worker w0 + i: its first run, but slot0 for w0
    return (((uint64_t)(w0 + i) * a.head_tiles + ht) * 2 + (i == 0 ? slot0 : 0)) * a.head_tile + hl;
  };
  const float m = t < n ? a.part_ml[row(t) * 2] : -INFINITY;
  const float l = t < n ? a.part_ml[row(t) * 2 + 1] : 0.0f;
  float top = m;
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, lane_xor(top, d));
  if ((t & 63) == 0) red[0][t >> 6] = top;
  __syncthreads();
  for (uint32_t w = 0; w < kJoinThreads / 64; ++w) top = fmaxf(top, red[0][w]);
  const float x = exp_of(m - (top == -INFINITY ? 0.0f : top));
  scale[t] = x;
  float sum = l * x;
  for (int d = 1; d < 64; d <<= 1) sum += lane_xor(sum, d);
  if ((t & 63) == 0) red[1][t >> 6] = sum;
  __syncthreads();
  sum = 0.0f;
  for (uint32_t w = 0; w < kJoinThreads / 64; ++w) sum += red[1][w];
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (v < a.values)
#pragma unroll 4
    for (uint32_t i = grp; i < n; i += groups)
      o += *(const HKV_GLOBAL v4f*)(a.part_o + row(i) * a.values + v) * scale[i];
  part[t] = o;
  __syncthreads();
  if (grp == 0 && v < a.values) {
    for (uint32_t k = 1; k < groups && k < n; ++k) o += part[k * lanes + lane];
    o *= sum == 0.0f ? 0.0f : a.cache_scale / sum;
    *(HKV_GLOBAL v2u*)out = v2u{T::pack(o[0], o[1]), T::pack(o[2], o[3])};
  }
  if (t == 0 && blockIdx.y == 0) write_lse(a, s, h, top, sum);
}

}  // namespace

// The 64-head kernels for 2-byte rows are 16 registers over what 12 waves leave
// each (60 bytes of scratch a lane); no other spills any but scalar ones.
#define HKV_ATTEND(name, T, fp8, heads)                                                     \
  extern "C" __global__ __launch_bounds__(attend_threads(heads)) void name(hkv::AttendArgs a) { \
    __shared__ __align__(16) Attend<T, fp8, heads>::Lds lds;                                \
    Attend<T, fp8, heads>::run(a, lds);                                                     \
  }
#define HKV_ATTEND_HEADS(suffix, T, fp8)               \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h16, T, fp8, 16) \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h32, T, fp8, 32) \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h64, T, fp8, 64)
HKV_ATTEND_HEADS(bf16, Bf16, false)
HKV_ATTEND_HEADS(fp16, Fp16, false)
HKV_ATTEND_HEADS(bf16_e4m3, Bf16, true)
HKV_ATTEND_HEADS(fp16_e4m3, Fp16, true)
#undef HKV_ATTEND
#undef HKV_ATTEND_HEADS

extern "C" __global__ __launch_bounds__(kJoinThreads) void hkv_mla_attend_join_bf16(
    hkv::AttendArgs a) {
  join<Bf16>(a);
}
extern "C" __global__ __launch_bounds__(kJoinThreads) void hkv_mla_attend_join_fp16(
    hkv::AttendArgs a) {
  join<Fp16>(a);
}

// weights[s][t] += sum over heads of exp(s_ht - lse_h), from the logits that
// the attention left in the workspace (4 bytes per head and token, where a
// second pass over the cache would read a row again).  kWeightParts threads
// share a token, each takes every so many heads, and their sums are added in
// order, so the result does not depend on the schedule.  Bound: the logits'
// bytes, and for few tokens the latency of the loads, for which the parts are:
// 1 sequence of 16000 tokens, 64 heads, 34.8 us with 4 parts, 37.2 with one
// (the whole call); with 8 parts, that is 32 tokens a workgroup, a large call
// loses (64 of 14001 tokens, 32 heads: 186 us, 206).
constexpr uint32_t kWeightParts = 4;
constexpr uint32_t kWeightTokens = 256 / kWeightParts;
constexpr uint32_t kWeightGroups = 16384;  // workgroups at most: several pieces each if need be

extern "C" __global__ __launch_bounds__(256) void hkv_mla_attend_weights(hkv::AttendArgs a) {
  __shared__ float part[kWeightParts][kWeightTokens];
  const uint32_t s = blockIdx.y, len = served_len(a, s);
  const uint32_t col = threadIdx.x % kWeightTokens, p = threadIdx.x / kWeightTokens;
  const float* norm = a.norm + (uint64_t)s * a.n_heads;
  for (uint32_t at = blockIdx.x * kWeightTokens; at < len; at += gridDim.x * kWeightTokens) {
    const uint32_t tok = at + col;
    // (tiles of null blocks have no logits)
    const bool live = tok < len && a.table[(int64_t)s * a.table_stride + tok / a.block_tokens] !=
                                       HKV_NULL_BLOCK;
    float sum = 0.0f;
    if (live) {
      const float* x = a.logits + ((uint64_t)s * a.max_tiles + tok / kTile) * a.n_heads * kTile +
                       tok % kTile;
#pragma unroll 4
      for (uint32_t h = p; h < a.n_heads; h += kWeightParts)
        sum += exp_of(x[(uint64_t)h * kTile] - norm[h]);
    }
    part[p][col] = sum;
    __syncthreads();
    if (p == 0 && live) {
      for (uint32_t k = 1; k < kWeightParts; ++k) sum += part[k][col];
      a.weights[(int64_t)s * a.weights_stride + tok] += sum;
    }
    __syncthreads();
  }
}

namespace hkv {

int launch_attend(const AttendArgs& a, int32_t dtype, int32_t cache_dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
#define HKV_SIZES(name) {HKV_FN(name##_h16), HKV_FN(name##_h32), HKV_FN(name##_h64)}
  static const void* const kKernels[2][2][3] = {
      {HKV_SIZES(hkv_mla_attend_bf16), HKV_SIZES(hkv_mla_attend_bf16_e4m3)},
      {HKV_SIZES(hkv_mla_attend_fp16), HKV_SIZES(hkv_mla_attend_fp16_e4m3)}};
#undef HKV_SIZES
  const uint32_t ty = dtype == HKV_FP16, fp8 = cache_dtype == HKV_E4M3;
  const void* main_fn = kKernels[ty][fp8][a.head_tile / 32];
  const void* join_fn = ty ? HKV_FN(hkv_mla_attend_join_fp16) : HKV_FN(hkv_mla_attend_join_bf16);
#undef HKV_FN
  AttendArgs arg = a;
  void* params[] = {&arg};
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipLaunchKernel(main_fn, dim3(a.workers, a.head_tiles),
                                 dim3(attend_threads(a.head_tile)), params, 0, st);
  if (e == hipSuccess)
    e = hipLaunchKernel(join_fn,
                        dim3(a.n_seqs * a.n_heads,
                             (a.values + (4u << a.join_shift) - 1) / (4u << a.join_shift)),
                        dim3(kJoinThreads), params, 0, st);
  if (e == hipSuccess && a.weights)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&hkv_mla_attend_weights),
                        dim3(std::min((a.max_tiles * kTile + kWeightTokens - 1) / kWeightTokens,
                                      std::max(kWeightGroups / a.n_seqs, 1u)),
                             a.n_seqs),
                        dim3(256), params, 0, st);
  return (int)e;
}

}  // namespace hkv
