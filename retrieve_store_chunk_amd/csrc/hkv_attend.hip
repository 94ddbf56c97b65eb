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
// output itself.  e4m3 rows are widened to the query's type as they are
// staged, which is exact.
//
// Bound: reading the cache once (row_bytes per token).  A tile's rows are
// loaded two tiles ahead into registers and written to the other of two LDS
// buffers one tile ahead, so a tile's loads have a whole tile's time to
// arrive.  LDS rows are padded to an odd multiple of 32 bytes: eight rows at
// the same column, and four rows of the transposing loads, then fall into
// different banks.
//
// The batch's tiles, all sequences after one another, are cut into equal
// runs, one per worker (workgroup), whatever the lengths are: a million-token
// sequence and a ragged batch both fill the card, and no length is needed on
// the host.  A worker whose run covers part of a sequence leaves a partial
// result (m, l, unnormalised O) that hkv_mla_attend_join adds up.
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))
#define HKV_LDS __attribute__((address_space(3)))

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
constexpr uint32_t kPitchMax = hkv::kAttendMaxWidth * 2 + 32;
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

// The block of 16 rows starting at a 16-aligned token lies in one page (a
// block is a multiple of 16 tokens), so a tile has two row groups, each with
// one address.  State: 0 present, 1 absent (null block or past the end), 2 a
// block id outside the pool.
struct RowGroup {
  const uint8_t* base;
  uint32_t state;
};

template <class T, bool kFp8, uint32_t kHeads, uint32_t kWaves>
struct Attend {
  static constexpr uint32_t kThreads = kWaves * 64;
  static constexpr uint32_t kHeadTiles = kHeads / 16;
  static constexpr uint32_t kSTiles = kHeadTiles * (kTile / 16);  // 16x16 tiles of S
  static_assert(kSTiles <= kWaves, "one S tile per wave");
  static constexpr uint32_t kRowThreads = kThreads / kTile;       // threads that load a row
  static constexpr uint32_t kRowChunks = hkv::kAttendMaxWidth * (kFp8 ? 1 : 2) / 16;
  static constexpr uint32_t kLoads = (kRowChunks + kRowThreads - 1) / kRowThreads;
  static constexpr uint32_t kOTiles = kValueTiles / kWaves;       // O column tiles per wave

  struct Lds {
    uint8_t k[2][kTile * kPitchMax];
    uint8_t p_hi[kHeads * kPPitch];
    uint8_t p_lo[kHeads * kPPitch];
    float top[kTile / 16][kHeads];  // a tile's maximum per head and 16 tokens; later the sums
    float alpha[kHeads];
    float m[kHeads];
    uint32_t sums[kWaves];
    uint32_t start[2];
  };

  // The block id of a row group, asked for a tile before group_of needs it.
  static __device__ __forceinline__ int32_t id_at(const hkv::AttendArgs& a, const int32_t* table,
                                                  uint32_t tok, uint32_t len) {
    return tok < len ? table[tok / a.block_tokens] : HKV_NULL_BLOCK;
  }
  static __device__ __forceinline__ RowGroup group_of(const hkv::AttendArgs& a, int32_t raw,
                                                      uint32_t tok) {
    const int32_t id = __builtin_amdgcn_readfirstlane(raw);
    RowGroup g{a.pages, id == HKV_NULL_BLOCK ? 1u : 2u};
    if (id >= 0 && (uint32_t)id < a.num_blocks) {
      g.state = 0;
      g.base = a.pages + (uint64_t)id * a.stride + (uint64_t)(tok % a.block_tokens) * a.row_bytes;
    }
    return g;
  }

  // This thread's part of a tile's rows (zeros where a row is absent, so that
  // 0 x anything the memory holds never reaches a sum).
  static __device__ __forceinline__ void load_tile(const hkv::AttendArgs& a, const RowGroup* g,
                                                   uint32_t tok, uint32_t len, v4u* stage) {
    const uint32_t row = threadIdx.x / kRowThreads, c = threadIdx.x % kRowThreads;
    const RowGroup& mine = row < 16 ? g[0] : g[1];
    const bool live = mine.state == 0 && tok + row < len;
    const HKV_GLOBAL v4u* p =
        (const HKV_GLOBAL v4u*)(mine.base + (uint64_t)(row & 15) * a.row_bytes) + c;
    const uint32_t chunks = a.row_bytes / 16;
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      v4u v = {0u, 0u, 0u, 0u};
      if (live && c + i * kRowThreads < chunks) v = p[i * kRowThreads];
      stage[i] = v;
    }
  }

  static __device__ __forceinline__ void stage_tile(const hkv::AttendArgs& a, uint32_t pitch,
                                                    const v4u* stage, HKV_LDS uint8_t* lds) {
    const uint32_t row = threadIdx.x / kRowThreads, c = threadIdx.x % kRowThreads;
    const uint32_t chunks = a.row_bytes / 16;
    HKV_LDS uint8_t* d = lds + row * pitch + c * (kFp8 ? 32 : 16);
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      if (c + i * kRowThreads >= chunks) continue;
      if constexpr (kFp8) {
        const v4u lo = {T::template widen<false>(stage[i][0]), T::template widen<true>(stage[i][0]),
                        T::template widen<false>(stage[i][1]), T::template widen<true>(stage[i][1])};
        const v4u hi = {T::template widen<false>(stage[i][2]), T::template widen<true>(stage[i][2]),
                        T::template widen<false>(stage[i][3]), T::template widen<true>(stage[i][3])};
        HKV_LDS v4u* to = (HKV_LDS v4u*)(d + i * kRowThreads * 32);
        to[0] = lo;
        to[1] = hi;
      } else {
        *(HKV_LDS v4u*)(d + i * kRowThreads * 16) = stage[i];
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

  static __device__ __forceinline__ void run(const hkv::AttendArgs& a, Lds& lds) {
    const uint32_t worker = blockIdx.x, ht = blockIdx.y;
    const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t col = lane & 15, quad = lane >> 4;
    const uint32_t pitch = a.width * 2 + 32;
    const uint32_t steps = a.width / 32, vtiles = a.values / 16;
    const uint32_t my_ht = wave % kHeadTiles, my_kt = wave / kHeadTiles;
    const bool scores = wave < kSTiles;
    uint64_t first, share, total, seq_start;
    uint32_t s = 0;
    find_run(a, lds, worker, &first, &share, &total, &s, &seq_start);
    if (first >= total) return;
    const uint64_t last = first + share < total ? first + share : total;

    for (uint64_t at = first; at < last && s < a.n_seqs;) {
      const uint32_t len = uniform(served_len(a, s));
      const uint32_t n_tiles = tiles_of(len);
      if (n_tiles == 0) {  // an empty sequence owns no tiles
        ++s;
        continue;
      }
      const uint32_t t0 = (uint32_t)(at - seq_start);
      const uint32_t t1 = last - seq_start < n_tiles ? (uint32_t)(last - seq_start) : n_tiles;
      const int32_t* table = a.table + (int64_t)s * a.table_stride;
      if (t0 == 0 && ht == 0 && threadIdx.x == 0) {
        a.spans[s * 4 + 0] = (int32_t)worker;
        a.spans[s * 4 + 1] = (int32_t)((seq_start + n_tiles - 1) / share);
        a.spans[s * 4 + 2] = at == first ? 0 : 1;
      }

      // The queries of this wave's head tile, as the S product's column operand.
      v4u q[kWidthSteps];
      {
        const uint32_t h = ht * kHeads + my_ht * 16 + col;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)s * a.q_seq_stride +
                              (int64_t)h * a.q_head_stride + quad * 8;
#pragma unroll
        for (uint32_t i = 0; i < kWidthSteps; ++i) {
          v4u v = {0u, 0u, 0u, 0u};
          if (scores && h < a.n_heads && i < steps) v = *(const HKV_GLOBAL v4u*)(src + i * 32);
          q[i] = v;
        }
      }
      v4f acc[kHeadTiles][kOTiles];
#pragma unroll
      for (uint32_t i = 0; i < kHeadTiles; ++i)
#pragma unroll
        for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      float m = -INFINITY, l = 0.0f;

      v4u stage[kLoads];
      RowGroup g[2], g_next[2];
      int32_t id[2], id_next[2];
      for (uint32_t i = 0; i < 2; ++i) id[i] = id_at(a, table, t0 * kTile + i * 16, len);
      for (uint32_t i = 0; i < 2; ++i) id_next[i] = id_at(a, table, (t0 + 1) * kTile + i * 16, len);
      for (uint32_t i = 0; i < 2; ++i) g[i] = group_of(a, id[i], t0 * kTile + i * 16);
      load_tile(a, g, t0 * kTile, len, stage);
      for (uint32_t i = 0; i < 2; ++i) {
        g_next[i] = group_of(a, id_next[i], (t0 + 1) * kTile + i * 16);
        id[i] = id_at(a, table, (t0 + 2) * kTile + i * 16, len);
      }
      stage_tile(a, pitch, stage, (HKV_LDS uint8_t*)lds.k[0]);
      if (t0 + 1 < t1) load_tile(a, g_next, (t0 + 1) * kTile, len, stage);
      lds_barrier();

      for (uint32_t t = t0; t < t1; ++t) {
        const HKV_LDS uint8_t* kb = (const HKV_LDS uint8_t*)lds.k[(t - t0) & 1];
        // S: 16 tokens x 16 heads per wave.
        v4f sc = {0.0f, 0.0f, 0.0f, 0.0f};
        if (scores) {
          const HKV_LDS uint8_t* row = kb + (my_kt * 16 + col) * pitch + quad * 16;
#pragma unroll
          for (uint32_t i = 0; i < kWidthSteps; ++i)
            if (i < steps) sc = T::mma(*(const HKV_LDS v4u*)(row + i * 64), q[i], sc);
          const uint32_t state = my_kt ? g[1].state : g[0].state;
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t tok = t * kTile + my_kt * 16 + quad * 4 + i;
            float x = sc[i] * a.scale;
            if (state == 1 || tok >= len) x = -INFINITY;
            else if (state == 2) x = NAN;
            sc[i] = x;
            top = fmaxf(top, x);
          }
          top = fmaxf(top, lane_xor(top, 16));
          top = fmaxf(top, lane_xor(top, 32));
          if (quad == 0) lds.top[my_kt][my_ht * 16 + col] = top;
          const uint32_t h = ht * kHeads + my_ht * 16 + col;
          if (a.logits && h < a.n_heads) {
            float* to = a.logits + (((uint64_t)s * a.max_tiles + t) * a.n_heads + h) * kTile +
                        my_kt * 16 + quad * 4;
            *(HKV_GLOBAL v4f*)to = sc;
          }
        }
        lds_barrier();
        if (scores) {
          const uint32_t h = my_ht * 16 + col;
          const float top = fmaxf(m, fmaxf(lds.top[0][h], lds.top[1][h]));
          const float base = top == -INFINITY ? 0.0f : top;
          const float alpha = exp_of(m - base);
          m = top;
          float p[4], sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = exp_of(sc[i] - base);
            sum += p[i];
          }
          l = l * alpha + sum;
          const uint32_t h01 = T::pack(p[0], p[1]), h23 = T::pack(p[2], p[3]);
          const uint32_t l01 = T::pack(p[0] - T::low(h01), p[1] - T::high(h01));
          const uint32_t l23 = T::pack(p[2] - T::low(h23), p[3] - T::high(h23));
          const uint32_t to = h * kPPitch + my_kt * 32 + quad * 8;
          *(HKV_LDS v2u*)((HKV_LDS uint8_t*)lds.p_hi + to) = v2u{h01, h23};
          *(HKV_LDS v2u*)((HKV_LDS uint8_t*)lds.p_lo + to) = v2u{l01, l23};
          if (my_kt == 0 && quad == 0) lds.alpha[h] = alpha;
        }
        g[0] = g_next[0];
        g[1] = g_next[1];
        if (t + 1 < t1) {
          stage_tile(a, pitch, stage, (HKV_LDS uint8_t*)lds.k[(t + 1 - t0) & 1]);
          for (uint32_t i = 0; i < 2; ++i) {
            g_next[i] = group_of(a, id[i], (t + 2) * kTile + i * 16);
            id[i] = id_at(a, table, (t + 3) * kTile + i * 16, len);
          }
          if (t + 2 < t1) load_tile(a, g_next, (t + 2) * kTile, len, stage);
        }
        lds_barrier();
        // O^T: this wave's value columns x all heads.
        v4u ph[kHeadTiles], pl[kHeadTiles];
#pragma unroll
        for (uint32_t i = 0; i < kHeadTiles; ++i) {
          const uint32_t from = (i * 16 + col) * kPPitch + quad * 16;
          ph[i] = *(const HKV_LDS v4u*)((const HKV_LDS uint8_t*)lds.p_hi + from);
          pl[i] = *(const HKV_LDS v4u*)((const HKV_LDS uint8_t*)lds.p_lo + from);
          const float alpha = lds.alpha[i * 16 + col];
          if (__any(alpha != 1.0f)) {
#pragma unroll
            for (uint32_t j = 0; j < kOTiles; ++j) acc[i][j] *= alpha;
          }
        }
        // Transposing loads: in each group of 16 lanes, lane x supplies four
        // columns of token x / 4 and receives column x of four tokens.
        const HKV_LDS uint8_t* vb = kb + (quad * 8 + (col >> 2)) * pitch + (col & 3) * 8;
#pragma unroll
        for (uint32_t j = 0; j < kOTiles; ++j) {
          const uint32_t vt = j * kWaves + wave;
          if (vt >= vtiles) continue;
          const HKV_LDS uint8_t* from = vb + vt * 32;
          const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((HKV_LDS v4s*)from);
          const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((HKV_LDS v4s*)(from + 4 * pitch));
          const v2u lo2 = __builtin_bit_cast(v2u, lo), hi2 = __builtin_bit_cast(v2u, hi);
          const v4u v = {lo2[0], lo2[1], hi2[0], hi2[1]};
#pragma unroll
          for (uint32_t i = 0; i < kHeadTiles; ++i) {
            acc[i][j] = T::mma(v, ph[i], acc[i][j]);
            acc[i][j] = T::mma(v, pl[i], acc[i][j]);
          }
        }
      }

      // The sums of the waves that hold a head's tokens, joined (lds.top was
      // last read before the loop's last barrier).
      if (scores) {
        l += lane_xor(l, 16);
        l += lane_xor(l, 32);
        if (quad == 0) {
          lds.top[my_kt][my_ht * 16 + col] = l;
          if (my_kt == 0) lds.m[my_ht * 16 + col] = m;
        }
      }
      lds_barrier();
      const bool whole = t0 == 0 && t1 == n_tiles;
      const uint64_t slot = ((uint64_t)worker * a.head_tiles + ht) * 2 + (at == first ? 0 : 1);
#pragma unroll
      for (uint32_t i = 0; i < kHeadTiles; ++i) {
        const uint32_t hl = i * 16 + col, h = ht * kHeads + hl;
        const float sum = lds.top[0][hl] + lds.top[1][hl];
        const float top = lds.m[hl];
        if (h >= a.n_heads) continue;
        const float inv = whole ? (sum == 0.0f ? 0.0f : a.cache_scale / sum) : 1.0f;
#pragma unroll
        for (uint32_t j = 0; j < kOTiles; ++j) {
          const uint32_t vt = j * kWaves + wave;
          if (vt >= vtiles) continue;
          const v4f o = acc[i][j] * inv;
          const uint32_t v = vt * 16 + quad * 4;
          if (whole) {
            uint16_t* to = static_cast<uint16_t*>(a.out) + (int64_t)s * a.out_seq_stride +
                           (int64_t)h * a.out_head_stride + v;
            *(HKV_GLOBAL v2u*)to = v2u{T::pack(o[0], o[1]), T::pack(o[2], o[3])};
          } else {
            *(HKV_GLOBAL v4f*)(a.part_o + (slot * kHeads + hl) * a.values + v) = o;
          }
        }
        if (wave == i % kWaves && quad == 0) {
          if (whole) {
            write_lse(a, s, h, top, sum);
          } else {
            a.part_ml[(slot * kHeads + hl) * 2 + 0] = top;
            a.part_ml[(slot * kHeads + hl) * 2 + 1] = sum;
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

// Adds up the partial results of a sequence's workers for one head and 128
// value columns; also writes the rows of sequences that own no tile (zeros for
// an empty one, NaN for a length the table cannot hold).
constexpr uint32_t kJoinThreads = 256;
constexpr uint32_t kJoinGroups = kJoinThreads / 32;  // 32 lanes x 4 columns each

template <class T>
__device__ __forceinline__ void join(const hkv::AttendArgs& a) {
  __shared__ float part[kJoinGroups][32][4];
  __shared__ float red[2][kJoinThreads / 64];
  const uint32_t s = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
  const uint32_t t = threadIdx.x, lane = t & 31, grp = t >> 5;
  const uint32_t v = blockIdx.y * 128 + lane * 4;
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
  float top = -INFINITY;
  for (uint32_t i = t; i < n; i += kJoinThreads) top = fmaxf(top, a.part_ml[row(i) * 2]);
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, lane_xor(top, d));
  if ((t & 63) == 0) red[0][t >> 6] = top;
  __syncthreads();
  for (uint32_t w = 0; w < kJoinThreads / 64; ++w) top = fmaxf(top, red[0][w]);
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (uint32_t i = t; i < n; i += kJoinThreads)
    sum += a.part_ml[row(i) * 2 + 1] * exp_of(a.part_ml[row(i) * 2] - base);
  for (int d = 1; d < 64; d <<= 1) sum += lane_xor(sum, d);
  if ((t & 63) == 0) red[1][t >> 6] = sum;
  __syncthreads();
  sum = 0.0f;
  for (uint32_t w = 0; w < kJoinThreads / 64; ++w) sum += red[1][w];
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (v < a.values)
    for (uint32_t i = grp; i < n; i += kJoinGroups)
      o += *(const HKV_GLOBAL v4f*)(a.part_o + row(i) * a.values + v) *
           exp_of(a.part_ml[row(i) * 2] - base);
#pragma unroll
  for (int i = 0; i < 4; ++i) part[grp][lane][i] = o[i];
  __syncthreads();
  if (grp == 0 && v < a.values) {
    for (uint32_t k = 1; k < kJoinGroups; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += part[k][lane][i];
    o *= sum == 0.0f ? 0.0f : a.cache_scale / sum;
    *(HKV_GLOBAL v2u*)out = v2u{T::pack(o[0], o[1]), T::pack(o[2], o[3])};
  }
  if (t == 0 && blockIdx.y == 0) write_lse(a, s, h, top, sum);
}

}  // namespace

#define HKV_ATTEND(name, T, fp8, heads, waves)                                              \
  extern "C" __global__ __launch_bounds__((waves) * 64, 2) void name(hkv::AttendArgs a) {   \
    __shared__ __align__(16) Attend<T, fp8, heads, waves>::Lds lds;                         \
    Attend<T, fp8, heads, waves>::run(a, lds);                                              \
  }
#define HKV_ATTEND_HEADS(suffix, T, fp8)                  \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h16, T, fp8, 16, 4) \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h32, T, fp8, 32, 4) \
  HKV_ATTEND(hkv_mla_attend_##suffix##_h64, T, fp8, 64, 8)
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
// second pass over the cache would read a row again): one thread per token,
// heads in order, so the result does not depend on the schedule.
extern "C" __global__ __launch_bounds__(256) void hkv_mla_attend_weights(hkv::AttendArgs a) {
  const uint32_t s = blockIdx.y;
  const uint32_t len = served_len(a, s);
  const uint32_t tok = blockIdx.x * 256 + threadIdx.x;
  if (tok >= len) return;
  const float* x = a.logits + ((uint64_t)s * a.max_tiles + tok / kTile) * a.n_heads * kTile +
                   tok % kTile;
  const float* norm = a.norm + (uint64_t)s * a.n_heads;
  float sum = 0.0f;
  for (uint32_t h = 0; h < a.n_heads; ++h) sum += exp_of(x[(uint64_t)h * kTile] - norm[h]);
  a.weights[(int64_t)s * a.weights_stride + tok] += sum;
}

namespace hkv {

int launch_attend(const AttendArgs& a, int32_t dtype, int32_t cache_dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
  static const void* const kKernels[2][2][3] = {
      {{HKV_FN(hkv_mla_attend_bf16_h16), HKV_FN(hkv_mla_attend_bf16_h32),
        HKV_FN(hkv_mla_attend_bf16_h64)},
       {HKV_FN(hkv_mla_attend_bf16_e4m3_h16), HKV_FN(hkv_mla_attend_bf16_e4m3_h32),
        HKV_FN(hkv_mla_attend_bf16_e4m3_h64)}},
      {{HKV_FN(hkv_mla_attend_fp16_h16), HKV_FN(hkv_mla_attend_fp16_h32),
        HKV_FN(hkv_mla_attend_fp16_h64)},
       {HKV_FN(hkv_mla_attend_fp16_e4m3_h16), HKV_FN(hkv_mla_attend_fp16_e4m3_h32),
        HKV_FN(hkv_mla_attend_fp16_e4m3_h64)}}};
  const uint32_t ty = dtype == HKV_FP16, fp8 = cache_dtype == HKV_E4M3;
  const void* main_fn = kKernels[ty][fp8][a.head_tile == 16 ? 0 : a.head_tile == 32 ? 1 : 2];
  const void* join_fn = ty ? HKV_FN(hkv_mla_attend_join_fp16) : HKV_FN(hkv_mla_attend_join_bf16);
#undef HKV_FN
  AttendArgs arg = a;
  void* params[] = {&arg};
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipLaunchKernel(main_fn, dim3(a.workers, a.head_tiles),
                                 dim3(a.head_tile == 64 ? 512 : 256), params, 0, st);
  if (e == hipSuccess)
    e = hipLaunchKernel(join_fn, dim3(a.n_seqs * a.n_heads, (a.values + 127) / 128),
                        dim3(kJoinThreads), params, 0, st);
  if (e == hipSuccess && a.weights)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&hkv_mla_attend_weights),
                        dim3((a.max_tiles * kTile + 255) / 256, a.n_seqs), dim3(256), params, 0,
                        st);
  return (int)e;
}

}  // namespace hkv
