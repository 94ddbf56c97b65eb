// Eviction from the MLA cache by accumulated attention weight (gfx950).
//
// Per (layer, sequence) longer than the budget B, a radix selection finds the
// B-th largest 32-bit key (protected slots above every weight, NaN below), a
// scan in slot order gives each kept slot past B the freed slot below B that
// it fills, and the move kernel copies those rows.  Kept slots past B and
// freed slots below B are equally many, a source is never a destination, so
// every row moves at most once, all at the same time and in place.
//
// The digits are 11, 11 and 10 bits wide: the first (sign, exponent and two
// bits) spreads weights over enough counters that lanes seldom meet on one
// (with 8 bits most weights share a handful of exponents' counters), and later
// digits only count keys that match so far.
//
// Rows of up to kSelectMax slots: one workgroup a row, which holds the row's
// keys in registers through all of it.  Longer rows: workgroups of
// kChunkSlots slots count into histograms in the workspace, one launch a
// digit, then one for each chunk's totals and one for the lists.
//
// Bound: 8 bytes read and 8 written per slot, and each moved row read and
// written once; only rows that must move do.
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t v4i_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ bool valid_len(const hkv::EvictArgs& a, int32_t len) {
  return len >= 0 && (uint64_t)len <= (uint64_t)a.max_blocks * a.block_tokens;
}

__device__ __forceinline__ int64_t meta_row(const hkv::EvictArgs& a, uint32_t row) {
  return (int64_t)(row / a.n_seqs) * a.layer_stride + (int64_t)(row % a.n_seqs) * a.seq_stride;
}

// Orders slots as the selection does: a larger key is kept first.
__device__ __forceinline__ uint32_t key_of(float w, bool held) {
  if (held) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool is_held(const hkv::EvictArgs& a, int32_t pos, int32_t next) {
  return pos < (int32_t)a.sinks || (int64_t)pos >= (int64_t)next - (int64_t)a.recent;
}

constexpr uint32_t kThreads = 1024;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kChunkSlots = hkv::kEvictChunkSlots;
constexpr uint32_t kChunkItems = kChunkSlots / kThreads;
static_assert(kBins == 2 * kThreads, "two bins a thread");

// Digit d of a key, counted from the top.
__device__ __forceinline__ uint32_t digit_shift(int d) { return d == 0 ? 21u : d == 1 ? 10u : 0u; }
__device__ __forceinline__ uint32_t digit_mask(int d) { return d == 2 ? 0x3FFu : 0x7FFu; }
// The bits above digit d.
__device__ __forceinline__ uint32_t above_mask(int d) {
  return d == 0 ? 0u : d == 1 ? 0xFFE00000u : 0xFFFFFC00u;
}

__device__ __forceinline__ uint32_t blocks_of(const hkv::EvictArgs& a, int32_t len) {
  return valid_len(a, len) ? ((uint32_t)len + a.block_tokens - 1) / a.block_tokens : 0u;
}

__device__ __forceinline__ void write_new_len(const hkv::EvictArgs& a, uint32_t s, bool ok) {
  const int32_t len = a.lens[s];
  if (a.new_lens)
    a.new_lens[s] = !ok ? -1 : (uint32_t)len < a.budget ? len : (int32_t)a.budget;
}

// Whether sequence s can be evicted from: a valid length, and every live block
// id in the pool and named once in the call.  By comparing each id with each
// (for calls with few ids; `own` holds the sequence's).
__device__ __forceinline__ bool check_by_pairs(const hkv::EvictArgs& a, uint32_t s, int32_t* own,
                                               uint32_t* bad) {
  const uint32_t t = threadIdx.x;
  const int32_t len = a.lens[s];
  const uint32_t blocks = blocks_of(a, len);
  if (t == 0) *bad = !valid_len(a, len);
  __syncthreads();
  for (uint32_t j = t; j < blocks; j += kThreads) {
    const int32_t id = a.table[(int64_t)s * a.table_stride + j];
    own[j] = id;
    if (id < 0 || (uint32_t)id >= a.num_blocks) *bad = 1;
  }
  __syncthreads();
  for (uint32_t i = t; i < a.n_seqs * a.max_blocks; i += kThreads) {
    const uint32_t s2 = i / a.max_blocks, j2 = i - s2 * a.max_blocks;
    if (j2 >= blocks_of(a, a.lens[s2])) continue;
    const int32_t id = a.table[(int64_t)s2 * a.table_stride + j2];
    bool same = false;
    for (uint32_t j = 0; j < blocks; ++j) same |= own[j] == id && !(s2 == s && j2 == j);
    if (same) *bad = 1;
  }
  __syncthreads();
  return *bad == 0;
}

// The exclusive prefix of `x` over the workgroup, and the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* waves, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t scan = x;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(scan, d, 64);
    if (lane >= (uint32_t)d) scan += up;
  }
  if (lane == 63) waves[wave] = scan;
  __syncthreads();
  uint32_t before = scan - x, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

// The bin that holds the `left`-th largest key, and the number of keys in
// larger bins.
__device__ __forceinline__ void find_bin(const uint32_t* hist, uint32_t left, uint32_t* waves,
                                         uint32_t* found, uint32_t* bin, uint32_t* above) {
  const uint32_t hi = kBins - 1 - 2 * threadIdx.x;  // thread 0 has the two largest
  const uint32_t n0 = hist[hi], n1 = hist[hi - 1];
  uint32_t all;
  const uint32_t before = block_scan(n0 + n1, waves, &all);
  if (before < left && left <= before + n0) {
    found[0] = hi;
    found[1] = before;
  } else if (before + n0 < left && left <= before + n0 + n1) {
    found[0] = hi - 1;
    found[1] = before + n0;
  }
  __syncthreads();
  *bin = found[0];
  *above = found[1];
  __syncthreads();
}

// Up to kItems consecutive slots of a row, from `first` on.
template <uint32_t kItems>
struct Slots {
  float w[kItems];
  int32_t pos[kItems];
  uint32_t key[kItems];
  uint32_t first, n;  // n of them exist
  __device__ __forceinline__ void load(const hkv::EvictArgs& a, const float* wp,
                                       const int32_t* pp, uint32_t at, uint32_t end,
                                       int32_t next) {
    first = at;
    n = at >= end ? 0 : end - at < kItems ? end - at : kItems;
    if (n == kItems) {  // four at a time (aligned to one: global loads may be)
#pragma unroll
      for (uint32_t i = 0; i < kItems; i += 4) {
        const v4f_a4 x = *(const HKV_GLOBAL v4f_a4*)(wp + at + i);
        const v4i_a4 y = *(const HKV_GLOBAL v4i_a4*)(pp + at + i);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
          w[i + k] = x[k];
          pos[i + k] = y[k];
        }
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < kItems; ++i) {
        w[i] = i < n ? wp[at + i] : 0.0f;
        pos[i] = i < n ? pp[at + i] : 0;
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i) key[i] = key_of(w[i], is_held(a, pos[i], next));
  }
  __device__ __forceinline__ void count(uint32_t* hist, uint32_t prefix, int d) const {
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i)
      if (i < n && (key[i] & above_mask(d)) == prefix)
        atomicAdd(&hist[(key[i] >> digit_shift(d)) & digit_mask(d)], 1u);
  }
};

// In slot order: which ties with the smallest kept key stay (the first `left`
// of them), and the number of each move.  `ties`, `holes`, `movers`: how many
// of each come before this thread's workgroup.  Writes the lists, and the
// weights and positions of every slot that does not move.
template <uint32_t kItems>
__device__ __forceinline__ void assign(const hkv::EvictArgs& a, const Slots<kItems>& x,
                                       uint32_t row, uint32_t least, uint32_t left,
                                       uint32_t* waves, uint32_t ties, uint32_t holes,
                                       uint32_t movers, uint32_t* all_holes) {
  uint32_t n = 0, all;
#pragma unroll
  for (uint32_t i = 0; i < kItems; ++i) n += i < x.n && x.key[i] == least;
  uint32_t rank = ties + block_scan(n, waves, &all);
  uint32_t keep = 0, n_holes = 0, n_movers = 0;  // keep: one bit a slot
#pragma unroll
  for (uint32_t i = 0; i < kItems; ++i) {
    if (i >= x.n) continue;
    const bool tie = x.key[i] == least;
    const bool k = x.key[i] > least || (tie && rank < left);
    rank += tie;
    keep |= (uint32_t)k << i;
    if (x.first + i < a.budget)
      n_holes += !k;
    else
      n_movers += k;
  }
  holes += block_scan(n_holes, waves, all_holes);
  movers += block_scan(n_movers, waves, &all);
  const int64_t base = meta_row(a, row);
  uint32_t* list = a.lists + (uint64_t)row * 2 * a.max_moves;
#pragma unroll
  for (uint32_t i = 0; i < kItems; ++i) {
    if (i >= x.n) continue;
    const uint32_t slot = x.first + i;
    const bool k = keep >> i & 1;
    if (slot < a.budget && k) {
      a.weights_out[base + slot] = x.w[i];
      a.positions_out[base + slot] = x.pos[i];
    } else if (slot < a.budget) {
      if (holes < a.max_moves) list[holes] = slot;
      ++holes;
    } else if (k) {
      if (movers < a.max_moves) list[a.max_moves + movers] = slot;
      ++movers;
    } else {
      a.weights_out[base + slot] = 0.0f;
      a.positions_out[base + slot] = -1;
    }
  }
}

// Copies the metadata of slots [first, end) of a row that keeps its rows.
__device__ __forceinline__ void copy_meta(const hkv::EvictArgs& a, uint32_t row, uint32_t first,
                                          uint32_t end) {
  const int64_t base = meta_row(a, row);
  if (a.weights_out != a.weights)
    for (uint32_t i = first + threadIdx.x; i < end; i += kThreads)
      a.weights_out[base + i] = a.weights[base + i];
  if (a.positions_out != a.positions)
    for (uint32_t i = first + threadIdx.x; i < end; i += kThreads)
      a.positions_out[base + i] = a.positions[base + i];
}

// One workgroup per (layer, sequence) of at most kItems x kThreads slots.
// (Measured against the chunked launches: 16 sequences of 8192 slots, 7 layers,
// 13 us here; one of 262144, 24 layers, 45 us there.)
template <uint32_t kItems>
__device__ __forceinline__ void select(const hkv::EvictArgs& a) {
  __shared__ uint32_t hist[kBins];
  __shared__ int32_t own[hkv::kEvictPairBlocks];
  __shared__ uint32_t waves[kWaves];
  __shared__ uint32_t found[2];
  __shared__ uint32_t bad;
  const uint32_t row = blockIdx.x, s = row % a.n_seqs, t = threadIdx.x;
  const int64_t base = meta_row(a, row);
  const int32_t raw_len = a.lens[s], next = a.next[s];
  const uint32_t len = valid_len(a, raw_len) ? (uint32_t)raw_len : 0u;
  // The loads are in flight while the block ids are checked.
  Slots<kItems> x;
  x.load(a, a.weights + base, a.positions + base, t * kItems, len > a.budget ? len : 0u, next);
  bool ok;
  if (a.by_pairs) {
    ok = check_by_pairs(a, s, own, &bad);
    if (t == 0 && row < a.n_seqs) write_new_len(a, s, ok);
  } else {
    ok = a.ok[s] != 0;
  }
  if (!ok || len <= a.budget) {
    copy_meta(a, row, 0, len);
    if (t == 0) a.moves[row] = 0;
    return;
  }
  uint32_t prefix = 0, left = a.budget;
  for (int d = 0; d < 3; ++d) {
    hist[t] = 0;
    hist[t + kThreads] = 0;
    __syncthreads();
    x.count(hist, prefix, d);
    __syncthreads();
    uint32_t bin, above;
    find_bin(hist, left, waves, found, &bin, &above);
    prefix |= bin << digit_shift(d);
    left -= above;
  }
  uint32_t holes;
  assign(a, x, row, prefix, left, waves, 0, 0, 0, &holes);
  if (t == 0) a.moves[row] = holes;
}

// ---------------------------------------------------------------- long rows
// Chunks of a row: those of [0, budget), then those of [budget, length), so
// that a chunk frees slots or fills them, never both.
struct Chunk {
  uint32_t first, end;  // slots
};
__device__ __forceinline__ Chunk chunk_at(const hkv::EvictArgs& a, uint32_t c, uint32_t len) {
  const uint32_t low = (a.budget + kChunkSlots - 1) / kChunkSlots;
  const uint32_t lo = c < low ? c * kChunkSlots : a.budget + (c - low) * kChunkSlots;
  const uint32_t limit = c < low ? (a.budget < len ? a.budget : len) : len;
  const uint32_t first = lo < limit ? lo : limit;
  return Chunk{first, limit - first < kChunkSlots ? limit : first + kChunkSlots};
}

struct Row {
  uint32_t row, s, len;
  int32_t next;
  bool evicts;
};
__device__ __forceinline__ Row row_at(const hkv::EvictArgs& a) {
  Row r;
  r.row = blockIdx.y;
  r.s = r.row % a.n_seqs;
  const int32_t len = a.lens[r.s];
  r.len = valid_len(a, len) ? (uint32_t)len : 0u;
  r.next = a.next[r.s];
  r.evicts = a.ok[r.s] != 0 && r.len > a.budget;
  return r;
}

// The first `digits` digits of the least kept key, from the histograms.
__device__ __forceinline__ void prefix_of(const hkv::EvictArgs& a, uint32_t row, int digits,
                                          uint32_t* waves, uint32_t* found, uint32_t* prefix,
                                          uint32_t* left) {
  *prefix = 0;
  *left = a.budget;
  for (int d = 0; d < digits; ++d) {
    uint32_t bin, above;
    find_bin(a.hist + ((uint64_t)row * 3 + d) * kBins, *left, waves, found, &bin, &above);
    *prefix |= bin << digit_shift(d);
    *left -= above;
  }
}

template <int kDigit>
__device__ __forceinline__ void count_digit(const hkv::EvictArgs& a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t waves[kWaves];
  __shared__ uint32_t found[2];
  const Row r = row_at(a);
  const Chunk c = chunk_at(a, blockIdx.x, r.len);
  if (!r.evicts || c.first == c.end) return;
  const uint32_t t = threadIdx.x;
  const int64_t base = meta_row(a, r.row);
  Slots<kChunkItems> x;
  x.load(a, a.weights + base, a.positions + base, c.first + t * kChunkItems, c.end, r.next);
  uint32_t prefix, left;
  prefix_of(a, r.row, kDigit, waves, found, &prefix, &left);
  hist[t] = 0;
  hist[t + kThreads] = 0;
  __syncthreads();
  x.count(hist, prefix, kDigit);
  __syncthreads();
  uint32_t* out = a.hist + ((uint64_t)r.row * 3 + kDigit) * kBins;
  for (uint32_t i = t; i < kBins; i += kThreads)
    if (hist[i])  // whole numbers: the order of the additions does not matter
      __hip_atomic_fetch_add(out + i, hist[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

#define HKV_SELECT(items)                                                             \
  extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_select_##items( \
      hkv::EvictArgs a) {                                                             \
    select<items>(a);                                                                 \
  }
HKV_SELECT(4)
HKV_SELECT(16)
#undef HKV_SELECT

// Which sequences can be evicted from, for calls with many block ids: one
// workgroup, which clears and counts only the ids that the tables name.
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_check(hkv::EvictArgs a) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int phase = 0; phase < 3; ++phase) {
    for (uint32_t s = wave; s < a.n_seqs; s += kWaves) {
      const int32_t len = a.lens[s];
      bool good = valid_len(a, len);
      const uint32_t blocks = blocks_of(a, len);
      for (uint32_t j = lane; j < blocks; j += 64) {
        const int32_t id = a.table[(int64_t)s * a.table_stride + j];
        if (id < 0 || (uint32_t)id >= a.num_blocks) {
          good = false;
          continue;
        }
        if (phase == 0)
          __hip_atomic_store(a.claims + id, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else if (phase == 1)
          __hip_atomic_fetch_add(a.claims + id, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else if (__hip_atomic_load(a.claims + id, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT) != 1)
          good = false;
      }
      if (phase == 2) {
        good = __all(good);
        if (lane == 0) {
          a.ok[s] = good;
          write_new_len(a, s, good);
        }
      }
    }
    __threadfence();
    __syncthreads();
  }
}

// Long rows, before the first digit: cleared histograms, and (for calls with
// few block ids) the check of each sequence.
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_clear(hkv::EvictArgs a) {
  __shared__ int32_t own[hkv::kEvictPairBlocks];
  __shared__ uint32_t bad;
  const uint32_t row = blockIdx.x;
  uint32_t* h = a.hist + (uint64_t)row * 3 * kBins;
  for (uint32_t i = threadIdx.x; i < 3 * kBins; i += kThreads) h[i] = 0;
  if (a.by_pairs && row < a.n_seqs) {
    const bool ok = check_by_pairs(a, row, own, &bad);
    if (threadIdx.x == 0) {
      a.ok[row] = ok;
      write_new_len(a, row, ok);
    }
  }
}

extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_digit0(hkv::EvictArgs a) {
  count_digit<0>(a);
}
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_digit1(hkv::EvictArgs a) {
  count_digit<1>(a);
}
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_digit2(hkv::EvictArgs a) {
  count_digit<2>(a);
}

// Long rows: each chunk's keys above the least kept one, and its ties.
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_totals(hkv::EvictArgs a) {
  __shared__ uint32_t waves[kWaves];
  __shared__ uint32_t found[2];
  const Row r = row_at(a);
  const Chunk c = chunk_at(a, blockIdx.x, r.len);
  if (!r.evicts) return;
  const int64_t base = meta_row(a, r.row);
  Slots<kChunkItems> x;
  x.load(a, a.weights + base, a.positions + base, c.first + threadIdx.x * kChunkItems, c.end,
         r.next);
  uint32_t prefix, left, above = 0, ties = 0;
  prefix_of(a, r.row, 3, waves, found, &prefix, &left);
#pragma unroll
  for (uint32_t i = 0; i < kChunkItems; ++i) {
    above += i < x.n && x.key[i] > prefix;
    ties += i < x.n && x.key[i] == prefix;
  }
  uint32_t all_above, all_ties;
  block_scan(above, waves, &all_above);
  block_scan(ties, waves, &all_ties);
  if (threadIdx.x == 0) {
    uint32_t* out = a.totals + ((uint64_t)r.row * a.chunks + blockIdx.x) * 2;
    out[0] = all_above;
    out[1] = all_ties;
    if (blockIdx.x == 0) {
      a.least[r.row * 2] = prefix;
      a.least[r.row * 2 + 1] = left;
    }
  }
}

// Long rows: the lists, and the weights and positions of slots that do not move.
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_assign(hkv::EvictArgs a) {
  __shared__ uint32_t waves[kWaves];
  const Row r = row_at(a);
  const Chunk c = chunk_at(a, blockIdx.x, r.len);
  if (!r.evicts) {
    copy_meta(a, r.row, c.first, c.end);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.moves[r.row] = 0;
    return;
  }
  const int64_t base = meta_row(a, r.row);
  Slots<kChunkItems> x;
  x.load(a, a.weights + base, a.positions + base, c.first + threadIdx.x * kChunkItems, c.end,
         r.next);
  const uint32_t least = a.least[r.row * 2], left = a.least[r.row * 2 + 1];
  // What comes before this chunk, from the chunks' totals; and over all of the
  // row's lower chunks the number of moves.
  const uint32_t low = (a.budget + kChunkSlots - 1) / kChunkSlots;
  uint32_t ties = 0, holes = 0, movers = 0, moves = 0, all_ties = 0;
  for (uint32_t i = 0; i < a.chunks && (i < blockIdx.x || i < low); ++i) {
    const uint32_t* tot = a.totals + ((uint64_t)r.row * a.chunks + i) * 2;
    const Chunk ci = chunk_at(a, i, r.len);
    const uint32_t open = all_ties < left ? left - all_ties : 0;  // ties that may still stay
    const uint32_t kept = tot[0] + (tot[1] < open ? tot[1] : open);
    const uint32_t freed = ci.end - ci.first - kept;
    if (i < low) moves += freed;
    if (i < blockIdx.x) {
      ties += tot[1];
      if (i < low)
        holes += freed;
      else
        movers += kept;
    }
    all_ties += tot[1];
  }
  uint32_t all;
  assign(a, x, r.row, least, left, waves, ties, holes, movers, &all);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.moves[r.row] = moves;
}

namespace {

constexpr uint32_t kMoveThreads = 256;
constexpr uint32_t kMoveRows = 8;  // rows a wave moves together

// The rows of one wave's moves, as one run of kUnit-byte pieces over all its
// lanes.  Lane i < count holds row i's addresses.
template <class V>
__device__ __forceinline__ void move_rows(uint64_t src, uint64_t dst, uint32_t count,
                                          uint32_t row_bytes) {
  const uint32_t lane = threadIdx.x & 63, per = row_bytes / sizeof(V), total = count * per;
  constexpr uint32_t kUnroll = 3;
  for (uint32_t c0 = 0; c0 < total; c0 += 64 * kUnroll) {
    V v[kUnroll];
    HKV_GLOBAL V* to[kUnroll];
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u) {
      const uint32_t c = c0 + u * 64 + lane;
      const uint32_t r = c < total ? c / per : 0, off = c - r * per;
      const uint64_t from = __shfl((unsigned long long)src, (int)r, 64);
      to[u] = (HKV_GLOBAL V*)__shfl((unsigned long long)dst, (int)r, 64) + off;
      if (c < total) v[u] = __builtin_nontemporal_load((const HKV_GLOBAL V*)from + off);
    }
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u)
      if (c0 + u * 64 + lane < total) __builtin_nontemporal_store(v[u], to[u]);
  }
}

}  // namespace

extern "C" __global__ __launch_bounds__(kMoveThreads) void hkv_mla_evict_move(
    hkv::EvictArgs a) {
  const uint32_t row = blockIdx.y, s = row % a.n_seqs, lane = threadIdx.x & 63;
  const uint32_t first = (blockIdx.x * (kMoveThreads / 64) + (threadIdx.x >> 6)) * kMoveRows;
  const uint32_t moves = a.moves[row];
  if (first >= moves) return;
  const uint32_t count = moves - first < kMoveRows ? moves - first : kMoveRows;
  uint64_t src = 0, dst = 0;
  if (lane < count) {
    const uint32_t* holes = a.lists + (uint64_t)row * 2 * a.max_moves;
    const uint32_t to = holes[first + lane], from = holes[a.max_moves + first + lane];
    const int32_t* table = a.table + (int64_t)s * a.table_stride;
    uint8_t* pages = a.pool + a.page_of[row / a.n_seqs];
    auto at = [&](uint32_t slot) {
      const uint32_t j = slot / a.block_tokens;
      return reinterpret_cast<uint64_t>(pages + (uint64_t)(uint32_t)table[j] * a.stride +
                                        (uint64_t)(slot - j * a.block_tokens) * a.row_bytes);
    };
    src = at(from);
    dst = at(to);
    const int64_t base = meta_row(a, row);
    const float w = a.weights[base + from];
    const int32_t p = a.positions[base + from];
    a.weights_out[base + to] = w;
    a.positions_out[base + to] = p;
    a.weights_out[base + from] = 0.0f;
    a.positions_out[base + from] = -1;
  }
  if (((a.row_bytes | a.stride | a.page_of[row / a.n_seqs]) & 15) == 0)
    move_rows<v4u>(src, dst, count, a.row_bytes);
  else
    move_rows<uint8_t>(src, dst, count, a.row_bytes);
}

namespace hkv {

int launch_evict(const EvictArgs& a, void* stream) {
  EvictArgs arg = a;
  void* params[] = {&arg};
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const uint32_t rows = a.n_layers * a.n_seqs;
  hipError_t e = hipSuccess;
  auto launch = [&](auto* fn, dim3 grid, uint32_t threads) {
    if (e == hipSuccess)
      e = hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, dim3(threads), params, 0, st);
  };
  if (!a.by_pairs) launch(&hkv_mla_evict_check, dim3(1), kThreads);
  const uint64_t slots = (uint64_t)a.max_blocks * a.block_tokens;
  if (slots <= 4 * kThreads) {
    launch(&hkv_mla_evict_select_4, dim3(rows), kThreads);
  } else if (slots <= kEvictSelectSlots) {
    launch(&hkv_mla_evict_select_16, dim3(rows), kThreads);
  } else {
    launch(&hkv_mla_evict_clear, dim3(rows), kThreads);
    launch(&hkv_mla_evict_digit0, dim3(a.chunks, rows), kThreads);
    launch(&hkv_mla_evict_digit1, dim3(a.chunks, rows), kThreads);
    launch(&hkv_mla_evict_digit2, dim3(a.chunks, rows), kThreads);
    launch(&hkv_mla_evict_totals, dim3(a.chunks, rows), kThreads);
    launch(&hkv_mla_evict_assign, dim3(a.chunks, rows), kThreads);
  }
  const uint32_t per_group = kMoveThreads / 64 * kMoveRows;
  if (a.max_moves)
    launch(&hkv_mla_evict_move, dim3((a.max_moves + per_group - 1) / per_group, rows),
           kMoveThreads);
  return (int)e;
}

}  // namespace hkv
