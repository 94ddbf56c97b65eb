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
// Rows of up to kEvictSelectSlots: one workgroup a row, which holds the row's
// keys in registers through all of it.  Longer rows: workgroups of
// kEvictChunkSlots slots count into histograms in the workspace, one launch a
// digit, then one for each chunk's totals and one for the lists.
//
// Bound: 8 bytes read and 8 written per slot, and each moved row read and
// written once; only rows that must move do.  Measured: 16 sequences of up to
// 8192 slots, 7 layers, bf16, half of them kept: 63 us, of which the selection
// 20 and the moves 43 to 47; 1 sequence of 262144 slots, 24 layers, e4m3, 100000
// kept: 485 us, the moves 370 at 4.6 TB/s (torch's copy reaches 4.8, the best
// copying kernel here 5.9 between contiguous buffers), the passes
// over the slots 112; 4 sequences of up to 1500, 1 layer: 13 us, two launches.
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef int32_t v4i __attribute__((ext_vector_type(4)));
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
__device__ __forceinline__ bool check_by_pairs(const hkv::EvictArgs& a, uint32_t s, v4i* own,
                                               uint32_t* bad) {
  const uint32_t t = threadIdx.x;
  const int32_t len = a.lens[s];
  const uint32_t blocks = blocks_of(a, len);
  if (t == 0) *bad = !valid_len(a, len);
  __syncthreads();
  const uint32_t quads = (blocks + 3) / 4;
  for (uint32_t j = t; j < quads * 4; j += kThreads) {
    const int32_t id = j < blocks ? a.table[(int64_t)s * a.table_stride + j] : -1;
    ((int32_t*)own)[j] = id;
    if (j < blocks && (id < 0 || (uint32_t)id >= a.num_blocks)) *bad = 1;
  }
  __syncthreads();
  for (uint32_t i = t; i < a.n_seqs * a.max_blocks; i += kThreads) {
    const uint32_t s2 = i / a.max_blocks, j2 = i - s2 * a.max_blocks;
    if (j2 >= blocks_of(a, a.lens[s2])) continue;
    const int32_t id = a.table[(int64_t)s2 * a.table_stride + j2];
    int same = s2 == s ? -1 : 0;  // it meets itself once
#pragma unroll 4
    for (uint32_t j = 0; j < quads; ++j) {
      const v4i o = own[j];
      same += (o[0] == id) + (o[1] == id) + (o[2] == id) + (o[3] == id);
    }
    if (id >= 0 && same > 0) *bad = 1;
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

// A workgroup's slots [first, end) of a row, at most kItems x kThreads: group g
// of four of thread t starts at first + (g x kThreads + t) x 4, so that a
// wave's loads and stores are of consecutive bytes.
template <uint32_t kItems>
struct Slots {
  static constexpr uint32_t kGroups = kItems / 4;
  static_assert(kGroups >= 1 && kGroups <= 4, "a count of each group in 16 bits of 64");
  float w[kItems];
  int32_t pos[kItems];
  uint32_t key[kItems];
  uint32_t first, end;
  __device__ __forceinline__ uint32_t slot(uint32_t i) const {
    return first + (i / 4 * kThreads + threadIdx.x) * 4 + i % 4;
  }
  __device__ __forceinline__ bool live(uint32_t i) const { return slot(i) < end; }
  __device__ __forceinline__ void load(const hkv::EvictArgs& a, const float* wp,
                                       const int32_t* pp, uint32_t from, uint32_t to,
                                       int32_t next) {
    first = from;
    end = to;
#pragma unroll
    for (uint32_t g = 0; g < kGroups; ++g) {
      const uint32_t at = slot(g * 4);
      v4f_a4 x = {0.0f, 0.0f, 0.0f, 0.0f};
      v4i_a4 y = {0, 0, 0, 0};
      if (at + 4 <= end) {  // (aligned to one value: global loads may be)
        x = *(const HKV_GLOBAL v4f_a4*)(wp + at);
        y = *(const HKV_GLOBAL v4i_a4*)(pp + at);
      } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          if (at + k < end) {
            x[k] = wp[at + k];
            y[k] = pp[at + k];
          }
      }
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        w[g * 4 + k] = x[k];
        pos[g * 4 + k] = y[k];
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i) key[i] = key_of(w[i], is_held(a, pos[i], next));
  }
  __device__ __forceinline__ void count(uint32_t* hist, uint32_t prefix, int d) const {
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i)
      if (live(i) && (key[i] & above_mask(d)) == prefix)
        atomicAdd(&hist[(key[i] >> digit_shift(d)) & digit_mask(d)], 1u);
  }
};

// The exclusive prefix over the workgroup of four 16-bit counts at once, and
// their totals.
__device__ __forceinline__ uint64_t block_scan4(uint64_t x, uint64_t* waves, uint64_t* total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t scan = x;
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t up = __shfl_up((unsigned long long)scan, d, 64);
    if (lane >= (uint32_t)d) scan += up;
  }
  if (lane == 63) waves[wave] = scan;
  __syncthreads();
  uint64_t before = scan - x, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

// In slot order: which ties with the smallest kept key stay (the first `left`
// of them), and the number of each move.  `ties`, `moves`: how many ties, and
// how many freed (or filling) slots, come before this workgroup's.  Writes the
// lists, and the weights and positions of every slot that does not move; the
// two slots of a move keep theirs for the move kernel.  kWhole: the workgroup
// has the whole row, else slots of one side of the budget.
template <uint32_t kItems, bool kWhole>
__device__ __forceinline__ void assign(const hkv::EvictArgs& a, const Slots<kItems>& x,
                                       uint32_t row, uint32_t least, uint32_t left,
                                       uint64_t* waves, uint32_t ties, uint32_t moves,
                                       uint32_t* all_moves) {
  constexpr uint32_t kGroups = Slots<kItems>::kGroups;
  auto add_group = [](uint64_t n, uint32_t g, uint32_t by) { return n + ((uint64_t)by << 16 * g); };
  auto group = [](uint64_t n, uint32_t g) { return (uint32_t)(n >> 16 * g) & 0xFFFFu; };
  uint64_t n = 0, all;
#pragma unroll
  for (uint32_t i = 0; i < kItems; ++i) n = add_group(n, i / 4, x.live(i) && x.key[i] == least);
  uint64_t before = block_scan4(n, waves, &all);
  uint32_t keep = 0;  // one bit a slot
  uint64_t m = 0;     // slots that are freed below the budget, or kept from it on
#pragma unroll
  for (uint32_t g = 0; g < kGroups; ++g) {
    uint32_t rank = ties + group(before, g);
#pragma unroll
    for (uint32_t i = g * 4; i < g * 4 + 4; ++i) {
      if (!x.live(i)) continue;
      const bool tie = x.key[i] == least;
      const bool k = x.key[i] > least || (tie && rank < left);
      rank += tie;
      keep |= (uint32_t)k << i;
      m = add_group(m, g, k != (x.slot(i) < a.budget));
    }
    ties += group(all, g);
  }
  before = block_scan4(m, waves, &all);
  uint32_t total = 0;
#pragma unroll
  for (uint32_t g = 0; g < kGroups; ++g) total += group(all, g);
  // Over a whole row as many slots are freed as fill them.
  *all_moves = kWhole ? total / 2 : total;
  const uint32_t fill0 = kWhole ? total / 2 : 0;
  const int64_t base = meta_row(a, row);
  uint32_t* list = a.lists + (uint64_t)row * 2 * a.max_moves;
#pragma unroll
  for (uint32_t g = 0; g < kGroups; ++g) {
    uint32_t number = moves + group(before, g);
    v4f_a4 wo;
    v4i_a4 po;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t i = g * 4 + k, slot = x.slot(i);
      const bool kept = keep >> i & 1, low = slot < a.budget;
      wo[k] = low || kept ? x.w[i] : 0.0f;
      po[k] = low || kept ? x.pos[i] : -1;
      if (x.live(i) && kept != low) {
        const uint32_t at = low ? number : number - fill0;
        if (at < a.max_moves) list[(low ? 0 : a.max_moves) + at] = slot;
        ++number;
      }
    }
    const uint32_t at = x.slot(g * 4);
    if (at + 4 <= x.end) {
      *(HKV_GLOBAL v4f_a4*)(a.weights_out + base + at) = wo;
      *(HKV_GLOBAL v4i_a4*)(a.positions_out + base + at) = po;
    } else {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (at + k < x.end) {
          a.weights_out[base + at + k] = wo[k];
          a.positions_out[base + at + k] = po[k];
        }
    }
    moves += group(all, g);
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
// One launch instead of the chunked path's six: 8000 slots 22 us for 38, 112 rows
// of 8192 23 for 42 (whole calls, when a chunked row of 20000 took 38; it takes 36
// now).  16 slots a thread, 48 registers of them, are
// as many as fit without spills; 4 a thread where they are enough (1500 slots: 13
// us, 19 with 16).
template <uint32_t kItems>
__device__ __forceinline__ void select(const hkv::EvictArgs& a) {
  __shared__ uint32_t hist[kBins];
  __shared__ v4i own[hkv::kEvictPairBlocks / 4];
  __shared__ uint32_t waves[kWaves];
  __shared__ uint64_t waves4[kWaves];
  __shared__ uint32_t found[2];
  __shared__ uint32_t bad;
  const uint32_t row = blockIdx.x, s = row % a.n_seqs, t = threadIdx.x;
  const int64_t base = meta_row(a, row);
  const int32_t raw_len = a.lens[s], next = a.next[s];
  const uint32_t len = valid_len(a, raw_len) ? (uint32_t)raw_len : 0u;
  // The loads are in flight while the block ids are checked.
  Slots<kItems> x;
  x.load(a, a.weights + base, a.positions + base, 0, len > a.budget ? len : 0u, next);
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
  uint32_t moves;
  assign<kItems, true>(a, x, row, prefix, left, waves4, 0, 0, &moves);
  if (t == 0) a.moves[row] = moves;
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

// The first `digits` digits of the least kept key and how many keys with them
// stay: the last of them from its histogram, the ones before it from what the
// launch before found.  The row's first workgroup leaves the result for the next.
__device__ __forceinline__ void prefix_of(const hkv::EvictArgs& a, uint32_t row, int digits,
                                          uint32_t* waves, uint32_t* found, uint32_t* prefix,
                                          uint32_t* left) {
  *prefix = 0;
  *left = a.budget;
  if (digits == 0) return;
  uint32_t* least = a.least + (uint64_t)row * 3 * 2 + (digits - 1) * 2;
  if (digits > 1) {
    *prefix = least[-2];
    *left = least[-1];
  }
  const int d = digits - 1;
  uint32_t bin, above;
  find_bin(a.hist + ((uint64_t)row * 3 + d) * kBins, *left, waves, found, &bin, &above);
  *prefix |= bin << digit_shift(d);
  *left -= above;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    least[0] = *prefix;
    least[1] = *left;
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
  x.load(a, a.weights + base, a.positions + base, c.first, c.end, r.next);
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
  __shared__ v4i own[hkv::kEvictPairBlocks / 4];
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
  x.load(a, a.weights + base, a.positions + base, c.first, c.end, r.next);
  uint32_t prefix, left, above = 0, ties = 0;
  prefix_of(a, r.row, 3, waves, found, &prefix, &left);
#pragma unroll
  for (uint32_t i = 0; i < kChunkItems; ++i) {
    above += x.live(i) && x.key[i] > prefix;
    ties += x.live(i) && x.key[i] == prefix;
  }
  uint32_t all_above, all_ties;
  block_scan(above, waves, &all_above);
  block_scan(ties, waves, &all_ties);
  if (threadIdx.x == 0) {
    uint32_t* out = a.totals + ((uint64_t)r.row * a.chunks + blockIdx.x) * 2;
    out[0] = all_above;
    out[1] = all_ties;
  }
}

// Long rows: the lists, and the weights and positions of slots that do not move.
extern "C" __global__ __launch_bounds__(kThreads) void hkv_mla_evict_assign(hkv::EvictArgs a) {
  __shared__ uint32_t waves[kWaves];
  __shared__ uint64_t waves4[kWaves];
  const Row r = row_at(a);
  const Chunk c = chunk_at(a, blockIdx.x, r.len);
  if (!r.evicts) {
    copy_meta(a, r.row, c.first, c.end);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.moves[r.row] = 0;
    return;
  }
  const int64_t base = meta_row(a, r.row);
  Slots<kChunkItems> x;
  x.load(a, a.weights + base, a.positions + base, c.first, c.end, r.next);
  const uint32_t least = a.least[r.row * 6 + 4], left = a.least[r.row * 6 + 5];
  // From the chunks' totals: the ties and the moves before this chunk, and the
  // row's moves.
  const uint32_t low = (a.budget + kChunkSlots - 1) / kChunkSlots;
  const uint32_t mine = blockIdx.x, lowest = mine < low ? 0 : low;
  uint32_t ties_all = 0, ties = 0, before = 0, moves = 0, all;
  for (uint32_t i0 = 0; i0 < a.chunks; i0 += kThreads) {
    const uint32_t i = i0 + threadIdx.x;
    uint32_t above = 0, n_ties = 0;
    if (i < a.chunks) {
      const uint32_t* tot = a.totals + ((uint64_t)r.row * a.chunks + i) * 2;
      above = tot[0];
      n_ties = tot[1];
    }
    const uint32_t at = ties_all + block_scan(n_ties, waves, &all);
    ties_all += all;
    const uint32_t open = at < left ? left - at : 0;  // ties that may still stay
    const uint32_t kept = above + (n_ties < open ? n_ties : open);
    const Chunk ci = chunk_at(a, i < a.chunks ? i : 0, r.len);
    const uint32_t n = i >= a.chunks ? 0 : i < low ? ci.end - ci.first - kept : kept;
    block_scan(i < mine ? n_ties : 0, waves, &all);
    ties += all;
    block_scan(i >= lowest && i < mine ? n : 0, waves, &all);
    before += all;
    block_scan(i < low ? n : 0, waves, &all);
    moves += all;
  }
  assign<kChunkItems, false>(a, x, r.row, least, left, waves4, ties, before, &all);
  if (mine == 0 && threadIdx.x == 0) a.moves[r.row] = moves;
}

namespace {

constexpr uint32_t kMoveThreads = 256;
constexpr uint32_t kMoveRows = 8;  // rows a wave moves together

// One wave's rows, 8 lanes to a row: each lane copies every eighth piece of its
// row, so that an instruction moves 128 consecutive bytes of each of 8 rows
// and a lane needs one address of each side.  Lane i < count holds row i's.
template <class V>
__device__ __forceinline__ void move_rows(uint64_t src, uint64_t dst, uint32_t count,
                                          uint32_t row_bytes) {
  const uint32_t lane = threadIdx.x & 63, r = lane / 8, pieces = row_bytes / sizeof(V);
  const uint64_t from = __shfl((unsigned long long)src, (int)r, 64);
  const uint64_t to = __shfl((unsigned long long)dst, (int)r, 64);
  if (r >= count) return;
  const HKV_GLOBAL V* f = (const HKV_GLOBAL V*)from;
  HKV_GLOBAL V* t = (HKV_GLOBAL V*)to;
  constexpr uint32_t kUnroll = 9;
  for (uint32_t c0 = lane & 7; c0 < pieces; c0 += 8 * kUnroll) {
    V v[kUnroll];
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u)
      if (c0 + u * 8 < pieces) v[u] = __builtin_nontemporal_load(f + c0 + u * 8);
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u)
      if (c0 + u * 8 < pieces) __builtin_nontemporal_store(v[u], t + c0 + u * 8);
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
