// Eviction from the MLA cache by accumulated attention weight (gfx950).
//
// Per (layer, sequence) longer than the budget B, a radix selection finds the
// B-th largest 32-bit key (protected slots above every weight, NaN below), a
// scan in slot order gives each kept slot past B the freed slot below B that
// it fills, and the move kernel copies those rows.  Kept slots past B and
// freed slots below B are equally many, a source is never a destination, so
// every row moves at most once, all at the same time and in place.
//
// Bound: 8 bytes read and 8 written per slot, and each moved row read and
// written once; only rows that must move do.
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

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

constexpr uint32_t kCheckThreads = 1024;
constexpr uint32_t kSelectThreads = 1024;
constexpr uint32_t kPerThread = 4;  // consecutive slots of a thread in the ordered scan

}  // namespace

// Which sequences can be evicted from: every live block id in the pool and
// named once in the call.  One workgroup: it clears and counts only the ids
// that the tables name.
extern "C" __global__ __launch_bounds__(kCheckThreads) void hkv_mla_evict_check(
    hkv::EvictArgs a) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  constexpr uint32_t kWaves = kCheckThreads / 64;
  for (int phase = 0; phase < 3; ++phase) {
    for (uint32_t s = wave; s < a.n_seqs; s += kWaves) {
      const int32_t len = a.lens[s];
      bool good = valid_len(a, len);
      const uint32_t blocks =
          good ? ((uint32_t)len + a.block_tokens - 1) / a.block_tokens : 0;
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
          if (a.new_lens)
            a.new_lens[s] = !good ? -1 : (uint32_t)len < a.budget ? len : (int32_t)a.budget;
        }
      }
    }
    __threadfence();
    __syncthreads();
  }
}

namespace {

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
  for (uint32_t w = 0; w < kSelectThreads / 64; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

}  // namespace

// One workgroup per (layer, sequence): the selection, the list of moves, and
// the weights and positions of every slot that does not move.
extern "C" __global__ __launch_bounds__(kSelectThreads) void hkv_mla_evict_select(
    hkv::EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t waves[kSelectThreads / 64];
  __shared__ uint32_t found[2];
  const uint32_t row = blockIdx.x, s = row % a.n_seqs, t = threadIdx.x;
  const int64_t base = meta_row(a, row);
  const float* w = a.weights + base;
  const int32_t* pos = a.positions + base;
  float* w_out = a.weights_out + base;
  int32_t* pos_out = a.positions_out + base;
  const int32_t raw_len = a.lens[s], next = a.next[s];
  const uint32_t len = valid_len(a, raw_len) ? (uint32_t)raw_len : 0u;
  if (!a.ok[s] || len <= a.budget) {
    if (w_out != w)
      for (uint32_t i = t; i < len; i += kSelectThreads) w_out[i] = w[i];
    if (pos_out != pos)
      for (uint32_t i = t; i < len; i += kSelectThreads) pos_out[i] = pos[i];
    if (t == 0) a.moves[row] = 0;
    return;
  }
  uint32_t prefix = 0, mask = 0, left = a.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (t < 256) hist[t] = 0;
    __syncthreads();
    for (uint32_t i = t; i < len; i += kSelectThreads) {
      const uint32_t key = key_of(w[i], is_held(a, pos[i], next));
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    if (t < 64) {  // four bins a lane, from the top: lane 0 has bins 252..255
      uint32_t n[4], sum = 0;
      for (int i = 0; i < 4; ++i) sum += n[i] = hist[255 - (t * 4 + i)];
      uint32_t scan = sum;
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(scan, d, 64);
        if (t >= (uint32_t)d) scan += up;
      }
      uint32_t above = scan - sum;
      for (int i = 0; i < 4; ++i) {
        if (above < left && left <= above + n[i]) {
          found[0] = 255 - (t * 4 + i);
          found[1] = above;
        }
        above += n[i];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= 255u << shift;
    left -= found[1];
    __syncthreads();
  }

  // In slot order: which ties stay, and the number of each move.
  uint32_t* holes = a.lists + (uint64_t)row * 2 * a.max_moves;
  uint32_t* movers = holes + a.max_moves;
  uint32_t ties = 0, n_holes = 0, n_movers = 0;
  for (uint32_t first = 0; first < len; first += kSelectThreads * kPerThread) {
    float wt[kPerThread];
    int32_t ps[kPerThread];
    uint32_t key[kPerThread], n = 0;
    const uint32_t i0 = first + t * kPerThread;
#pragma unroll
    for (uint32_t i = 0; i < kPerThread; ++i) {
      wt[i] = 0.0f;
      ps[i] = 0;
      if (i0 + i < len) {
        wt[i] = w[i0 + i];
        ps[i] = pos[i0 + i];
      }
      key[i] = key_of(wt[i], is_held(a, ps[i], next));
      n += i0 + i < len && key[i] == prefix;
    }
    uint32_t all;
    uint32_t rank = ties + block_scan(n, waves, &all);
    ties += all;
    bool keep[kPerThread];
    uint32_t flags = 0;  // holes below, movers in the upper half (at most 4096 of each)
#pragma unroll
    for (uint32_t i = 0; i < kPerThread; ++i) {
      const bool tie = key[i] == prefix;
      keep[i] = key[i] > prefix || (tie && rank < left);
      rank += i0 + i < len && tie;
      if (i0 + i < len) {
        if (i0 + i < a.budget)
          flags += !keep[i];
        else
          flags += (uint32_t)keep[i] << 16;
      }
    }
    const uint32_t before = block_scan(flags, waves, &all);
    uint32_t hole = n_holes + (before & 0xFFFF), mover = n_movers + (before >> 16);
    n_holes += all & 0xFFFF;
    n_movers += all >> 16;
#pragma unroll
    for (uint32_t i = 0; i < kPerThread; ++i) {
      const uint32_t slot = i0 + i;
      if (slot >= len) continue;
      if (slot < a.budget) {
        if (keep[i]) {
          w_out[slot] = wt[i];
          pos_out[slot] = ps[i];
        } else if (hole < a.max_moves) {
          holes[hole++] = slot;
        }
      } else if (keep[i]) {
        if (mover < a.max_moves) movers[mover++] = slot;
      } else {
        w_out[slot] = 0.0f;
        pos_out[slot] = -1;
      }
    }
  }
  if (t == 0) a.moves[row] = n_holes;
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
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&hkv_mla_evict_check), dim3(1),
                                 dim3(kCheckThreads), params, 0, st);
  if (e == hipSuccess)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&hkv_mla_evict_select), dim3(rows),
                        dim3(kSelectThreads), params, 0, st);
  const uint32_t per_group = kMoveThreads / 64 * kMoveRows;
  if (e == hipSuccess && a.max_moves)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&hkv_mla_evict_move),
                        dim3((a.max_moves + per_group - 1) / per_group, rows),
                        dim3(kMoveThreads), params, 0, st);
  return (int)e;
}

}  // namespace hkv
