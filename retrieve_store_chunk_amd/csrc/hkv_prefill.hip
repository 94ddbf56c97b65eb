// The KDA layers' prompt form: many tokens of each sequence, from the state
// page of one block to the pages of the sequence's blocks (gfx950).
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

struct Bf16 {
  typedef __bf16 type;
  static __device__ __forceinline__ void store4(void* p, v4f x) {
    const v2b a = {(__bf16)x[0], (__bf16)x[1]}, b = {(__bf16)x[2], (__bf16)x[3]};
    *(HKV_GLOBAL v2u*)p = v2u{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  }
};
struct Fp16 {
  typedef _Float16 type;
  static __device__ __forceinline__ void store4(void* p, v4f x) {
    const v2h a = {(_Float16)x[0], (_Float16)x[1]}, b = {(_Float16)x[2], (_Float16)x[3]};
    *(HKV_GLOBAL v2u*)p = v2u{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  }
};
struct Fp32 {
  typedef float type;
  static __device__ __forceinline__ void store4(void* p, v4f x) { *(HKV_GLOBAL v4f*)p = x; }
};

// ---------------------------------------------------------------- plan
constexpr uint32_t kPlanThreads = 256;

// A sequence's rows of the call and the blocks that its tokens lie in.  `known`:
// the rows lie in [0, n_tokens); `blocks`: its positions lie in its table.
struct Span {
  int32_t row, tokens, position;
  uint32_t first, last;  // table entries
  bool known, blocks;
};
__device__ __forceinline__ Span span_of(const hkv::PrefillArgs& a, uint32_t s) {
  Span p;
  const int32_t lo = a.starts[s], hi = a.starts[s + 1];
  p.known = lo >= 0 && hi >= lo && hi <= (int32_t)a.n_tokens;
  p.row = lo;
  p.tokens = p.known ? hi - lo : 0;
  p.position = a.positions[s];
  const int64_t cap = (int64_t)a.max_blocks * a.block_tokens;
  p.blocks = p.tokens > 0 && p.position >= 0 && (int64_t)p.position + p.tokens <= cap;
  p.first = p.blocks ? (uint32_t)p.position / a.block_tokens : 0;
  p.last = p.blocks ? (uint32_t)(p.position + (p.tokens - 1)) / a.block_tokens : 0;
  return p;
}

__device__ __forceinline__ bool outside(int32_t id, uint32_t num_blocks) {
  return id != HKV_NULL_BLOCK && (id < 0 || (uint32_t)id >= num_blocks);
}

// What becomes of each sequence (hkv.h), one workgroup each.  Blocks are compared
// with those of all sequences: entries are few (a block holds hundreds of tokens).
__device__ __forceinline__ void plan(const hkv::PrefillArgs& a) {
  __shared__ int32_t most;
  __shared__ uint32_t refused;
  const uint32_t s = blockIdx.x, t = threadIdx.x;
  if (t == 0) {
    most = INT32_MIN;
    refused = 0;
  }
  __syncthreads();
  const Span me = span_of(a, s);
  int32_t top = INT32_MIN;  // starts decrease somewhere before: the rows may be another's
  for (uint32_t r = t; r < s; r += kPlanThreads) top = max(top, a.starts[r]);
  if (top > INT32_MIN) atomicMax(&most, top);
  const int32_t* own = a.table + (int64_t)s * a.table_stride;
  const int32_t src = a.src[s];
  bool bad = !me.blocks || me.tokens > (int32_t)a.max_seq_tokens || outside(src, a.num_blocks);
  if (!bad) {
    for (uint32_t j = me.first + t; j <= me.last; j += kPlanThreads) {
      const int32_t id = own[j];
      bad |= outside(id, a.num_blocks);
      for (uint32_t i = me.first; i < j; ++i) bad |= id >= 0 && own[i] == id;
    }
    for (uint32_t r = t; r < a.n_seqs; r += kPlanThreads) {
      if (r == s) continue;
      const Span p = span_of(a, r);
      if (p.tokens == 0) continue;
      const int32_t from = a.src[r];
      const int32_t* theirs = a.table + (int64_t)r * a.table_stride;
      for (uint32_t j = me.first; j <= me.last; ++j) {
        const int32_t id = own[j];
        if (id < 0) continue;
        bad |= id == from;
        if (p.blocks)
          for (uint32_t i = p.first; i <= p.last; ++i) bad |= theirs[i] == id;
      }
    }
  }
  if (bad) atomicOr(&refused, 1u);
  __syncthreads();
  if (t == 0)
    a.status[s] = !me.known || me.tokens == 0 || most > me.row ? hkv::kPrefillNoRows
                  : refused                                    ? hkv::kPrefillRefused
                                                               : hkv::kPrefillRuns;
}

// ---------------------------------------------------------------- token by token
// hkv_kda_step's arithmetic with the state and the conv's taps kept in registers
// from token to token: one workgroup per (head, sequence).
template <class T, uint32_t kD, uint32_t kThreads>
__device__ __forceinline__ void tokens(const hkv::PrefillArgs& a) {
  using E = typename T::type;
  constexpr uint32_t kRowThreads = kD / 4;               // threads that hold a row
  constexpr uint32_t kGroups = kThreads / kRowThreads;   // rows held at a time
  constexpr uint32_t kRows = kD / kGroups;               // rows per thread
  constexpr uint32_t kWaves = kThreads / 64;
  constexpr uint32_t kChannels = (3 * kD + kThreads - 1) / kThreads;  // conv rows per thread
  static_assert(kGroups * kRows == kD && kRowThreads <= 64, "a head splits into whole rows");
  // two of each, by the token's parity: the next token's are written while slower
  // waves still read this one's
  __shared__ float y[2][3][kD];  // q, k, v after the conv
  __shared__ float decay[2][kD];
  __shared__ v4f sums[2][kWaves][kRowThreads];
  const uint32_t h = blockIdx.x, s = blockIdx.y, t = threadIdx.x, lane = t & 63;
  const uint32_t c = t % kRowThreads, r0 = t / kRowThreads;
  const int32_t status = a.status[s];
  if (status == hkv::kPrefillNoRows) return;
  const int32_t row0 = a.starts[s], n = a.starts[s + 1] - row0;
  E* const out = static_cast<E*>(a.out) + (int64_t)row0 * a.out_stride + (int64_t)h * kD + c * 4;
  if (status == hkv::kPrefillRefused) {
    for (uint32_t i = r0; i < (uint32_t)n; i += kGroups)
      T::store4(out + (int64_t)i * a.out_stride, v4f{NAN, NAN, NAN, NAN});
    return;
  }
  const int32_t src = a.src[s], position = a.positions[s];
  const int32_t* const table = a.table + (int64_t)s * a.table_stride;
  const uint64_t state_off = a.conv_bytes + (uint64_t)h * kD * kD * 4;
  const uint32_t state_at = r0 * kRowThreads + c;  // in units of four values
  const uint32_t keep = a.taps - 1;

  v4f st[kRows];
  {
    const HKV_GLOBAL v4f* p =
        (const HKV_GLOBAL v4f*)(a.pages + (uint64_t)(src < 0 ? 0 : src) * a.stride + state_off) +
        state_at;
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      st[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (src >= 0) st[i] = p[i * kGroups * kRowThreads];
    }
  }
  // One thread per channel: its weights, its last `keep` values (oldest first).
  E taps[kChannels][hkv::kKdaMaxKernel - 1];
  float weight[kChannels][hkv::kKdaMaxKernel];
#pragma unroll
  for (uint32_t i = 0; i < kChannels; ++i) {
    const uint32_t w = t + i * kThreads;
    if (w >= 3 * kD) break;
    const uint64_t ch = ((uint64_t)(w / kD) * a.heads + h) * kD + w % kD;
    const E* wt = static_cast<const E*>(a.conv_weight) + ch * a.taps;
    const E* old = reinterpret_cast<const E*>(a.pages + (uint64_t)(src < 0 ? 0 : src) * a.stride) +
                   ch * keep;
#pragma unroll
    for (uint32_t j = 0; j < hkv::kKdaMaxKernel; ++j) weight[i][j] = j <= keep ? (float)wt[j] : 0.0f;
#pragma unroll
    for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
      taps[i][j] = j < keep && src >= 0 ? old[j] : (E)0.0f;
  }

  for (int32_t m = 0; m < n; ++m) {
    const int64_t row = (int64_t)row0 + m;
    const uint32_t b = m & 1;
#pragma unroll
    for (uint32_t i = 0; i < kChannels; ++i) {
      const uint32_t w = t + i * kThreads;
      if (w >= 3 * kD) break;
      const uint64_t ch = ((uint64_t)(w / kD) * a.heads + h) * kD + w % kD;
      const E x = static_cast<const E*>(a.x)[row * a.x_stride + (int64_t)ch];
      float sum = 0.0f;
#pragma unroll
      for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
        if (j < keep) sum += weight[i][j] * (float)taps[i][j];
#pragma unroll
      for (uint32_t j = 0; j < hkv::kKdaMaxKernel; ++j)
        if (j == keep) sum += weight[i][j] * (float)x;
#pragma unroll
      for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j) {
        if (j + 1 < keep) taps[i][j] = taps[i][j + 1 < hkv::kKdaMaxKernel - 1 ? j + 1 : j];
        if (j + 1 == keep) taps[i][j] = x;
      }
      y[b][w / kD][w % kD] = sum / (1.0f + expf(-sum));
    }
    for (uint32_t i = t; i < kD; i += kThreads) {
      const float g = a.log_decay[row * a.decay_stride + (int64_t)h * kD + i];
      decay[b][i] = expf(g > 0.0f ? 0.0f : g);
    }
    const float beta = a.beta[row * a.beta_stride + h];
    __syncthreads();

    // |q|^2, |k|^2 and q.k, by every wave for itself.
    float qq = 0.0f, kk = 0.0f, qk = 0.0f;
    for (uint32_t i = lane; i < kD; i += 64) {
      const float q = y[b][0][i], k = y[b][1][i];
      qq += q * q;
      kk += k * k;
      qk += q * k;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      qq += __shfl_xor(qq, d, 64);
      kk += __shfl_xor(kk, d, 64);
      qk += __shfl_xor(qk, d, 64);
    }
    const float nq = a.scale / sqrtf(qq + a.eps), nk = 1.0f / sqrtf(kk + a.eps);

    v4f sk = {0.0f, 0.0f, 0.0f, 0.0f}, sq = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      const uint32_t r = r0 + i * kGroups;
      st[i] *= decay[b][r];
      sk += st[i] * (y[b][1][r] * nk);
      sq += st[i] * (y[b][0][r] * nq);
    }
#pragma unroll
    for (uint32_t d = kRowThreads; d < 64; d <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sk[i] += __shfl_xor(sk[i], (int)d, 64);
        sq[i] += __shfl_xor(sq[i], (int)d, 64);
      }
    if (kWaves > 1) {
      if (lane < kRowThreads) {
        sums[0][t >> 6][c] = sk;
        sums[1][t >> 6][c] = sq;
      }
      __syncthreads();
      sk = sums[0][0][c];
      sq = sums[1][0][c];
#pragma unroll
      for (uint32_t w = 1; w < kWaves; ++w) {
        sk += sums[0][w][c];
        sq += sums[1][w][c];
      }
    }
    v4f u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = beta * (y[b][2][c * 4 + i] - sk[i]);
    if (r0 == 0) T::store4(out + (int64_t)m * a.out_stride, sq + u * (qk * nq * nk));
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) st[i] += u * (y[b][1][r0 + i * kGroups] * nk);

    const uint32_t at = (uint32_t)(position + m);
    if ((at + 1) % a.block_tokens != 0 && m != n - 1) continue;
    const int32_t dst = table[at / a.block_tokens];
    if (dst < 0) continue;
    HKV_GLOBAL v4f* p =
        (HKV_GLOBAL v4f*)(a.pages + (uint64_t)dst * a.stride + state_off) + state_at;
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) p[i * kGroups * kRowThreads] = st[i];
#pragma unroll
    for (uint32_t i = 0; i < kChannels; ++i) {
      const uint32_t w = t + i * kThreads;
      if (w >= 3 * kD) break;
      const uint64_t ch = ((uint64_t)(w / kD) * a.heads + h) * kD + w % kD;
      E* to = reinterpret_cast<E*>(a.pages + (uint64_t)dst * a.stride) + ch * keep;
#pragma unroll
      for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
        if (j < keep) to[j] = taps[i][j];
    }
  }
}

}  // namespace

extern "C" __global__ __launch_bounds__(kPlanThreads) void hkv_kda_prefill_plan(
    hkv::PrefillArgs a) {
  plan(a);
}

// Threads by head dim, as in the step's kernels.
#define HKV_TOKENS(name, T, d, threads)                                     \
  extern "C" __global__ __launch_bounds__(threads, 4) void name(            \
      hkv::PrefillArgs a) {                                                 \
    tokens<T, d, threads>(a);                                               \
  }
#define HKV_TOKENS_DIMS(suffix, T)                        \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d16, T, 16, 64)    \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d32, T, 32, 64)    \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d64, T, 64, 256)   \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d128, T, 128, 512) \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d256, T, 256, 1024)
HKV_TOKENS_DIMS(bf16, Bf16)
HKV_TOKENS_DIMS(fp16, Fp16)
HKV_TOKENS_DIMS(fp32, Fp32)
#undef HKV_TOKENS
#undef HKV_TOKENS_DIMS

namespace hkv {

int launch_prefill(const PrefillArgs& a, int32_t dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
#define HKV_DIMS(suffix)                                                                \
  {HKV_FN(hkv_kda_tokens_##suffix##_d16), HKV_FN(hkv_kda_tokens_##suffix##_d32),        \
   HKV_FN(hkv_kda_tokens_##suffix##_d64), HKV_FN(hkv_kda_tokens_##suffix##_d128),       \
   HKV_FN(hkv_kda_tokens_##suffix##_d256)}
  static const void* const kTokens[3][5] = {HKV_DIMS(bf16), HKV_DIMS(fp16), HKV_DIMS(fp32)};
#undef HKV_DIMS
  static const uint32_t kThreads[5] = {64, 64, 256, 512, 1024};
  uint32_t i = 0;
  while (i < 4 && (16u << i) != a.head_dim) ++i;
  PrefillArgs arg = a;
  void* params[] = {&arg};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipLaunchKernel(HKV_FN(hkv_kda_prefill_plan), dim3(a.n_seqs), dim3(kPlanThreads),
                                 params, 0, st);
  if (e != hipSuccess) return (int)e;
  return (int)hipLaunchKernel(kTokens[dtype][i], dim3(a.heads, a.n_seqs), dim3(kThreads[i]),
                              params, 0, st);
#undef HKV_FN
}

}  // namespace hkv
