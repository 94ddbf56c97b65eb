// The KDA layers' prompt form: many tokens of each sequence, from the state
// page of one block to the pages of the sequence's blocks (gfx950).
//
// Short runs go token by token (`tokens`), heads of 128 in longer runs by chunks of up
// to 64 tokens (`form`, then `scan`); other head dims, conv kernels but 4 and fp32
// inputs always go token by token.  `plan` looks the sequences through.
//
// Bound: the inputs, outputs and pages for short runs (61 runs of up to 5 tokens, 6 heads:
// 20 us for 50 MB) and a token's chain for longer ones (1500 tokens, us a token: heads of
// 16 to 64 0.7 to 0.9, of 128 1.4 to 1.5, of 256 2.9 to 3.1, which spill); for chunks
// `form`'s arithmetic and, where a sequence has few heads, `scan`'s chain from chunk to
// chunk.  Measured (us, form + scan): 1500 tokens, 6 heads 24 + 30; 1887 tokens, 16 heads
// 34 + 45; 16384 tokens, 6 heads 88 + 200 (in parts); 20011 tokens, 32 heads 528 to 597
// + 685 to 724; 16 runs of up to 2000, 32 heads 487 to 583 + 422 to 463, for 1.0 GB each, of
// which a copy at 4.7 TB/s would take 0.21 ms.
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
constexpr uint32_t kC = hkv::kPrefillChunk;

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

// Tokens up to the first block's end.
__device__ __forceinline__ uint32_t chunk_lead(const hkv::PrefillArgs& a, const Span& p) {
  if (!p.blocks) return 0;
  return min((uint32_t)p.tokens,
             a.block_tokens - (uint32_t)p.position % a.block_tokens);
}
__device__ __forceinline__ uint32_t chunks_of(const hkv::PrefillArgs& a, const Span& p) {
  if (!p.blocks || p.tokens <= (int32_t)a.short_tokens || p.tokens > (int32_t)a.max_seq_tokens)
    return 0;
  const uint32_t lead = chunk_lead(a, p), rest = (uint32_t)p.tokens - lead;
  return (lead + kC - 1) / kC + rest / a.block_tokens * ((a.block_tokens + kC - 1) / kC) +
         (rest % a.block_tokens + kC - 1) / kC;
}

// What a thread finds against sequence s, which shares the other sequences and the
// sequence's blocks among a workgroup's threads: 1: its rows may be another's, 2: it is
// refused.  Blocks are compared with those of all sequences where the call has few, as
// blocks of hundreds of tokens make it (at worst 26 entries with 26, on one thread);
// otherwise they were counted.
__device__ __forceinline__ uint32_t look_through(const hkv::PrefillArgs& a, uint32_t s,
                                                 const Span& me, uint32_t t, uint32_t threads) {
  uint32_t found = 0;
  for (uint32_t r = t; r < s; r += threads) found |= a.starts[r] > me.row ? 1u : 0u;
  const int32_t* own = a.table + (int64_t)s * a.table_stride;
  if (!me.blocks || me.tokens > (int32_t)a.max_seq_tokens || outside(a.src[s], a.num_blocks))
    return found | 2u;
  bool bad = false;
  if (a.counted) {
    const int32_t from = a.src[s];
    for (uint32_t j = me.first + t; j <= me.last; j += threads) {
      const int32_t id = own[j];
      bad |= outside(id, a.num_blocks);
      if (id < 0 || (uint32_t)id >= a.num_blocks) continue;
      const uint32_t* const uses = a.uses + (uint64_t)id * 2;
      bad |= uses[0] > 1 || uses[1] > (id == from ? 1u : 0u);
    }
    return found | (bad ? 2u : 0u);
  }
  for (uint32_t j = me.first + t; j <= me.last; j += threads) {
    const int32_t id = own[j];
    bad |= outside(id, a.num_blocks);
    for (uint32_t i = me.first; i < j; ++i) bad |= id >= 0 && own[i] == id;
  }
  for (uint32_t r = t; r < a.n_seqs; r += threads) {
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
  return found | (bad ? 2u : 0u);
}

// How many entries and how many sources of the call's sequences name a block, one
// workgroup a sequence: first the counts of the blocks that it names are cleared, then, in
// a launch of its own, they are counted (integers: their order does not matter).
__device__ __forceinline__ void count_uses(const hkv::PrefillArgs& a, bool clear) {
  const uint32_t s = blockIdx.x, t = threadIdx.x;
  const Span me = span_of(a, s);
  if (me.tokens == 0) return;
  auto use = [&](int32_t id, uint32_t which) {
    if (id < 0 || (uint32_t)id >= a.num_blocks) return;
    uint32_t* const uses = a.uses + (uint64_t)id * 2;
    if (clear)
      uses[0] = uses[1] = 0;
    else
      atomicAdd(uses + which, 1u);
  };
  if (t == 0) use(a.src[s], 1);
  if (!me.blocks) return;
  const int32_t* const own = a.table + (int64_t)s * a.table_stride;
  for (uint32_t j = me.first + t; j <= me.last; j += kPlanThreads) use(own[j], 0);
}

// What becomes of a sequence (hkv.h), from what its threads found.
__device__ __forceinline__ int32_t verdict(const Span& me, uint32_t found) {
  if (!me.known || me.tokens == 0 || (found & 1)) return hkv::kPrefillNoRows;
  return found & 2 ? hkv::kPrefillRefused : hkv::kPrefillRuns;
}

// The verdict on each sequence and its chunks, one workgroup each.
__device__ __forceinline__ void plan(const hkv::PrefillArgs& a) {
  __shared__ uint32_t found, before;
  const uint32_t s = blockIdx.x, t = threadIdx.x;
  if (t == 0) found = before = 0;
  __syncthreads();
  const Span me = span_of(a, s);
  const int32_t* own = a.table + (int64_t)s * a.table_stride;
  const uint32_t mine_found = look_through(a, s, me, t, kPlanThreads);
  if (mine_found) atomicOr(&found, mine_found);
  uint32_t mine = 0;  // chunks of the sequences before
  if (a.chunked)
    for (uint32_t r = t; r < s; r += kPlanThreads) mine += chunks_of(a, span_of(a, r));
  if (mine) atomicAdd(&before, mine);
  __syncthreads();
  const int32_t status = verdict(me, found);
  const bool rows = status != hkv::kPrefillNoRows;
  if (t == 0) a.status[s] = status;
  if (!a.chunked) return;
  // Starts that go backwards can give more chunks than the workspace has records
  // for: the first sequence that does not fit leaves its part of them empty.
  const uint32_t all = chunks_of(a, me);
  const uint32_t first = min(before, a.max_chunks), room = a.max_chunks - first;
  const uint32_t count = all <= room ? all : 0;
  if (t == 0) {
    if (all > room && rows) a.status[s] = hkv::kPrefillNoRows;
    a.first_chunk[s] = (int32_t)first;
    a.first_chunk[s + a.n_seqs] = (int32_t)count;
    if (s == a.n_seqs - 1) a.first_chunk[2 * a.n_seqs] = (int32_t)(first + count);
  }
  if (all > room)
    for (uint32_t c = first + t; c < a.max_chunks; c += kPlanThreads)
      a.chunks[c] = hkv::PrefillChunk{};
  // A chunk of a sequence that does not run is empty.
  const bool runs = status == hkv::kPrefillRuns;
  const uint32_t lead = chunk_lead(a, me), lead_chunks = (lead + kC - 1) / kC;
  const uint32_t per = (a.block_tokens + kC - 1) / kC;
  for (uint32_t c = t; c < count; c += kPlanThreads) {
    uint32_t off = c * kC, end = lead;
    if (c >= lead_chunks) {
      const uint32_t k = c - lead_chunks;
      end = lead + (k / per + 1) * a.block_tokens;
      off = lead + k / per * a.block_tokens + k % per * kC;
    }
    end = min(end, (uint32_t)me.tokens);
    hkv::PrefillChunk ck;
    ck.seq = (int32_t)s;
    ck.row = me.row + (int32_t)off;
    ck.len = runs ? (int32_t)min(kC, end - off) : 0;
    ck.off = (int32_t)off;
    ck.dst = HKV_NULL_BLOCK;
    if (runs && off + kC >= end) ck.dst = own[(uint32_t)(me.position + (int32_t)off) / a.block_tokens];
    a.chunks[first + c] = ck;
  }
}

// ---------------------------------------------------------------- lanes
__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float real(uint32_t x) { return __builtin_bit_cast(float, x); }

template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return real((uint32_t)__builtin_amdgcn_update_dpp(0, (int)bits(x), kCtrl, 0xf, 0xf, true));
}

// Sums over lanes that differ in bits 4 and 5.
__device__ __forceinline__ float sum_rows(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  x = real(r0) + real(r1);
  const auto q = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
  const uint32_t q0 = q[0], q1 = q[1];
  return real(q0) + real(q1);
}
// Over those that differ in bits 2 to 5.
__device__ __forceinline__ float sum_fours(float x) {
  x += dpp<0x128>(x);  // row_ror:8
  x += dpp<0x124>(x);  // row_ror:4
  return sum_rows(x);
}
// Over all.
__device__ __forceinline__ float sum_wave(float x) {
  x += dpp<0xb1>(x);  // quad_perm [1,0,3,2]
  x += dpp<0x4e>(x);  // quad_perm [2,3,0,1]
  return sum_fours(x);
}

// 1 / sqrt(x).  The instruction takes numbers below 2^-126, where sums of squares without
// an eps may lie, for 0.
__device__ __forceinline__ float inverse_root(float x) {
  const bool tiny = x < 0x1p-126f;
  return __builtin_amdgcn_rsqf(tiny ? x * 0x1p64f : x) * (tiny ? 0x1p32f : 1.0f);
}

// ---------------------------------------------------------------- token by token
// hkv_kda_step's recurrence with the state and the conv's taps kept in registers
// from token to token, and the hardware's exp2, rcp and rsq where the step has expf, a
// division and sqrtf, since they lie on a token's chain (x log2 e is rounded to fp32: a
// decay of e^-x is off by up to 6e-8 (1 + x) of itself).  One workgroup per (head,
// sequence), a wave for 16 columns.  Thread t has 4 columns of kDim / 16 rows, so that the
// sums over rows stay within a wave, and one channel of the conv or of the decays; the only thing that the waves
// exchange is a token's q, k, v and decays: one barrier a token (61 runs of up to
// 5 tokens, 6 heads: 20 us; the form before, without this split, 28).  Heads of 256 have
// 1024 threads and so 128 registers, of which 20 (bf16, fp16) or 22 (fp32) are spilled.
template <class T, uint32_t kDim>
__device__ __forceinline__ void tokens(const hkv::PrefillArgs& a) {
  using E = typename T::type;
  constexpr uint32_t kThreads = kDim * 4, kWaves = kThreads / 64, kRows = kDim / 16;
  // two of each, by the token's parity: the next token's are written while slower
  // waves still read this one's
  __shared__ __attribute__((aligned(16))) float y[2][4][kDim];  // q, k, v after the conv; decays
  __shared__ uint32_t found[kWaves];
  const uint32_t h = blockIdx.x, s = blockIdx.y, t = threadIdx.x, lane = t & 63;
  const uint32_t col = (t >> 6) * 16 + (lane & 3) * 4, r0 = (lane >> 2) * kRows;
  const int32_t row0 = a.starts[s];
  const int32_t n = a.starts[s + 1] - row0;
  if (a.chunked && n > (int32_t)a.short_tokens) return;
  E* const out = static_cast<E*>(a.out) + (int64_t)row0 * a.out_stride + (int64_t)h * kDim + col;
  const int32_t position = a.positions[s];
  int32_t src = a.src[s];
  if (outside(src, a.num_blocks)) src = HKV_NULL_BLOCK;  // until the verdict below
  const int32_t* const table = a.table + (int64_t)s * a.table_stride;
  const uint64_t state_off =
      a.conv_bytes + (((uint64_t)h * kDim + r0) * kDim + col) * 4;

  v4f st[kRows];
  {
    const HKV_GLOBAL uint8_t* p =
        (const HKV_GLOBAL uint8_t*)(a.pages + (uint64_t)(src < 0 ? 0 : src) * a.stride + state_off);
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      st[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (src >= 0) st[i] = *(const HKV_GLOBAL v4f*)(p + i * kDim * 4);
    }
  }
  // The verdict on the sequence, while its state is under way.
  int32_t status;
  if (a.planned) {
    status = a.status[s];
  } else {
    const Span me = span_of(a, s);
    const uint32_t mine = look_through(a, s, me, t, kThreads);
    const uint32_t all = (__any(mine & 1) ? 1u : 0u) | (__any(mine & 2) ? 2u : 0u);
    if (lane == 0) found[t >> 6] = all;
    __syncthreads();
    uint32_t any = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) any |= found[w];
    status = verdict(me, any);
  }
  if (status == hkv::kPrefillNoRows) return;
  if (status == hkv::kPrefillRefused) {
    for (uint32_t i = lane >> 2; i < (uint32_t)n; i += 16)
      T::store4(out + (int64_t)i * a.out_stride, v4f{NAN, NAN, NAN, NAN});
    return;
  }
  // Threads below 3 kDim: a channel's weights, its last `keep` values (oldest first).
  // The others: a channel's decay.
  const uint32_t keep = a.taps - 1, part = t / kDim, in_part = t % kDim;
  const uint64_t ch = ((uint64_t)part * a.heads + h) * kDim + in_part;
  E taps[hkv::kKdaMaxKernel - 1];
  float weight[hkv::kKdaMaxKernel];
  if (part < 3) {
    const E* wt = static_cast<const E*>(a.conv_weight) + ch * a.taps;
    const E* old = reinterpret_cast<const E*>(a.pages + (uint64_t)(src < 0 ? 0 : src) * a.stride) +
                   ch * keep;
#pragma unroll
    for (uint32_t j = 0; j < hkv::kKdaMaxKernel; ++j) weight[j] = j <= keep ? (float)wt[j] : 0.0f;
#pragma unroll
    for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
      taps[j] = j < keep && src >= 0 ? old[j] : (E)0.0f;
  }

  // A token's inputs are fetched while the one before is computed.
  E x_next = (E)0.0f;
  float g_next = 0.0f, beta_next;
  auto fetch = [&](int32_t m) {
    const int64_t row = (int64_t)row0 + m;
    if (part < 3)
      x_next = static_cast<const E*>(a.x)[row * a.x_stride + (int64_t)ch];
    else
      g_next = a.log_decay[row * a.decay_stride + (int64_t)h * kDim + in_part];
    beta_next = a.beta[row * a.beta_stride + h];
  };
  fetch(0);
  for (int32_t m = 0; m < n; ++m) {
    const uint32_t b = m & 1;
    if (part < 3) {
      const E x = x_next;
      float sum = 0.0f;
      if (keep == 3) {
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j) sum += weight[j] * (float)taps[j];
        sum += weight[3] * (float)x;
        taps[0] = taps[1];
        taps[1] = taps[2];
        taps[2] = x;
      } else {
#pragma unroll
        for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
          if (j < keep) sum += weight[j] * (float)taps[j];
#pragma unroll
        for (uint32_t j = 0; j < hkv::kKdaMaxKernel; ++j)
          if (j == keep) sum += weight[j] * (float)x;
#pragma unroll
        for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j) {
          if (j + 1 < keep) taps[j] = taps[j + 1 < hkv::kKdaMaxKernel - 1 ? j + 1 : j];
          if (j + 1 == keep) taps[j] = x;
        }
      }
      y[b][part][in_part] =
          sum * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(sum * -1.44269504f));
    } else {
      y[b][3][in_part] = __builtin_amdgcn_exp2f((g_next > 0.0f ? 0.0f : g_next) * 1.44269504f);
    }
    const float beta = beta_next;
    if (m + 1 < n) fetch(m + 1);
    __syncthreads();

    // |q|^2, |k|^2 and q.k, by every wave for itself.
    float qq = 0.0f, kk = 0.0f, qk = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < (kDim + 63) / 64; ++i)
      if (kDim >= 64 || lane < kDim) {
        const float q = y[b][0][lane + i * 64], k = y[b][1][lane + i * 64];
        qq += q * q;
        kk += k * k;
        qk += q * k;
      }
    qq = sum_wave(qq);
    kk = sum_wave(kk);
    qk = sum_wave(qk);
    const float nq = a.scale * inverse_root(qq + a.eps);
    const float nk = inverse_root(kk + a.eps);

    float k[kRows];
    v4f sk = {0.0f, 0.0f, 0.0f, 0.0f}, sq = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      k[i] = y[b][1][r0 + i] * nk;
      st[i] *= y[b][3][r0 + i];
      sk += st[i] * k[i];
      sq += st[i] * (y[b][0][r0 + i] * nq);
    }
    const v4f v = *reinterpret_cast<const v4f*>(&y[b][2][col]);
    v4f u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = beta * (v[i] - sum_fours(sk[i]));
      sq[i] = sum_fours(sq[i]) + u[i] * (qk * nq * nk);
    }
    if (lane < 4) T::store4(out + (int64_t)m * a.out_stride, sq);
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) st[i] += u * k[i];

    const uint32_t at = (uint32_t)(position + m);
    if (m != n - 1 && (at + 1) % a.block_tokens != 0) continue;
    const int32_t dst = table[at / a.block_tokens];
    if (dst < 0) continue;
    HKV_GLOBAL uint8_t* p =
        (HKV_GLOBAL uint8_t*)(a.pages + (uint64_t)dst * a.stride + state_off);
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) *(HKV_GLOBAL v4f*)(p + i * kDim * 4) = st[i];
    if (part < 3) {
      E* to = reinterpret_cast<E*>(a.pages + (uint64_t)dst * a.stride) + ch * keep;
#pragma unroll
      for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
        if (j < keep) to[j] = taps[j];
    }
  }
}

// ---------------------------------------------------------------- chunks
// A chunk is up to 64 tokens of one sequence that end no later than their block.
// With a_t the token's decays, R_t = a_1 .. a_t and D_ts = a_{s+1} .. a_t (products
// per channel, all <= 1):
//   A_ts = beta_t sum_c k_tc k_sc D_tsc (s < t),  P_ts = sum_c q_tc k_sc D_tsc (s <= t)
//   T = (1 + A)^-1 diag(beta),  W = T (k R),  U0 = T V
// do not depend on the state, so `form` computes them for all chunks and heads at
// once; `scan` then goes through a sequence's chunks in order:
//   U = U0 - W S,  O = (q R) S + P U,  S <- diag(R_64) S + (k D_64)^T U.
// Decays are multiplied up, never divided: where t lies in the later half of 16, 32 or
// 64 tokens and s in the earlier, D_ts is (decays since the later half's start) x (decays
// up to it), both <= 1, so that no factor overflows; within 8 tokens the pairs are
// summed one by one in fp32.  Products of matrices run in fp16 with each operand as two terms, hi +
// lo (22 bits), and three products (lo lo is below 2^-22); what is scaled by a
// power of two to lie well inside fp16's range says so.  V's and S's columns never
// mix, so each has a power of two of its own.  (Two bf16 terms would have
// 16 bits.)  The low term is a multiple of 2^-24 like all of fp16, so what is far below its
// scale has fewer bits: 2^-25 of 16 k in K, say, is 2^-29 of the longest key, far below
// the column's own rounding, but all that a channel of 1e-6 of a key has for its row.
//
// `form`: one workgroup of eight waves a chunk and head, a wave 8 tokens, a lane two
// channels.  With 20011 tokens of 32 heads a wave has 2290 vector instructions and waits 36%
// of its cycles, LDS is active in 37% of a CU's (37% of that are conflicts), the matrix
// units in 11%.  Four waves of 16 tokens, with the halves of 16 tokens pair by pair, took
// 569 us there where this split first took 554.  Two workgroups a CU: 80 KB of LDS, 128 registers.
constexpr uint32_t kD = hkv::kPrefillChunkDim;
constexpr uint32_t kFormThreads = 512;
constexpr float kUnit = 64.0f;  // scale of k and q operands (each at most 1 in size)

typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef int32_t v2i __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// x = hi + lo, to 2^-22 of x.
struct Terms2 {
  v2h hi, lo;
};
__device__ __forceinline__ Terms2 terms(float x, float y) {
  // one v_fma_mix a remainder: the compiler makes two instructions of a difference
  float minus = -1.0f;
  __asm__("" : "+s"(minus));
  Terms2 t;
  t.hi = __builtin_convertvector(v2f{x, y}, v2h);
  t.lo = __builtin_convertvector(v2f{__builtin_fmaf((float)t.hi[0], minus, x),
                                     __builtin_fmaf((float)t.hi[1], minus, y)}, v2h);
  return t;
}
struct Terms8 {
  v8h hi, lo;
};
__device__ __forceinline__ Terms8 terms(v4f x, v4f y) {
  const Terms2 a = terms(x[0], x[1]), b = terms(x[2], x[3]);
  const Terms2 c = terms(y[0], y[1]), d = terms(y[2], y[3]);
  Terms8 t;
  t.hi = v8h{a.hi[0], a.hi[1], b.hi[0], b.hi[1], c.hi[0], c.hi[1], d.hi[0], d.hi[1]};
  t.lo = v8h{a.lo[0], a.lo[1], b.lo[0], b.lo[1], c.lo[0], c.lo[1], d.lo[0], d.lo[1]};
  return t;
}

__device__ __forceinline__ v4f mfma(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void mfma3(const Terms8& a, const Terms8& b, v4f (&c)[3]) {
  c[0] = mfma(a.lo, b.hi, c[0]);
  c[1] = mfma(a.hi, b.lo, c[1]);
  c[2] = mfma(a.hi, b.hi, c[2]);
}

// Sums 16 values over the wave: lane l gets the sum of value l / 4.
__device__ __forceinline__ float sum16(const float (&v)[16], uint32_t lane) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(bits(v[i]), bits(v[i + 8]), false, false);
    const uint32_t x = r[0], y = r[1];
    a[i] = real(x) + real(y);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(bits(a[i]), bits(a[i + 4]), false, false);
    const uint32_t x = r[0], y = r[1];
    b[i] = real(x) + real(y);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    c[i] = (up ? b[i + 2] : b[i]) + dpp<0x128>(up ? b[i] : b[i + 2]);  // row_ror:8
  }
  const bool up = lane & 4;
  float r = (up ? c[1] : c[0]) + dpp<0x141>(up ? c[0] : c[1]);  // row_half_mirror
  r += dpp<0x4e>(r);                                            // quad_perm [2,3,0,1]
  return r + dpp<0xb1>(r);                                      // quad_perm [1,0,3,2]
}

// The wave's place in its workgroup, as a scalar.
__device__ __forceinline__ uint32_t wave_index() {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// Orders a wave's own LDS accesses (its instructions run in order).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// LDS of `form`, bytes.  Planes: rows of 128 channels (`row`) or of 64 tokens.
constexpr uint32_t kRowPlane = 16 * (kD * 2 + 16);   // 16 tokens
constexpr uint32_t kRowStride = kD * 2 + 16;
constexpr uint32_t kTokStride = kC * 2 + 16;
constexpr uint32_t kTokPlane = kD * kTokStride;      // 128 channels x 64 tokens
constexpr uint32_t kTPlane = kC * kTokStride;        // T: 64 x 64
constexpr uint32_t kMStride = 68;                    // floats
constexpr uint32_t kTmpStride = 36;
constexpr uint32_t kOffM = 2 * kTPlane + 2 * kTokPlane;
constexpr uint32_t kOffTmp = kOffM + kC * kMStride * 4;
constexpr uint32_t kOffBeta = kOffTmp + 32 * kTmpStride * 4;
constexpr uint32_t kOffTotal = kOffBeta + kC * 4;
constexpr uint32_t kFormLds = kOffTotal + 8 * kD * 4;
static_assert(12 * kRowPlane <= kOffM && kFormLds <= 80 * 1024, "two workgroups of `form` fit a CU");

// One chunk's result in the workspace, as the scan's lanes load it (1 KiB for 64
// lanes of 16 bytes; lane l: row or column l % 16, group g = l / 16).
//   W, Q   [token tile][32 channels][hi, lo]: 8 channels 4 g + 0..3 and 16 + 4 g + 0..3,
//          where a 16x16 product leaves two tiles of the state
//   K      [channel tile][32 tokens][hi, lo]: 8 tokens 8 g + 0..7
//   P      [tile of 16 x 32 tokens][hi, lo]: the same
//   U0     [channel tile][token tile]: 4 tokens 4 g + 0..3, fp32
//   decay  [channel], fp32
//   exps   [channel]: V's largest value is below 2^exps; -1000: V is zero
constexpr uint32_t kRecW = 0;
constexpr uint32_t kRecQ = kRecW + 4 * (kD / 32) * 2048;
constexpr uint32_t kRecK = kRecQ + 4 * (kD / 32) * 2048;
constexpr uint32_t kRecP = kRecK + (kD / 16) * 2 * 2048;
constexpr uint32_t kRecU = kRecP + 6 * 2048;
constexpr uint32_t kRecDecay = kRecU + (kD / 16) * 4 * 1024;
constexpr uint32_t kRecExps = kRecDecay + kD * 4;
static_assert(kRecExps + kD * 4 == hkv::kPrefillRecord, "the workspace holds a record");

// Two channels of one row, aligned as one.
typedef uint32_t pair16 __attribute__((aligned(2)));
typedef float pair32 __attribute__((ext_vector_type(2), aligned(4)));

template <class E>
__device__ __forceinline__ v2f widen(uint32_t x) {
  typedef E pair __attribute__((ext_vector_type(2)));
  return __builtin_convertvector(__builtin_bit_cast(pair, x), v2f);
}

__device__ __forceinline__ v8h join(v4h a, v4h b) {
  return v8h{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// A chunk as scalars, through the constant address space: a vector load would have to
// wait for the operands that are under way.
__device__ __forceinline__ hkv::PrefillChunk read_chunk(const hkv::PrefillArgs& a, uint32_t slot) {
  typedef __attribute__((address_space(4))) const int32_t word;
  word* const p = (word*)(uintptr_t)(a.chunks + slot);
  hkv::PrefillChunk ck;
  ck.seq = p[0];
  ck.row = p[1];
  ck.len = p[2];
  ck.off = p[3];
  ck.dst = p[4];
  return ck;
}

template <class T>
__device__ __forceinline__ void form(const hkv::PrefillArgs& a, uint32_t slot, uint32_t h,
                                     uint8_t* lds) {
  using E = typename T::type;
  const uint32_t t = threadIdx.x, w = wave_index(), lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const hkv::PrefillChunk ck = read_chunk(a, slot);
  const int32_t len = ck.len;
  const int32_t src = a.src[ck.seq];
  uint8_t* const rec = a.records + ((uint64_t)slot * a.heads + h) * hkv::kPrefillRecord;
  float* const M = reinterpret_cast<float*>(lds + kOffM);
  float* const tmp = reinterpret_cast<float*>(lds + kOffTmp);
  float* const beta = reinterpret_cast<float*>(lds + kOffBeta);
  float* const total = reinterpret_cast<float*>(lds + kOffTotal);
  const int32_t t0 = (int32_t)w * 8;   // the wave's first token of the chunk
  const uint32_t ch = lane * 2;        // the lane's channels: ch, ch + 1

  // Loads: the wave's 8 tokens and the three before them; tokens behind the chunk's
  // last read the last one's row and are blanked below.
  uint32_t raw[3][11];
  float g0[8], g1[8];
#pragma unroll
  for (int r = 0; r < 11; ++r) {
    const int32_t o = min(t0 + r - 3, len - 1);
    const int64_t row = (int64_t)ck.row + (ck.off + o < 0 ? 0 : o);
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride + (uint64_t)h * kD;
#pragma unroll
    for (int p = 0; p < 3; ++p)
      raw[p][r] = *(const HKV_GLOBAL pair16*)((const HKV_GLOBAL uint8_t*)(x + (uint64_t)p * a.heads * kD) + lane * 4);
    if (r >= 3) {
      const v2f g = *(const HKV_GLOBAL pair32*)(
          (const HKV_GLOBAL uint8_t*)(a.log_decay + row * a.decay_stride + (uint64_t)h * kD) + lane * 8);
      g0[r - 3] = g[0];
      g1[r - 3] = g[1];
    }
  }
  float b_t = 0.0f;  // lane i: token i's beta
  if (t0 + (int32_t)(lane & 7) < len)
    b_t = a.beta[((int64_t)ck.row + t0 + (lane & 7)) * a.beta_stride + h];
  if (ck.off + t0 < 3) {  // taps from before the sequence's first row
#pragma unroll
    for (int r = 0; r < 3; ++r) {
      const int32_t o = ck.off + t0 + r - 3;
      if (o >= 0) continue;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint32_t v = 0;
        if (src >= 0) {
          const uint16_t* old = reinterpret_cast<const uint16_t*>(
              a.pages + (uint64_t)src * a.stride) +
              (((uint64_t)p * a.heads + h) * kD + ch) * 3 + (3 + o);
          v = (uint32_t)old[0] | ((uint32_t)old[3] << 16);
        }
        raw[p][r] = v;
      }
    }
  }

  // y = silu(conv), two channels of 8 tokens a lane.
  v2f y[3][8];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const E* wt = static_cast<const E*>(a.conv_weight) +
                  (((uint64_t)p * a.heads + h) * kD + ch) * 4;
    v2f w4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w4[j] = v2f{(float)wt[j], (float)wt[j + 4]};
    v2f x[11];
#pragma unroll
    for (int r = 0; r < 11; ++r) x[r] = widen<E>(raw[p][r]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v2f s = w4[0] * x[i];
#pragma unroll
      for (int j = 1; j < 4; ++j) s += w4[j] * x[i + j];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float e = __builtin_amdgcn_exp2f(s[c] * -1.44269504f);
        y[p][i][c] = s[c] * __builtin_amdgcn_rcpf(1.0f + e);
      }
    }
  }
  v2f av[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = g0[i] > 0.0f ? 0.0f : g0[i], x1 = g1[i] > 0.0f ? 0.0f : g1[i];
    av[i] = v2f{__builtin_amdgcn_exp2f(x0 * 1.44269504f), __builtin_amdgcn_exp2f(x1 * 1.44269504f)};
  }
  if (t0 + 8 > len) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i >= len) {
        y[0][i] = y[1][i] = y[2][i] = v2f{0.0f, 0.0f};
        av[i] = v2f{1.0f, 1.0f};
      }
  }

  // q and k over their norms (16 sums at once, each lane's root goes to all), times
  // kUnit.  Blanked tokens get a factor of 0: without an eps theirs would be infinite.
  {
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = y[0][i][0] * y[0][i][0] + y[0][i][1] * y[0][i][1];
      v[8 + i] = y[1][i][0] * y[1][i][0] + y[1][i][1] * y[1][i][1];
    }
    const float sum = sum16(v, lane);  // of token lane / 4 % 8
    const float by = t0 + (int32_t)(lane >> 2 & 7) < len ? kUnit / sqrtf(sum + a.eps) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float nq = real((uint32_t)__builtin_amdgcn_readlane((int)bits(by), 4 * i));
      const float nk = real((uint32_t)__builtin_amdgcn_readlane((int)bits(by), 32 + 4 * i));
      y[0][i] *= nq;
      y[1][i] *= nk;
    }
  }
  constexpr float kUnits = 1.0f / (kUnit * kUnit);

  // Pairs within the wave's 8 tokens.  Columns s = b and 7 - b together give 16 sums;
  // lane 4 n gets sum n.  M holds A (without beta) below its diagonal and P's transpose
  // above: P_ts at [s][t + 1].
  {
    const uint32_t n = lane >> 2, m = n & 7;
    float* const block = M + t0 * kMStride + t0;
    float* const waste = tmp + w * 8;
    float sums[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float v[16];
      v2f p = y[1][b];
      v[b] = y[0][b][0] * p[0] + y[0][b][1] * p[1];
#pragma unroll
      for (int i = b + 1; i < 8; ++i) {
        p *= av[i];
        v[i] = y[1][i][0] * p[0] + y[1][i][1] * p[1];
        v[8 + i] = y[0][i][0] * p[0] + y[0][i][1] * p[1];
      }
      p = y[1][7 - b];
#pragma unroll
      for (int k = 0; k <= b; ++k) {
        const int i = 7 - b + k;
        if (k > 0) {
          p *= av[i];
          v[k - 1] = y[1][i][0] * p[0] + y[1][i][1] * p[1];
        }
        v[8 + k] = y[0][i][0] * p[0] + y[0][i][1] * p[1];
      }
      sums[b] = sum16(v, lane) * kUnits;
      // n < b: A(8 - b + n, 7 - b); n = b: P(b, b); b < n < 8: A(n, b);
      // 8 <= n <= 8 + b: P(7 - b + m, 7 - b); n > 8 + b: P(m, b).  Lanes with A write to
      // where nobody reads.
      const uint32_t to = n >= 8 && m <= (uint32_t)b ? (7 - b) * (kMStride + 1) : b * kMStride;
      (n >= 8 || m == (uint32_t)b ? block : waste)[to + m + 1] = sums[b];
    }
    // (1 + A)^-1: lane j solves for column j, with A's values as scalars from the lanes
    // that have them.
    float acc[8], x[8];  // acc: sum_s A(i, s) x_s
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float b_s = real((uint32_t)__builtin_amdgcn_readlane((int)bits(b_t), s));
      x[s] = (lane == (uint32_t)s ? 1.0f : 0.0f) - b_s * acc[s];
#pragma unroll
      for (int i = s + 1; i < 8; ++i) {
        // A(i, s): in sums[s] at i for s < 4, in sums[7 - s] at i - s - 1 otherwise
        const int from = s < 4 ? i : i - s - 1;
        const float as = real(
            (uint32_t)__builtin_amdgcn_readlane((int)bits(sums[s < 4 ? s : 7 - s]), 4 * from));
        acc[i] += as * x[s];
      }
    }
    if (lane < 8) {
      beta[t0 + lane] = b_t;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= (int)lane) block[i * kMStride + lane] = x[i];
    }
  }

  // Decays of the 8 tokens: up to a token with it go to k and q, behind it to k.
  v2f kr[8], kd[8], qr[8];
  {
    v2f r = av[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > 0) r *= av[i];
      kr[i] = y[1][i] * r;
      qr[i] = y[0][i] * r;
    }
    *reinterpret_cast<v2f*>(total + w * kD + ch) = r;
    r = v2f{1.0f, 1.0f};
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      kd[i] = y[1][i] * r;
      r *= av[i];
    }
  }

  // A row plane holds 16 tokens' channels of one term; a wave has half of its rows.
  auto put_row = [&](uint32_t at, uint32_t lo, const v2f (&x)[8], v2f by) {
    uint8_t* const to = lds + at + ch * 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const v2f z = x[i] * by;
      const Terms2 s = terms(z[0], z[1]);
      *reinterpret_cast<v2h*>(to + i * kRowStride) = s.hi;
      *reinterpret_cast<v2h*>(to + lo + i * kRowStride) = s.lo;
    }
  };
  auto get_row = [&](uint32_t at, uint32_t lo, uint32_t row, uint32_t kb) {
    const uint8_t* const from = lds + at + row * kRowStride + kb * 64 + lg * 16;
    Terms8 s;
    s.hi = *reinterpret_cast<const v8h*>(from);
    s.lo = *reinterpret_cast<const v8h*>(from + lo);
    return s;
  };
  const v2f one = {1.0f, 1.0f};
  const uint32_t tile = w >> 1, late = w & 1;  // of the chunk's four tiles of 16 tokens
  constexpr uint32_t kHalf = kRowPlane / 2;
  // A 16x16 tile of A or of P's transpose goes to M.
  auto put_m = [&](bool is_p, uint32_t row_tile, uint32_t col_tile, v4f x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t row = row_tile * 16 + lg * 4 + j, col = col_tile * 16 + lr;
      M[is_p ? col * kMStride + row + 1 : row * kMStride + col] = x[j] * kUnits;
    }
  };

  // Halves of 16 tokens: a tile's plane of k has the earlier half's columns in rows 0..7
  // and the later's in 8..15, which meet at the later half's start: its product with
  // itself has A in one quarter.  Behind the four planes' terms those of the later
  // halves' q.
  constexpr uint32_t kQ8 = 8 * kRowPlane;
  if (late) {
    put_row(tile * 2 * kRowPlane + kHalf, kRowPlane, kr, one);
    put_row(kQ8 + tile * kRowPlane, kHalf, qr, one);
  } else {
    put_row(tile * 2 * kRowPlane, kRowPlane, kd, one);
  }
  __syncthreads();
  {
    v4f acc[3] = {};  // by term: a sum waits for the one before
#pragma unroll
    for (uint32_t kb = 0; kb < kD / 32; ++kb) {
      const Terms8 k = get_row(tile * 2 * kRowPlane, kRowPlane, lr, kb);
      if (late)
        mfma3(get_row(kQ8 + tile * kRowPlane, kHalf, lr & 7, kb), k, acc);
      else
        mfma3(k, k, acc);
    }
    const v4f z = acc[0] + acc[1] + acc[2];
    if (lg >= 2 && lr < 8) put_m(late, tile, tile, z);
    // T_10 = -T_11 (beta A_10 T_00), in fp32.
    if (!late) {
      wave_fence();
      const uint32_t r0 = tile * 16 + 8, c0 = tile * 16;
      float* const x = tmp + tile * 8 * kTmpStride;
      v4f y2 = {};
#pragma unroll
      for (uint32_t kk = 0; kk < 2; ++kk) {
        const uint32_t k = kk * 4 + lg;
        const float p = lr < 8 ? M[(r0 + lr) * kMStride + c0 + k] : 0.0f;
        const float q = lr < 8 && k >= lr ? M[(c0 + k) * kMStride + c0 + lr] : 0.0f;
        y2 = __builtin_amdgcn_mfma_f32_16x16x4f32(p, q, y2, 0, 0, 0);
      }
      if (lg < 2 && lr < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[(lg * 4 + j) * kTmpStride + lr] = y2[j] * beta[r0 + lg * 4 + j];
      wave_fence();
      y2 = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t kk = 0; kk < 2; ++kk) {
        const uint32_t k = kk * 4 + lg;
        const float p = lr < 8 && k <= lr ? M[(r0 + lr) * kMStride + r0 + k] : 0.0f;
        const float q = lr < 8 ? x[k * kTmpStride + lr] : 0.0f;
        y2 = __builtin_amdgcn_mfma_f32_16x16x4f32(p, q, y2, 0, 0, 0);
      }
      if (lg < 2 && lr < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) M[(r0 + lg * 4 + j) * kMStride + c0 + lr] = -y2[j];
    }
  }
  // The products of the other blocks' decays between a token's block and where it is
  // met: by halves of 16, 32 and 64 tokens, from the chunk's start, to its end.
  v2f by32, by64, before;
  {
    auto of = [&](uint32_t b) { return *reinterpret_cast<const v2f*>(total + b * kD + ch); };
    v2f left = one, right = one;  // of the tiles before and behind the wave's
    v2f near = one;               // of the half's other tile, where it lies between
#pragma unroll
    for (uint32_t b = 0; b < 4; ++b) {
      const v2f x = of(2 * b) * of(2 * b + 1);
      if (b < tile) left *= x;
      if (b > tile) right *= x;
      if ((tile == 3 && b == 2) || (tile == 0 && b == 1)) near = x;
    }
    const v2f up = late ? of(w - 1) : one, down = late ? one : of(w + 1);
    by32 = tile & 1 ? up : down;
    by64 = (w >= 4 ? up : down) * near;
    before = up * left;
    const v2f after = down * right;
    if (w == 0) *reinterpret_cast<v2f*>(rec + kRecDecay + ch * 4) = after * of(0);
    // k D_64 (16 times itself): a lane has 8 tokens of its two channels, as the scan
    // takes them.
    const v2f by = after * v2f{16.0f / kUnit, 16.0f / kUnit};
    uint8_t* const to = rec + kRecK + (lane >> 3) * 4096 + (w >> 2) * 2048 + (w & 3) * 256;
#pragma unroll
    for (uint32_t c = 0; c < 2; ++c) {
      v4f z[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i >> 2][i & 3] = kd[i][c] * by[c];
      const Terms8 x = terms(z[0], z[1]);
      *reinterpret_cast<v8h*>(to + ((ch + c) & 15) * 16) = x.hi;
      *reinterpret_cast<v8h*>(to + ((ch + c) & 15) * 16 + 1024) = x.lo;
    }
  }
  __syncthreads();

  // Halves of 32: tiles 1 x 0 and 3 x 2.
  {
    const uint32_t at = (w >> 2) * 6 * kRowPlane + late * kHalf;
    if (tile & 1) {
      put_row(at + 2 * kRowPlane, kRowPlane, kr, by32);
      put_row(at + 4 * kRowPlane, kRowPlane, qr, by32);
    } else {
      put_row(at, kRowPlane, kd, by32);
    }
  }
  __syncthreads();
  if (w < 4) {
    const uint32_t pair = w & 1, is_p = w >> 1;
    v4f acc[3] = {};
#pragma unroll
    for (uint32_t kb = 0; kb < kD / 32; ++kb)
      mfma3(get_row((pair * 6 + 2 + 2 * is_p) * kRowPlane, kRowPlane, lr, kb),
            get_row(pair * 6 * kRowPlane, kRowPlane, lr, kb), acc);
    put_m(is_p, 2 * pair + 1, 2 * pair, acc[0] + acc[1] + acc[2]);
    if (!is_p) {
      wave_fence();
      const uint32_t r0 = pair * 32 + 16, c0 = pair * 32;
      float* const x = tmp + pair * 16 * kTmpStride;
      v4f y2[2] = {};
#pragma unroll
      for (uint32_t kk = 0; kk < 4; ++kk) {
        const uint32_t k = kk * 4 + lg;
        const float p = M[(r0 + lr) * kMStride + c0 + k];
        const float q = k >= lr ? M[(c0 + k) * kMStride + c0 + lr] : 0.0f;
        y2[kk & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(p, q, y2[kk & 1], 0, 0, 0);
      }
      v4f z = y2[0] + y2[1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[(lg * 4 + j) * kTmpStride + lr] = z[j] * beta[r0 + lg * 4 + j];
      wave_fence();
      y2[0] = y2[1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t kk = 0; kk < 4; ++kk) {
        const uint32_t k = kk * 4 + lg;
        const float p = k <= lr ? M[(r0 + lr) * kMStride + r0 + k] : 0.0f;
        y2[kk & 1] =
            __builtin_amdgcn_mfma_f32_16x16x4f32(p, x[k * kTmpStride + lr], y2[kk & 1], 0, 0, 0);
      }
      z = y2[0] + y2[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) M[(r0 + lg * 4 + j) * kMStride + c0 + lr] = -z[j];
    }
  }
  __syncthreads();

  // Halves of 64.  Planes 0..3 hold the columns' tiles, 4..11 the rows'.
  if (w >= 4) {
    const uint32_t at = (4 + (tile - 2) * 4) * kRowPlane + late * kHalf;
    put_row(at, kRowPlane, kr, by64);
    put_row(at + 2 * kRowPlane, kRowPlane, qr, by64);
  } else {
    put_row(tile * 2 * kRowPlane + late * kHalf, kRowPlane, kd, by64);
  }
  __syncthreads();
  {
    const uint32_t is_p = w >> 2, i = (w >> 1) & 1, j = w & 1;
    v4f acc[3] = {};
#pragma unroll
    for (uint32_t kb = 0; kb < kD / 32; ++kb)
      mfma3(get_row((4 + i * 4 + is_p * 2) * kRowPlane, kRowPlane, lr, kb),
            get_row(j * 2 * kRowPlane, kRowPlane, lr, kb), acc);
    put_m(is_p, 2 + i, j, acc[0] + acc[1] + acc[2]);
  }
  __syncthreads();

  // T_10 of the halves, in fp32; meanwhile q R (256 times itself) goes out.
  put_row(tile * 2 * kRowPlane + late * kHalf, kRowPlane, qr, before * v2f{256.0f / kUnit, 256.0f / kUnit});
  if (w < 4) {
    const uint32_t i = w >> 1, j = w & 1;
    v4f y2[2] = {};
#pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) {
      const uint32_t k = kk * 4 + lg, col = j * 16 + lr;
      const float p = M[(32 + i * 16 + lr) * kMStride + k];
      const float q = k >= col ? M[k * kMStride + col] : 0.0f;
      y2[kk & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(p, q, y2[kk & 1], 0, 0, 0);
    }
    const v4f z = y2[0] + y2[1];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const uint32_t row = i * 16 + lg * 4 + n;
      tmp[row * kTmpStride + j * 16 + lr] = z[n] * beta[32 + row];
    }
  }
  __syncthreads();
  if (w < 4) {
    const uint32_t i = w >> 1, j = w & 1;
    v4f y2[2] = {};
#pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) {
      const uint32_t k = kk * 4 + lg, row = i * 16 + lr;
      const float p = k <= row ? M[(32 + row) * kMStride + 32 + k] : 0.0f;
      y2[kk & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(p, tmp[k * kTmpStride + j * 16 + lr],
                                                        y2[kk & 1], 0, 0, 0);
    }
    const v4f z = y2[0] + y2[1];
#pragma unroll
    for (int n = 0; n < 4; ++n) M[(32 + i * 16 + lg * 4 + n) * kMStride + j * 16 + lr] = -z[n];
  }
  // q R in the scan's order: a wave has half of its tile's channels.
#pragma unroll
  for (uint32_t k2 = 0; k2 < kD / 64; ++k2) {
    const uint32_t kb = late * (kD / 64) + k2;
    const uint8_t* const from = lds + tile * 2 * kRowPlane + lr * kRowStride + kb * 64 + lg * 8;
    uint8_t* const to = rec + kRecQ + (tile * (kD / 32) + kb) * 2048 + lane * 16;
#pragma unroll
    for (uint32_t x = 0; x < 2; ++x) {
      const v4h lo = *reinterpret_cast<const v4h*>(from + x * kRowPlane);
      const v4h hi = *reinterpret_cast<const v4h*>(from + x * kRowPlane + 32);
      *reinterpret_cast<v8h*>(to + x * 1024) = join(lo, hi);
    }
  }
  // P (4096 times itself): tiles (0,0) (1,0) (2,0) (2,1) (3,0) (3,1) of 16 x 32.
  if (w >= 2) {
    const uint32_t part = w - 2, ti = part < 2 ? part : 1 + (part >> 1), kb = part < 2 ? 0 : part & 1;
    const uint32_t row = ti * 16 + lr, s0 = kb * 32 + lg * 8;
    v4f x[2];
#pragma unroll
    for (int n = 0; n < 8; ++n)
      x[n >> 2][n & 3] = s0 + n <= row ? M[(s0 + n) * kMStride + row + 1] * 4096.0f : 0.0f;
    const Terms8 z = terms(x[0], x[1]);
    uint8_t* const to = rec + kRecP + part * 2048 + lane * 16;
    *reinterpret_cast<v8h*>(to) = z.hi;
    *reinterpret_cast<v8h*>(to + 1024) = z.lo;
  }
  __syncthreads();

  // T's terms (256 times itself) and k R (kUnit times), transposed: rows of 64 tokens.
  uint8_t* const tok = lds + 2 * kTPlane;
  auto put_tokens = [&](uint8_t* to, const v2f (&x)[8], v2f scale) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      v4f z[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i >> 2][i & 3] = x[i][c] * scale[c];
      const Terms8 s = terms(z[0], z[1]);
      uint8_t* const at = to + (ch + c) * kTokStride + t0 * 2;
      *reinterpret_cast<v8h*>(at) = s.hi;
      *reinterpret_cast<v8h*>(at + kTokPlane) = s.lo;
    }
  };
  {
    const uint32_t row = t >> 3, c0 = (t & 7) * 8;
    v4f z[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t col = c0 + i;
      z[i >> 2][i & 3] = col <= row ? M[row * kMStride + col] * beta[col] * 256.0f : 0.0f;
    }
    const Terms8 s = terms(z[0], z[1]);
    uint8_t* const at = lds + row * kTokStride + c0 * 2;
    *reinterpret_cast<v8h*>(at) = s.hi;
    *reinterpret_cast<v8h*>(at + kTPlane) = s.lo;
    put_tokens(tok, kr, before);
    // V's largest values by the wave, over the totals, which all have read
    v2f big = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      big[0] = fmaxf(big[0], fabsf(y[2][i][0]));
      big[1] = fmaxf(big[1], fabsf(y[2][i][1]));
    }
    *reinterpret_cast<v2f*>(total + w * kD + ch) = big;
  }
  __syncthreads();
  auto get_t = [&](uint32_t ti, uint32_t kb) {
    const uint8_t* const from = lds + (ti * 16 + lr) * kTokStride + kb * 64 + lg * 16;
    Terms8 s;
    s.hi = *reinterpret_cast<const v8h*>(from);
    s.lo = *reinterpret_cast<const v8h*>(from + kTPlane);
    return s;
  };
  auto get_tok = [&](uint32_t tile, uint32_t kb) {
    const uint8_t* const from = tok + (tile * 16 + lr) * kTokStride + kb * 64 + lg * 16;
    Terms8 s;
    s.hi = *reinterpret_cast<const v8h*>(from);
    s.lo = *reinterpret_cast<const v8h*>(from + kTokPlane);
    return s;
  };
  // Two channel tiles and two token tiles a wave: 0 and 3, or 1 and 2 (tiles 0 and 1
  // have no tokens past 32 before them).
  const uint32_t pair = w >> 1, ta = late, tb = 3 - late;
  {
    // -W (256 times itself): its transpose's tiles.
    v4f z[2][2] = {};
#pragma unroll
    for (uint32_t kb = 0; kb < 2; ++kb) {
      Terms8 k[2];
#pragma unroll
      for (uint32_t c = 0; c < 2; ++c) k[c] = get_tok(pair * 2 + c, kb);
      const Terms8 xa = get_t(ta, 0), xb = get_t(tb, kb);
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const v8h left = term == 0 ? k[c].lo : k[c].hi;
          if (kb == 0) z[0][c] = mfma(left, term == 1 ? xa.lo : xa.hi, z[0][c]);
          z[1][c] = mfma(left, term == 1 ? xb.lo : xb.hi, z[1][c]);
        }
    }
#pragma unroll
    for (uint32_t x = 0; x < 2; ++x) {
      const Terms8 s = terms(z[x][0] * (-1.0f / kUnit), z[x][1] * (-1.0f / kUnit));
      uint8_t* const to = rec + kRecW + ((x ? tb : ta) * (kD / 32) + pair) * 2048 + lane * 16;
      *reinterpret_cast<v8h*>(to) = s.hi;
      *reinterpret_cast<v8h*>(to + 1024) = s.lo;
    }
  }
  // V, each column scaled by 2^e to have its largest value in [2^8, 2^9).
  int32_t e[2];
  {
    v2f big = {0.0f, 0.0f};
#pragma unroll
    for (uint32_t b = 0; b < 8; ++b) {
      const v2f x = *reinterpret_cast<const v2f*>(total + b * kD + ch);
      big[0] = fmaxf(big[0], x[0]);
      big[1] = fmaxf(big[1], x[1]);
    }
    v2i top;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      top[c] = big[c] > 0.0f ? __builtin_amdgcn_frexp_expf(big[c]) : -1000;
      e[c] = big[c] > 0.0f ? 9 - top[c] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[2][i][c] = __builtin_ldexpf(y[2][i][c], e[c]);
    }
    if (w == 0) *reinterpret_cast<v2i*>(rec + kRecExps + ch * 4) = top;
  }
  __syncthreads();
  int32_t* const exps = reinterpret_cast<int32_t*>(tmp);
  put_tokens(tok, y[2], one);
  if (w == 0) {
    exps[ch] = e[0];
    exps[ch + 1] = e[1];
  }
  __syncthreads();
  {
    v4f z[2][2] = {};
#pragma unroll
    for (uint32_t kb = 0; kb < 2; ++kb) {
      Terms8 v[2];
#pragma unroll
      for (uint32_t c = 0; c < 2; ++c) v[c] = get_tok(pair * 2 + c, kb);
      const Terms8 xa = get_t(ta, 0), xb = get_t(tb, kb);
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const v8h right = term == 1 ? v[c].lo : v[c].hi;
          if (kb == 0) z[0][c] = mfma(term == 0 ? xa.lo : xa.hi, right, z[0][c]);
          z[1][c] = mfma(term == 0 ? xb.lo : xb.hi, right, z[1][c]);
        }
    }
#pragma unroll
    for (uint32_t c = 0; c < 2; ++c) {
      const uint32_t ct = pair * 2 + c;
      const int32_t back = -8 - exps[ct * 16 + lr];  // T is 256 times itself
#pragma unroll
      for (uint32_t x = 0; x < 2; ++x) {
#pragma unroll
        for (int n = 0; n < 4; ++n) z[x][c][n] = __builtin_ldexpf(z[x][c][n], back);
        *reinterpret_cast<v4f*>(rec + kRecU + (ct * 4 + (x ? tb : ta)) * 1024 + lane * 16) = z[x][c];
      }
    }
  }
}

// A sequence's chunks in order, kCt x 16 columns of a head's state a workgroup of four
// waves.  Wave w has rows 32 w .. 32 w + 31 of the state in registers (tile i: rows
// 16 i + 4 g + 0..3 of column lane % 16) and computes tokens 16 w .. 16 w + 15 of U and
// O, so that every operand that comes from memory is read by one wave alone: it
// goes straight to that wave's registers, a chunk ahead.  What the waves need of each
// other, the state's and U's terms, goes through LDS, in the order in which
// products take them: two barriers a chunk.
//
// A chunk takes 1.45 us (16 columns), of which 0.75 are the 116 KB that a CU takes in at
// 64 bytes a cycle; 2.2 us with 256 workgroups at once whose records come from HBM.  Before:
// one wave of 16 columns a workgroup, its operands as they were needed, 13 to 20 us; two
// waves computing and two staging through LDS 3.4 us.  Operands two chunks ahead were no
// faster (20011 tokens, 32 heads in all: 1191 us for 1166).
constexpr uint32_t kScanThreads = 256;

// The state's terms by 32 rows, U's by 32 tokens, the columns' largest values by wave.
template <uint32_t kCt>
struct ScanShared {
  v8h s[kCt][kD / 32][2][64];
  v8h u[kCt][2][2][64];
  float most[kCt][16][4];
};

// At a uniform address and a lane's offset.
__device__ __forceinline__ Terms8 read_terms(const uint8_t* p, uint32_t at) {
  Terms8 t;
  t.hi = *(const HKV_GLOBAL v8h*)((const HKV_GLOBAL uint8_t*)p + at);
  t.lo = *(const HKV_GLOBAL v8h*)((const HKV_GLOBAL uint8_t*)p + 1024 + at);
  return t;
}

// The part of a sequence that a workgroup goes through: chunks c0 .. c1 - 1 from
//   kSource  the source page's state, or
//   kJoined  the state before it, joined from what `parts` parts made.
// Without outputs (two column tiles, both of the same columns): what the part makes of any
// state S before it, M S + B, where B's tile starts from zeros and M's from the unit
// matrix, without V.
enum Start { kSource, kJoined, kNothing };
struct Part {
  Start start;
  uint32_t c0, c1;
  float* end;         // [kCt][kD][kD] the state behind the part (B and M), or nullptr
  const float* made;  // [parts][2][kD][kD]: B and M of each part before
  uint32_t parts;
};

template <class T, uint32_t kCt, bool kOut>
__device__ __forceinline__ void scan(const hkv::PrefillArgs& a, uint32_t s, uint32_t h,
                                     uint32_t group, const Part& part, ScanShared<kCt>& lds) {
  using E = typename T::type;
  const uint32_t w = wave_index(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int32_t row0 = a.starts[s], n = a.starts[s + 1] - row0;
  const uint32_t col0 = group * (kOut ? kCt : 1) * 16;
  E* const out = static_cast<E*>(a.out) + (int64_t)h * kD + col0 + lg * 4;
  if (a.status[s] == hkv::kPrefillRefused) {
    if (kOut)
      for (int32_t i = (int32_t)(lr + w * 16); i < n; i += 64)
#pragma unroll
        for (uint32_t ct = 0; ct < kCt; ++ct)
          T::store4(out + (int64_t)(row0 + i) * a.out_stride + ct * 16, v4f{NAN, NAN, NAN, NAN});
    return;
  }
  const int32_t src = a.src[s];
  const uint32_t slot0 = (uint32_t)a.first_chunk[s];
  const uint8_t* rec =
      a.records + ((uint64_t)(slot0 + part.c0) * a.heads + h) * hkv::kPrefillRecord;
  const uint64_t step = (uint64_t)a.heads * hkv::kPrefillRecord;
  const uint32_t state_at = (w * 32 + lg * 4) * kD + col0 + lr;  // of a head's [kD][kD]
  const uint64_t state_off = a.conv_bytes + ((uint64_t)h * kD * kD + state_at) * 4;
  v4f st[2][kCt];
  {
    const HKV_GLOBAL float* from = nullptr;
    if (part.start == kJoined)
      from = (const HKV_GLOBAL float*)(part.made + state_at);
    else if (part.start == kSource && src >= 0)
      from = (const HKV_GLOBAL float*)(a.pages + (uint64_t)src * a.stride + state_off);
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool one = !kOut && ct == 1 && w * 32 + i * 16 + lg * 4 + j == col0 + lr;
          st[i][ct][j] = one ? 1.0f : 0.0f;
          if (from) st[i][ct][j] = from[(i * 16 + j) * kD + ct * 16];
        }
  }

  // A chunk's operands of this wave.
  Terms8 wf[kD / 32], qf[kD / 32], pf[2], kf[2][2];
  v4f u0[kCt], decay[2];
  int32_t ve[kCt];  // exponents of V's columns, of the chunk after
  const uint32_t p_first = w < 2 ? w : 2 * w - 2;
  const uint32_t at = lane * 16;
  auto fetch_wq = [&](const uint8_t* r, uint32_t kb) {
    wf[kb] = read_terms(r + kRecW + (w * (kD / 32) + kb) * 2048, at);
    if (kOut) qf[kb] = read_terms(r + kRecQ + (w * (kD / 32) + kb) * 2048, at);
  };
  auto fetch_u = [&](const uint8_t* r) {
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct)
      if (!kOut && ct == 1)
        u0[ct] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      else
        u0[ct] = *(const HKV_GLOBAL v4f*)(r + kRecU + ((col0 / 16 + ct) * 4 + w) * 1024 + at);
  };
  auto fetch_k = [&](const uint8_t* r, uint32_t i, uint32_t kb) {
    kf[i][kb] = read_terms(r + kRecK + ((w * 2 + i) * 2 + kb) * 2048, at);
  };
  auto fetch_d = [&](const uint8_t* r) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
      decay[i] = *(const HKV_GLOBAL v4f*)(r + kRecDecay + (w * 32 + i * 16) * 4 + lg * 16);
  };
  auto fetch_p = [&](const uint8_t* r) {
    pf[0] = read_terms(r + kRecP + p_first * 2048, at);
    if (w >= 2) pf[1] = read_terms(r + kRecP + (p_first + 1) * 2048, at);
  };
  auto fetch_e = [&](const uint8_t* r) {
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct)
      ve[ct] = !kOut && ct == 1
                   ? -1000
                   : *(const HKV_GLOBAL int32_t*)(r + kRecExps + (col0 + ct * 16) * 4 + lr * 4);
  };

  // Columns are held 2^e times themselves.  The state's terms for the products of the
  // next chunk, scaled so that the largest value that the column's state, U and the
  // next chunk's V have lies in [2^3, 2^8): a state after a chunk is at most 65 times
  // the larger of the state before it and U, below fp16's limit of 2^16, and U at most
  // 23 times the state and 256 times V, below 16 times that.
  int e[kCt];
#pragma unroll
  for (uint32_t ct = 0; ct < kCt; ++ct) e[ct] = 0;
  auto put_most = [&](const v4f (&u)[kCt], float by) {
    float m[kCt];
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct) {
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x = fmaxf(x, fmaxf(fabsf(st[0][ct][j]), fabsf(st[1][ct][j])));
        y = fmaxf(y, fabsf(u[ct][j]));
      }
      x = fmaxf(x, y * by);
      const auto r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
      const uint32_t r0 = r[0], r1 = r[1];
      x = fmaxf(real(r0), real(r1));
      const auto q = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
      const uint32_t q0 = q[0], q1 = q[1];
      m[ct] = fmaxf(real(q0), real(q1));
    }
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct)
      if (lg == ct) lds.most[ct][lr][w] = m[ct];
  };
  int to[kCt];  // the columns' next exponents
  auto get_most = [&]() {
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct) {
      const v4f m = *reinterpret_cast<const v4f*>(lds.most[ct][lr]);
      const float big = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      const int top = max(big > 0.0f ? __builtin_amdgcn_frexp_expf(big) : -1000,
                          ve[ct] > -1000 ? ve[ct] + e[ct] : -1000);
      to[ct] = top > -1000 && (top < 4 || top > 8) ? e[ct] + 6 - top : e[ct];
    }
  };
  auto put_state = [&]() {
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct) {
      if (__any(to[ct] != e[ct])) {
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st[i][ct][j] = __builtin_ldexpf(st[i][ct][j], to[ct] - e[ct]);
        e[ct] = to[ct];
      }
      const Terms8 x = terms(st[0][ct], st[1][ct]);
      lds.s[ct][w][0][lane] = x.hi;
      lds.s[ct][w][1][lane] = x.lo;
    }
  };
  v4f none[kCt];
#pragma unroll
  for (uint32_t ct = 0; ct < kCt; ++ct) none[ct] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  // The state before the part: S <- M S + B for each of the parts between the first and
  // this one.  In fp32, since a part may be hundreds of chunks long: M's rows, S and B can
  // lie many powers of two apart, which no exponent of a column covers, and a small row
  // that stays counts as much as a large one that fades.  The columns of S go through LDS,
  // four rows 80 floats apart, so that the four lane groups read different banks.
  if constexpr (kOut) {
    if (part.start == kJoined) {
      float* const shared = reinterpret_cast<float*>(&lds);
      constexpr uint32_t kFour = 80, kTile = kD / 4 * kFour;
      static_assert(kCt * kTile * sizeof(float) <= sizeof(lds), "a state fits the scan's LDS");
      for (uint32_t x = 1; x < part.parts; ++x) {
        const HKV_GLOBAL float* const b =
            (const HKV_GLOBAL float*)(part.made + (uint64_t)x * 2 * kD * kD);
        const HKV_GLOBAL float* const m = b + kD * kD + (w * 32 + lr) * kD + lg * 4;
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
          for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              shared[ct * kTile + (w * 8 + i * 4 + lg) * kFour + j * 16 + lr] = st[i][ct][j];
              st[i][ct][j] = b[state_at + (i * 16 + j) * kD + ct * 16];
            }
        __syncthreads();
#pragma unroll
        for (uint32_t kb = 0; kb < kD / 16; ++kb) {
          const v4f row[2] = {*(const HKV_GLOBAL v4f*)(m + kb * 16),
                              *(const HKV_GLOBAL v4f*)(m + 16 * kD + kb * 16)};
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (uint32_t ct = 0; ct < kCt; ++ct) {
              const float s = shared[ct * kTile + (kb * 4 + lg) * kFour + n * 16 + lr];
#pragma unroll
              for (uint32_t i = 0; i < 2; ++i)
                st[i][ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(row[i][n], s, st[i][ct], 0, 0, 0);
            }
        }
        __syncthreads();
      }
    }
  }
  fetch_e(rec);
  fetch_u(rec);
#pragma unroll
  for (uint32_t kb = 0; kb < kD / 32; ++kb) fetch_wq(rec, kb);
  fetch_d(rec);
#pragma unroll
  for (uint32_t x = 0; x < 4; ++x) fetch_k(rec, x & 1, x >> 1);
  if (kOut) fetch_p(rec);
  put_most(none, 0.0f);
  __syncthreads();
  get_most();
  put_state();
  __syncthreads();
  hkv::PrefillChunk ck = read_chunk(a, slot0 + part.c0);
  for (uint32_t c = part.c0; c < part.c1; ++c) {
    const bool more = c + 1 < part.c1;
    const hkv::PrefillChunk ck_next = read_chunk(a, slot0 + (more ? c + 1 : c));
    // the last chunk's operands are fetched once more instead of none
    const uint8_t* const next = more ? rec + step : rec;
    fetch_e(next);
    Terms8 sf[2][kCt];
    auto get_state = [&](uint32_t kb) {
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct) {
        sf[kb & 1][ct].hi = lds.s[ct][kb][0][lane];
        sf[kb & 1][ct].lo = lds.s[ct][kb][1][lane];
      }
    };
    get_state(0);
    // U = U0 - W S, 256 2^e times itself.
    v4f u[kCt], o[kCt];
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[ct][j] = __builtin_ldexpf(u0[ct][j], e[ct] + 8);
        o[ct][j] = 0.0f;
      }
    // O's part from the state, 256 2^e times itself and transposed (a lane's token is
    // lane % 16 of its tile, its columns 4 g + 0..3), side by side with U: the products
    // of one sum lie 2 kCt apart.
    fetch_u(next);
#pragma unroll
    for (uint32_t kb = 0; kb < kD / 32; ++kb) {
      if (kb + 1 < kD / 32) get_state(kb + 1);
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (uint32_t ct = 0; ct < kCt; ++ct) {
          const v8h x = term == 1 ? sf[kb & 1][ct].lo : sf[kb & 1][ct].hi;
          u[ct] = mfma(term == 0 ? wf[kb].lo : wf[kb].hi, x, u[ct]);
          if (kOut) o[ct] = mfma(x, term == 0 ? qf[kb].lo : qf[kb].hi, o[ct]);
        }
      // operands of the next chunk as their registers become free: a CU takes 64
      // bytes a cycle, so that all of them in a row would hold up the products
      __builtin_amdgcn_sched_barrier(0);
      fetch_wq(next, kb);
      __builtin_amdgcn_sched_barrier(0);
    }
    // U over 16: P U, 4096 times itself, comes to 256 times, 16 (k D)^T U to itself.
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct) {
      u[ct] *= 1.0f / 4096.0f;
      const Terms2 x = terms(u[ct][0], u[ct][1]), y = terms(u[ct][2], u[ct][3]);
      // tokens 16 w + 4 g + 0..3: half of the 8 that group 2 (w % 2) + g / 2 takes
      const uint32_t to = lr + 32 * (w & 1) + 16 * (lg >> 1);
      v4h* const hi = reinterpret_cast<v4h*>(&lds.u[ct][w >> 1][0][to]) + (lg & 1);
      v4h* const lo = reinterpret_cast<v4h*>(&lds.u[ct][w >> 1][1][to]) + (lg & 1);
      *hi = v4h{x.hi[0], x.hi[1], y.hi[0], y.hi[1]};
      *lo = v4h{x.lo[0], x.lo[1], y.lo[0], y.lo[1]};
    }
    put_most(u, 16.0f);
    __syncthreads();
    // S <- D S + (k D)^T U.
    Terms8 uf[kCt][2];
#pragma unroll
    for (uint32_t kb = 0; kb < 2; ++kb)
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct) {
        uf[ct][kb].hi = lds.u[ct][kb][0][lane];
        uf[ct][kb].lo = lds.u[ct][kb][1][lane];
      }
    get_most();
    int back[kCt][4];  // the scales of the columns that the lane has of O
#pragma unroll
    for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
      for (int j = 0; j < 4; ++j) back[ct][j] = -8 - __shfl(e[ct], (int)(lg * 4 + j), 64);
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct) st[i][ct] *= decay[i];
    fetch_d(next);
#pragma unroll
    for (uint32_t kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
          for (uint32_t ct = 0; ct < kCt; ++ct)
            st[i][ct] = mfma(term == 0 ? kf[i][kb].lo : kf[i][kb].hi,
                             term == 1 ? uf[ct][kb].lo : uf[ct][kb].hi, st[i][ct]);
      __builtin_amdgcn_sched_barrier(0);
      fetch_k(next, 0, kb);
      fetch_k(next, 1, kb);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kOut && ck.dst >= 0) {
      HKV_GLOBAL float* p = (HKV_GLOBAL float*)(a.pages + (uint64_t)ck.dst * a.stride + state_off);
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            p[(i * 16 + j) * kD + ct * 16] = __builtin_ldexpf(st[i][ct][j], -e[ct]);
    }
    put_state();
    if constexpr (kOut) {
      // O's part from U.
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (uint32_t ct = 0; ct < kCt; ++ct)
          o[ct] = mfma(term == 1 ? uf[ct][0].lo : uf[ct][0].hi,
                       term == 0 ? pf[0].lo : pf[0].hi, o[ct]);
      if (w >= 2)
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
          for (uint32_t ct = 0; ct < kCt; ++ct)
            o[ct] = mfma(term == 1 ? uf[ct][1].lo : uf[ct][1].hi,
                         term == 0 ? pf[1].lo : pf[1].hi, o[ct]);
      fetch_p(next);
      const int32_t i = (int32_t)(w * 16 + lr);
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct) {
        v4f x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __builtin_ldexpf(o[ct][j], back[ct][j]) * a.scale;
        if (i < ck.len) T::store4(out + (int64_t)(ck.row + i) * a.out_stride + ct * 16, x);
      }
    }
    rec = next;
    ck = ck_next;
    __syncthreads();
  }
  if (part.end) {
    HKV_GLOBAL float* const p = (HKV_GLOBAL float*)(part.end + state_at);
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
      for (uint32_t ct = 0; ct < kCt; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          p[(kOut ? ct * 16 : ct * kD * kD) + (i * 16 + j) * kD] =
              __builtin_ldexpf(st[i][ct][j], -e[ct]);
  }
}

// Whether a sequence has chunks, or rows that are refused.
__device__ __forceinline__ bool scanned(const hkv::PrefillArgs& a, uint32_t s) {
  return a.status[s] != hkv::kPrefillNoRows &&
         a.starts[s + 1] - a.starts[s] > (int32_t)a.short_tokens;
}

template <class T, uint32_t kCt>
__device__ __forceinline__ void scan_all(const hkv::PrefillArgs& a, uint32_t s, uint32_t h,
                                         uint32_t, uint32_t group, ScanShared<kCt>& lds) {
  if (!scanned(a, s)) return;
  const Part part = {kSource, 0, (uint32_t)a.first_chunk[s + a.n_seqs], nullptr, nullptr, 0};
  scan<T, kCt, true>(a, s, h, group, part, lds);
}

// Few heads and long sequences: a sequence's chunks in a.parts parts (16384 tokens, 6 heads,
// in all: 279 to 291 us in 6 parts, 488 in one, 331 in 4, 308 in 8, where workgroups share
// CUs).  First the first
// part is gone through, and at the same time the others but the last make M and B; then
// every other part joins the state before it and is gone through.
constexpr uint32_t kLeastPart = 6;  // chunks
__device__ __forceinline__ uint32_t part_chunks(const hkv::PrefillArgs& a, uint32_t count) {
  return max((count + a.parts - 1) / a.parts, kLeastPart);
}
__device__ __forceinline__ float* made_by(const hkv::PrefillArgs& a, uint32_t s, uint32_t h,
                                          uint32_t part) {
  return a.made + (((uint64_t)s * a.heads + h) * (a.parts - 1) + part) * 2 * kD * kD;
}
template <class T>
__device__ __forceinline__ void scan_first(const hkv::PrefillArgs& a, uint32_t s, uint32_t h,
                                           uint32_t which, uint32_t group, ScanShared<2>& lds) {
  if (!scanned(a, s)) return;
  const uint32_t count = (uint32_t)a.first_chunk[s + a.n_seqs], each = part_chunks(a, count);
  Part part = {};
  part.c0 = which * each;
  part.c1 = min(part.c0 + each, count);
  if (part.c1 < count) part.end = made_by(a, s, h, which);
  if (which == 0) {
    part.start = kSource;
    scan<T, 1, true>(a, s, h, group, part, reinterpret_cast<ScanShared<1>&>(lds));
  } else if (part.c1 < count) {
    part.start = kNothing;
    scan<T, 2, false>(a, s, h, group, part, lds);
  }
}
template <class T>
__device__ __forceinline__ void scan_rest(const hkv::PrefillArgs& a, uint32_t s, uint32_t h,
                                          uint32_t set, uint32_t group, ScanShared<1>& lds) {
  if (!scanned(a, s) || a.status[s] != hkv::kPrefillRuns) return;
  const uint32_t which = set + 1;
  const uint32_t count = (uint32_t)a.first_chunk[s + a.n_seqs], each = part_chunks(a, count);
  Part part = {};
  part.c0 = which * each;
  part.c1 = min(part.c0 + each, count);
  if (part.c0 >= count) return;
  part.start = kJoined;
  part.made = made_by(a, s, h, 0);
  part.parts = which;
  scan<T, 1, true>(a, s, h, group, part, lds);
}

// The conv states of a sequence's blocks, a head's channels by one workgroup: it reads the
// source's before it writes any, since the source may be one of the blocks.
__device__ __forceinline__ void conv_states(const hkv::PrefillArgs& a, uint32_t s, uint32_t h) {
  if (a.status[s] != hkv::kPrefillRuns || !scanned(a, s)) return;
  const int32_t src = a.src[s], row0 = a.starts[s];
  const Span me = span_of(a, s);
  const int32_t* const own = a.table + (int64_t)s * a.table_stride;
  constexpr uint32_t kEach = (3 * kD + kScanThreads - 1) / kScanThreads;
  uint16_t old[kEach][3];
#pragma unroll
  for (uint32_t i = 0; i < kEach; ++i) {
    const uint32_t m = threadIdx.x + i * kScanThreads;
    const uint64_t ch = ((uint64_t)(m / kD) * a.heads + h) * kD + m % kD;
#pragma unroll
    for (int j = 0; j < 3; ++j)
      old[i][j] = src < 0 || m >= 3 * kD
                      ? 0
                      : reinterpret_cast<const uint16_t*>(a.pages + (uint64_t)src * a.stride)[ch * 3 + j];
  }
  for (uint32_t b = me.first; b <= me.last; ++b) {
    const int32_t dst = own[b];
    if (dst < 0) continue;
    // tokens up to the block's end, or the last
    const int32_t done =
        b < me.last ? (int32_t)((b + 1) * a.block_tokens) - me.position : me.tokens;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      const uint32_t m = threadIdx.x + i * kScanThreads;
      if (m >= 3 * kD) break;
      const uint64_t ch = ((uint64_t)(m / kD) * a.heads + h) * kD + m % kD;
      uint16_t* const to = reinterpret_cast<uint16_t*>(a.pages + (uint64_t)dst * a.stride) + ch * 3;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int32_t k = done - 3 + j;  // of the sequence's tokens
        uint16_t v = k == -3 ? old[i][0] : k == -2 ? old[i][1] : old[i][2];
        if (k >= 0)
          v = static_cast<const uint16_t*>(a.x)[(int64_t)(row0 + k) * a.x_stride + (int64_t)ch];
        to[j] = v;
      }
    }
  }
}

}  // namespace

extern "C" __global__ __launch_bounds__(kPlanThreads) void hkv_kda_prefill_clear(
    hkv::PrefillArgs a) {
  count_uses(a, true);
}
extern "C" __global__ __launch_bounds__(kPlanThreads) void hkv_kda_prefill_count(
    hkv::PrefillArgs a) {
  count_uses(a, false);
}
extern "C" __global__ __launch_bounds__(kPlanThreads) void hkv_kda_prefill_plan(
    hkv::PrefillArgs a) {
  plan(a);
}

#define HKV_TOKENS(name, T, d)                                                     \
  extern "C" __global__ __launch_bounds__(d * 4, d <= 128 ? 4 : 1) void name(      \
      hkv::PrefillArgs a) {                                                        \
    tokens<T, d>(a);                                                               \
  }
#define HKV_TOKENS_DIMS(suffix, T)                 \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d16, T, 16)    \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d32, T, 32)    \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d64, T, 64)    \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d128, T, 128)  \
  HKV_TOKENS(hkv_kda_tokens_##suffix##_d256, T, 256)
HKV_TOKENS_DIMS(bf16, Bf16)
HKV_TOKENS_DIMS(fp16, Fp16)
HKV_TOKENS_DIMS(fp32, Fp32)
#undef HKV_TOKENS
#undef HKV_TOKENS_DIMS

// The column groups of one part of a (sequence, head) pair lie 8 workgroups apart: on one
// XCD, which reads the part's records once.  The conv states' workgroups come last.
#define HKV_SCAN(name, tiles, columns, sets, convs, call)                                   \
  extern "C" __global__ __launch_bounds__(kScanThreads, 2) void name(hkv::PrefillArgs a) {  \
    __shared__ ScanShared<tiles> lds;                                                       \
    constexpr uint32_t kGroups = kD / (columns);                                            \
    const uint32_t n_sets = sets, pairs = a.n_seqs * a.heads, items = pairs * n_sets;       \
    const uint32_t scans = (items + 7) / 8 * 8 * kGroups;                                   \
    if (convs && blockIdx.x >= scans) {                                                     \
      const uint32_t pair = blockIdx.x - scans;                                             \
      conv_states(a, pair / a.heads, pair % a.heads);                                       \
      return;                                                                               \
    }                                                                                       \
    const uint32_t item = blockIdx.x / (8 * kGroups) * 8 + blockIdx.x % 8;                  \
    const uint32_t pair = item / n_sets, set = item % n_sets;                               \
    if (item < items)                                                                       \
      call(a, pair / a.heads, pair % a.heads, set, blockIdx.x / 8 % kGroups, lds);          \
  }
#define HKV_CHUNKS(suffix, T)                                                               \
  extern "C" __global__ __launch_bounds__(kFormThreads, 4) void hkv_kda_form_##suffix(      \
      hkv::PrefillArgs a) {                                                                 \
    __shared__ __attribute__((aligned(16))) uint8_t lds[kFormLds];                          \
    const uint32_t slot = blockIdx.x / a.heads;                                             \
    if (slot >= (uint32_t)a.first_chunk[2 * a.n_seqs] || a.chunks[slot].len == 0) return;   \
    form<T>(a, slot, blockIdx.x % a.heads, lds);                                            \
  }                                                                                         \
  HKV_SCAN(hkv_kda_scan_##suffix##_16, 1, 16, 1, true, scan_all<T>)                         \
  HKV_SCAN(hkv_kda_scan_##suffix##_32, 2, 32, 1, true, scan_all<T>)                         \
  HKV_SCAN(hkv_kda_scan_first_##suffix, 2, 16, a.parts - 1, true, scan_first<T>)            \
  HKV_SCAN(hkv_kda_scan_rest_##suffix, 1, 16, a.parts - 1, false, scan_rest<T>)
HKV_CHUNKS(bf16, Bf16)
HKV_CHUNKS(fp16, Fp16)
#undef HKV_CHUNKS
#undef HKV_SCAN

namespace hkv {

int launch_prefill(const PrefillArgs& a, int32_t dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
#define HKV_DIMS(suffix)                                                                \
  {HKV_FN(hkv_kda_tokens_##suffix##_d16), HKV_FN(hkv_kda_tokens_##suffix##_d32),        \
   HKV_FN(hkv_kda_tokens_##suffix##_d64), HKV_FN(hkv_kda_tokens_##suffix##_d128),       \
   HKV_FN(hkv_kda_tokens_##suffix##_d256)}
  static const void* const kTokens[3][5] = {HKV_DIMS(bf16), HKV_DIMS(fp16), HKV_DIMS(fp32)};
#undef HKV_DIMS
  uint32_t i = 0;
  while (i < 4 && (16u << i) != a.head_dim) ++i;
  PrefillArgs arg = a;
  void* params[] = {&arg};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  auto by_sequence = [&](const void* kernel) {
    if (e == hipSuccess)
      e = hipLaunchKernel(kernel, dim3(a.n_seqs), dim3(kPlanThreads), params, 0, st);
  };
  if (a.counted) {
    by_sequence(HKV_FN(hkv_kda_prefill_clear));
    by_sequence(HKV_FN(hkv_kda_prefill_count));
  }
  if (a.planned) by_sequence(HKV_FN(hkv_kda_prefill_plan));
  if (e != hipSuccess) return (int)e;
  if (a.chunked) {
    static const void* const kForm[2] = {HKV_FN(hkv_kda_form_bf16), HKV_FN(hkv_kda_form_fp16)};
    static const void* const kScan[2][2] = {
        {HKV_FN(hkv_kda_scan_bf16_16), HKV_FN(hkv_kda_scan_bf16_32)},
        {HKV_FN(hkv_kda_scan_fp16_16), HKV_FN(hkv_kda_scan_fp16_32)}};
    static const void* const kFirst[2] = {HKV_FN(hkv_kda_scan_first_bf16),
                                          HKV_FN(hkv_kda_scan_first_fp16)};
    static const void* const kRest[2] = {HKV_FN(hkv_kda_scan_rest_bf16),
                                         HKV_FN(hkv_kda_scan_rest_fp16)};
    const uint32_t pairs = a.n_seqs * a.heads;
    auto groups = [&](uint32_t sets, uint32_t tiles) {
      return (pairs * sets + 7) / 8 * 8 * (kD / 16 / tiles);
    };
    e = hipLaunchKernel(kForm[dtype], dim3(a.max_chunks * a.heads), dim3(kFormThreads), params, 0,
                        st);
    if (e != hipSuccess) return (int)e;
    if (a.parts > 1) {
      e = hipLaunchKernel(kFirst[dtype], dim3(groups(a.parts - 1, 1) + pairs),
                          dim3(kScanThreads), params, 0, st);
      if (e != hipSuccess) return (int)e;
      e = hipLaunchKernel(kRest[dtype], dim3(groups(a.parts - 1, 1)), dim3(kScanThreads),
                          params, 0, st);
    } else {
      const uint32_t tiles = a.column_tiles;
      e = hipLaunchKernel(kScan[dtype][tiles - 1], dim3(groups(1, tiles) + pairs),
                          dim3(kScanThreads), params, 0, st);
    }
    if (e != hipSuccess || a.short_tokens == 0) return (int)e;
  }
  return (int)hipLaunchKernel(kTokens[dtype][i], dim3(a.heads, a.n_seqs), dim3(64u << i), params,
                              0, st);
#undef HKV_FN
}

}  // namespace hkv
