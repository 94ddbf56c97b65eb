// Appending tokens to an MLA layer's paged cache, and rotating their queries
// (gfx950).
//
// A row: latent columns c x w / sqrt(mean c^2 + eps), rotary columns turned by
// the position's angle, all divided by the cache's scale and rounded once; the
// sum of squares and everything else in fp32.  One wave holds a row, 8 values (16
// bytes) a lane and step; the norm needs one sum over the wave and no LDS.  The
// queries' rotary parts are independent 16-byte pieces, four a thread, in
// workgroups behind those of the rows.
//
// Bound: reading and writing each row and query once, a launch where they are few (us of
// the kernel): 15813 tokens, 32 heads, bf16 (170 MB) 35, 4.8 TB/s, the rate of a large
// copy; 5491 tokens, 64 heads, e4m3 (101 MB) 21; 255 sequences of one token, 16 heads 5.5; one
// 3.1.
#include <hip/hip_runtime.h>

#include "hkv.h"
#include "hkv_ops.hpp"

#define HKV_GLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v8f __attribute__((ext_vector_type(8)));

struct Bf16 {
  static __device__ __forceinline__ v8f widen(v4u x) {
    return __builtin_convertvector(__builtin_bit_cast(v8b, x), v8f);
  }
  static __device__ __forceinline__ v4u narrow(v8f x) {
    return __builtin_bit_cast(v4u, __builtin_convertvector(x, v8b));
  }
};
struct Fp16 {
  static __device__ __forceinline__ v8f widen(v4u x) {
    return __builtin_convertvector(__builtin_bit_cast(v8h, x), v8f);
  }
  static __device__ __forceinline__ v4u narrow(v8f x) {
    return __builtin_bit_cast(v4u, __builtin_convertvector(x, v8h));
  }
};

template <class T>
__device__ __forceinline__ v8f load8(const void* p) {
  return T::widen(*(const HKV_GLOBAL v4u*)p);
}

__device__ __forceinline__ float fp8_range(float x) {
  return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f);
}

// Eight e4m3 values; what lies beyond the type's range becomes its largest.
__device__ __forceinline__ v2u narrow_fp8(v8f x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fp8_range(x[i]);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return v2u{(uint32_t)lo, (uint32_t)hi};
}

struct Angles {
  v4f cos[2], sin[2];
};

// cos and sin of `count` (4 or 8) pairs from pair j on.
__device__ __forceinline__ Angles angles(const hkv::AppendArgs& a, int32_t position, uint32_t j,
                                         bool eight) {
  Angles g;
  if ((uint32_t)position >= a.n_positions) {
    g.cos[0] = g.cos[1] = g.sin[0] = g.sin[1] = v4f{NAN, NAN, NAN, NAN};
    return g;
  }
  const float* at = a.cos_sin + (uint64_t)(uint32_t)position * a.rotary + j;
  g.cos[0] = *(const HKV_GLOBAL v4f*)at;
  g.sin[0] = *(const HKV_GLOBAL v4f*)(at + a.rotary / 2);
  if (eight) {
    g.cos[1] = *(const HKV_GLOBAL v4f*)(at + 4);
    g.sin[1] = *(const HKV_GLOBAL v4f*)(at + a.rotary / 2 + 4);
  }
  return g;
}

// Eight columns that hold four pairs side by side.
__device__ __forceinline__ v8f turn_pairs(v8f x, const Angles& g) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float p = x[2 * j], q = x[2 * j + 1], c = g.cos[0][j], s = g.sin[0][j];
    x[2 * j] = p * c - q * s;
    x[2 * j + 1] = p * s + q * c;
  }
  return x;
}

// Eight pairs, whose other halves are in `y`: the first halves of the pairs with
// `low`, else the second.
__device__ __forceinline__ v8f turn_half(v8f x, v8f y, const Angles& g, bool low) {
  v8f r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = g.cos[j >> 2][j & 3], s = g.sin[j >> 2][j & 3];
    r[j] = low ? x[j] * c - y[j] * s : y[j] * s + x[j] * c;
  }
  return r;
}

// The sequence that row i belongs to: the last whose start is not past i.  Every
// lane of the wave asks for the same row; 64 starts are looked at in a step.
__device__ __forceinline__ uint32_t sequence_of(const int32_t* starts, uint32_t n, int32_t i,
                                                uint32_t lane) {
  uint32_t lo = 0, span = n;
  while (span > 1) {
    const uint32_t step = (span + 63) / 64, at = lane * step;
    const bool below = at < span && starts[lo + at] <= i;
    const uint32_t k = (uint32_t)__popcll(__ballot(below));
    if (k > 1) lo += (k - 1) * step, span -= (k - 1) * step;
    span = span < step ? span : step;
  }
  return lo;
}

template <class T, bool kFp8>
__device__ __forceinline__ void append_row(const hkv::AppendArgs& a, uint32_t i, uint32_t lane) {
  const uint32_t pieces = a.width / 8, latent = a.latent / 8;
  const uint32_t first = (a.width - a.rotary) / 8;  // the rotary part's first piece
  const uint8_t* row = static_cast<const uint8_t*>(a.kv) + (int64_t)i * a.kv_stride * 2;
  // what the wave reads does not depend on the sequence: it is in flight while
  // the sequence is looked for
  v8f x[2], y[2];
  const int32_t position = a.rotary ? a.positions[i] : 0;
#pragma unroll
  for (uint32_t k = 0; k < 2; ++k) {
    const uint32_t c = lane + 64 * k;
    x[k] = y[k] = v8f{};
    if (c >= pieces) continue;
    x[k] = load8<T>(row + c * 16);
    if (a.halves && c >= first) {
      const uint32_t half = a.rotary / 16;
      y[k] = load8<T>(row + (c - first < half ? c + half : c - half) * 16);
    }
  }
  uint32_t s = i;
  int32_t before = 0, after = 1;  // the sequence's rows of this call before and from this one on
  if (a.starts) {
    s = sequence_of(a.starts, a.n_seqs, (int32_t)i, lane);
    const int32_t lo = a.starts[s], hi = a.starts[s + 1];
    if (lo < 0 || lo > (int32_t)i || hi <= (int32_t)i || hi > (int32_t)a.n_tokens) return;
    before = (int32_t)i - lo;
    after = hi - (int32_t)i;
  }
  const int32_t len = a.lens[s];
  const int64_t cap = (int64_t)a.max_blocks * a.block_tokens;
  if (len < before + after || (int64_t)len > cap) return;
  const uint32_t slot = (uint32_t)(len - after);
  const int32_t block = a.table[(int64_t)s * a.table_stride + slot / a.block_tokens];
  if (block < 0 || (uint32_t)block >= a.num_blocks) return;  // HKV_NULL_BLOCK too

  if (a.norm) {
    float sum = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k)
      if (lane + 64 * k < latent)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += x[k][j] * x[k][j];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    const float by = 1.0f / sqrtf(sum / (float)a.latent + a.eps);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k)
      if (lane + 64 * k < latent)
        x[k] = x[k] * by *
               load8<T>(static_cast<const uint8_t*>(a.norm) + (lane + 64 * k) * 16);
  }
  uint8_t* to = a.pages + (uint64_t)(uint32_t)block * a.stride +
                (uint64_t)(slot % a.block_tokens) * (a.width * (kFp8 ? 1 : 2));
#pragma unroll
  for (uint32_t k = 0; k < 2; ++k) {
    const uint32_t c = lane + 64 * k;
    if (c >= pieces) continue;
    if (c >= first) {
      const uint32_t u = c - first, half = a.rotary / 16;
      if (a.halves) {
        const bool low = u < half;
        x[k] = turn_half(x[k], y[k], angles(a, position, 8 * (low ? u : u - half), true), low);
      } else {
        x[k] = turn_pairs(x[k], angles(a, position, 4 * u, false));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[k][j] = x[k][j] / a.cache_scale;
    if constexpr (kFp8)
      *(HKV_GLOBAL v2u*)(to + c * 8) = narrow_fp8(x[k]);
    else
      *(HKV_GLOBAL v4u*)(to + c * 16) = T::narrow(x[k]);
  }
}

constexpr uint32_t kThreads = 256;
constexpr uint32_t kRows = kThreads / 64;   // rows a workgroup
constexpr uint32_t kPieces = 4;             // query pieces a thread

// A piece of a query: eight columns, or with halves eight of either half.
template <class T>
__device__ __forceinline__ void turn_query(const hkv::AppendArgs& a, uint32_t i, uint32_t piece,
                                           uint32_t per_head) {
  const uint32_t h = piece / per_head, u = piece % per_head;
  const int32_t position = a.positions[i];
  const uint8_t* from = static_cast<const uint8_t*>(a.q_in) +
                        ((int64_t)i * a.q_in_token + (int64_t)h * a.q_in_head) * 2 + u * 16;
  uint8_t* to = static_cast<uint8_t*>(a.q_out) +
                ((int64_t)i * a.q_out_token + (int64_t)h * a.q_out_head) * 2 + u * 16;
  if (a.halves) {
    const Angles g = angles(a, position, 8 * u, true);
    const v8f x = load8<T>(from), y = load8<T>(from + a.rotary);
    *(HKV_GLOBAL v4u*)to = T::narrow(turn_half(x, y, g, true));
    *(HKV_GLOBAL v4u*)(to + a.rotary) = T::narrow(turn_half(y, x, g, false));
  } else {
    *(HKV_GLOBAL v4u*)to = T::narrow(turn_pairs(load8<T>(from), angles(a, position, 4 * u, false)));
  }
}

template <class T, bool kFp8>
__device__ __forceinline__ void append(const hkv::AppendArgs& a, uint32_t row_groups) {
  const uint32_t t = threadIdx.x;
  if (blockIdx.x < row_groups) {
    const uint32_t i = blockIdx.x * kRows + (t >> 6);
    if (i < a.n_tokens) append_row<T, kFp8>(a, i, t & 63);
    return;
  }
  const uint32_t per_head = a.halves ? a.rotary / 16 : a.rotary / 8;
  const uint32_t per_token = a.n_heads * per_head;
  const uint32_t tokens = (kThreads * kPieces + per_token - 1) / per_token;
  const uint32_t i0 = (blockIdx.x - row_groups) * tokens;
  uint32_t lo = 0, hi = a.n_tokens;  // the rows of the call's sequences
  if (a.starts) {
    const int32_t b = a.starts[0], e = a.starts[a.n_seqs];
    lo = b < 0 ? 0 : (uint32_t)b;
    hi = e < 0 ? 0 : (uint32_t)e < hi ? (uint32_t)e : hi;
  }
  for (uint32_t p = t; p < tokens * per_token; p += kThreads) {
    const uint32_t i = i0 + p / per_token;
    if (i >= lo && i < hi) turn_query<T>(a, i, p % per_token, per_head);
  }
}

}  // namespace

#define HKV_APPEND(name, T, fp8)                                                     \
  extern "C" __global__ __launch_bounds__(kThreads) void name(hkv::AppendArgs a,     \
                                                              uint32_t row_groups) { \
    append<T, fp8>(a, row_groups);                                                   \
  }
HKV_APPEND(hkv_mla_append_bf16, Bf16, false)
HKV_APPEND(hkv_mla_append_fp16, Fp16, false)
HKV_APPEND(hkv_mla_append_bf16_fp8, Bf16, true)
HKV_APPEND(hkv_mla_append_fp16_fp8, Fp16, true)
#undef HKV_APPEND

namespace hkv {

int launch_append(const AppendArgs& a, int32_t dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
  static const void* const kKernels[2][2] = {
      {HKV_FN(hkv_mla_append_bf16), HKV_FN(hkv_mla_append_bf16_fp8)},
      {HKV_FN(hkv_mla_append_fp16), HKV_FN(hkv_mla_append_fp16_fp8)}};
#undef HKV_FN
  AppendArgs arg = a;
  uint32_t row_groups = (a.n_tokens + kRows - 1) / kRows, groups = row_groups;
  if (a.n_heads) {
    const uint32_t per_token = a.n_heads * (a.halves ? a.rotary / 16 : a.rotary / 8);
    const uint32_t tokens = (kThreads * kPieces + per_token - 1) / per_token;
    groups += (a.n_tokens + tokens - 1) / tokens;
  }
  void* params[] = {&arg, &row_groups};
  return (int)hipLaunchKernel(kKernels[dtype == HKV_FP16][a.cache_bytes == 1], dim3(groups),
                              dim3(kThreads), params, 0, reinterpret_cast<hipStream_t>(stream));
}

}  // namespace hkv
