// One token's step of a KDA layer on the pool's state pages (gfx950).
//
// Per head: with e = exp(log_decay), S' = diag(e) S, the step is
//   u = beta (v - S'^T k),  S = S' + k u^T,  out = S^T q = S'^T q + u (k . q)
// so one pass over S gives both column sums S'^T k and S'^T q, and the state
// is read once and written once.  A workgroup holds a head's d x d state in
// registers between the two: each thread has 4 columns of every kGroups-th
// row, the sums over rows are joined across the workgroup through LDS.
//
// Bound: reading and writing the page (2 x heads x d x d x 4 bytes a
// sequence); the arithmetic is 7 flops a value.  Measured: 256 sequences, 32
// heads of 128, a fifth without a state (1.01 GB) 183 us, 5.5 TB/s; 1 sequence, 16
// heads 6.7 us, a launch.  The state's loads are issued first, and the conv, the
// norms and the check of the block ids run while they are in flight.
//
// One workgroup owns a head entirely (its q, k and v channels of the conv
// state too), so a page may be updated in place without any other workgroup
// reading what this one writes.
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

template <class T, uint32_t kD, uint32_t kThreads>
__device__ __forceinline__ void step(const hkv::KdaArgs& a) {
  using E = typename T::type;
  constexpr uint32_t kRowThreads = kD / 4;               // threads that hold a row
  constexpr uint32_t kGroups = kThreads / kRowThreads;   // rows held at a time
  constexpr uint32_t kRows = kD / kGroups;               // rows per thread
  constexpr uint32_t kWaves = kThreads / 64;
  static_assert(kGroups * kRows == kD && kRowThreads <= 64, "a head splits into whole rows");
  __shared__ float y[3][kD];        // q, k, v after the conv
  __shared__ float decay[kD];
  __shared__ v4f sums[2][kWaves][kRowThreads];
  __shared__ uint32_t clashes[kWaves];
  const uint32_t h = blockIdx.x, s = blockIdx.y, t = threadIdx.x, lane = t & 63;
  const uint32_t c = t % kRowThreads, r0 = t / kRowThreads;
  const int32_t src = a.src[s], dst = a.dst[s];
  const bool bad_id = (src != HKV_NULL_BLOCK && (src < 0 || (uint32_t)src >= a.num_blocks)) ||
                      (dst != HKV_NULL_BLOCK && (dst < 0 || (uint32_t)dst >= a.num_blocks));
  const bool hit = src >= 0 && !bad_id;
  const uint64_t state_off = a.conv_bytes + (uint64_t)h * kD * kD * 4;

  v4f st[kRows];
  {
    const HKV_GLOBAL v4f* p =
        (const HKV_GLOBAL v4f*)(a.pages + (uint64_t)(hit ? src : 0) * a.stride + state_off) +
        r0 * kRowThreads + c;
#pragma unroll
    for (uint32_t i = 0; i < kRows; ++i) {
      st[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (hit) st[i] = __builtin_nontemporal_load(p + i * kGroups * kRowThreads);
    }
  }
  // A destination that another sequence of the call reads or writes.
  bool clash = false;
  if (dst >= 0)
    for (uint32_t i = t; i < a.n_seqs; i += kThreads)
      clash |= i != s && (a.src[i] == dst || a.dst[i] == dst);

  // The conv: one thread per channel, which also moves the channel's taps.
  E taps_new[(3 * kD + kThreads - 1) / kThreads][hkv::kKdaMaxKernel - 1];
  const uint32_t keep = a.taps - 1;
#pragma unroll
  for (uint32_t i = 0; i < (3 * kD + kThreads - 1) / kThreads; ++i) {
    const uint32_t w = t + i * kThreads;  // channel of this head: part * kD + column
    if (w >= 3 * kD) break;
    const uint64_t ch = ((uint64_t)(w / kD) * a.heads + h) * kD + w % kD;
    const E* wt = static_cast<const E*>(a.conv_weight) + ch * a.taps;
    const E* old = reinterpret_cast<const E*>(a.pages + (uint64_t)(hit ? src : 0) * a.stride) +
                   ch * keep;
    const E x = static_cast<const E*>(a.x)[(int64_t)s * a.x_stride + (int64_t)ch];
    float sum = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j) {
      if (j >= keep) continue;
      const E tap = hit ? old[j] : (E)0.0f;
      sum += (float)wt[j] * (float)tap;
      if (j > 0) taps_new[i][j - 1] = tap;
    }
#pragma unroll
    for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
      if (j + 1 == keep) taps_new[i][j] = x;
    sum += (float)wt[keep] * (float)x;
    y[w / kD][w % kD] = sum / (1.0f + expf(-sum));
  }
  for (uint32_t i = t; i < kD; i += kThreads)
    decay[i] = expf(a.log_decay[(int64_t)s * a.decay_stride + (int64_t)h * kD + i]);
  clash = __any(clash);
  if (lane == 0) clashes[t >> 6] = clash;
  __syncthreads();
  bool refused = bad_id;
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) refused |= clashes[w] != 0;

  // |q|^2, |k|^2 and q.k, by every wave for itself.
  float qq = 0.0f, kk = 0.0f, qk = 0.0f;
  for (uint32_t i = lane; i < kD; i += 64) {
    const float q = y[0][i], k = y[1][i];
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
    st[i] *= decay[r];
    sk += st[i] * (y[1][r] * nk);
    sq += st[i] * (y[0][r] * nq);
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
  const float beta = a.beta[(int64_t)s * a.beta_stride + h];
  v4f u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = beta * (y[2][c * 4 + i] - sk[i]);
  if (r0 == 0) {
    v4f o = sq + u * (qk * nq * nk);
    if (refused) o = v4f{NAN, NAN, NAN, NAN};
    T::store4(static_cast<E*>(a.out) + (int64_t)s * a.out_stride + (int64_t)h * kD + c * 4, o);
  }
  if (refused || dst < 0) return;
  HKV_GLOBAL v4f* p = (HKV_GLOBAL v4f*)(a.pages + (uint64_t)dst * a.stride + state_off) +
                      r0 * kRowThreads + c;
#pragma unroll
  for (uint32_t i = 0; i < kRows; ++i)
    __builtin_nontemporal_store(st[i] + u * (y[1][r0 + i * kGroups] * nk),
                                p + i * kGroups * kRowThreads);
#pragma unroll
  for (uint32_t i = 0; i < (3 * kD + kThreads - 1) / kThreads; ++i) {
    const uint32_t w = t + i * kThreads;
    if (w >= 3 * kD) break;
    const uint64_t ch = ((uint64_t)(w / kD) * a.heads + h) * kD + w % kD;
    E* to = reinterpret_cast<E*>(a.pages + (uint64_t)dst * a.stride) + ch * keep;
#pragma unroll
    for (uint32_t j = 0; j + 1 < hkv::kKdaMaxKernel; ++j)
      if (j < keep) to[j] = taps_new[i][j];
  }
}

}  // namespace

// Threads by head dim, so that a thread holds up to 16 rows of 4 columns and its
// state stays in registers (256 sequences, 32 heads: d = 64 67 us with 256
// threads, 70 with 512, 625 with 128, which spill; d = 128 210 us with 512, 212
// with 256, 311 with 1024, with a fifth of them without a state 183, 187, 259; 61
// sequences 54, 51, 75; 16 sequences 13.7, 14.6, 19.5; 4 7.5, 8.2, 8.8; 16 heads of
// d = 256 386 us with 1024, 666 with 512; d = 32 23 us with 64, 22 with 128, 29
// with 256).
#define HKV_KDA(name, T, d, threads)                                                        \
  extern "C" __global__ __launch_bounds__(threads, 4) void name(                            \
      hkv::KdaArgs a) {                                                                     \
    step<T, d, threads>(a);                                                                 \
  }
#define HKV_KDA_DIMS(suffix, T)                  \
  HKV_KDA(hkv_kda_step_##suffix##_d16, T, 16, 64)   \
  HKV_KDA(hkv_kda_step_##suffix##_d32, T, 32, 64)   \
  HKV_KDA(hkv_kda_step_##suffix##_d64, T, 64, 256)  \
  HKV_KDA(hkv_kda_step_##suffix##_d128, T, 128, 512) \
  HKV_KDA(hkv_kda_step_##suffix##_d256, T, 256, 1024)
HKV_KDA_DIMS(bf16, Bf16)
HKV_KDA_DIMS(fp16, Fp16)
HKV_KDA_DIMS(fp32, Fp32)
#undef HKV_KDA
#undef HKV_KDA_DIMS

namespace hkv {

int launch_kda(const KdaArgs& a, int32_t dtype, void* stream) {
#define HKV_FN(f) reinterpret_cast<const void*>(&f)
#define HKV_DIMS(suffix)                                                            \
  {HKV_FN(hkv_kda_step_##suffix##_d16), HKV_FN(hkv_kda_step_##suffix##_d32),        \
   HKV_FN(hkv_kda_step_##suffix##_d64), HKV_FN(hkv_kda_step_##suffix##_d128),       \
   HKV_FN(hkv_kda_step_##suffix##_d256)}
  static const void* const kKernels[3][5] = {HKV_DIMS(bf16), HKV_DIMS(fp16), HKV_DIMS(fp32)};
#undef HKV_DIMS
#undef HKV_FN
  static const uint32_t kThreads[5] = {64, 64, 256, 512, 1024};
  uint32_t i = 0;
  while (i < 4 && (16u << i) != a.head_dim) ++i;
  KdaArgs arg = a;
  void* params[] = {&arg};
  return (int)hipLaunchKernel(kKernels[dtype][i], dim3(a.heads, a.n_seqs), dim3(kThreads[i]),
                              params, 0, reinterpret_cast<hipStream_t>(stream));
}

}  // namespace hkv
