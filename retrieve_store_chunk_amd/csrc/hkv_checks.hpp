// Host checks that the operators on the pool's pages share (hkv_ops.cpp,
// hkv_prompt.cpp).
#pragma once

#include <cstddef>
#include <cstdint>
#include <exception>
#include <string>
#include <utility>

#include "hkv.h"
#include "hkv_handle.hpp"

namespace hkv {

// Nothing may leave a C entry point but a status.
template <class F>
hkv_status guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    return HKV_E_ARG;  // out of host memory while a message was put together
  }
}

// A buffer of the call: [lo, lo + bytes).  `written`: it must not overlap any
// other.
struct Buffer {
  const void* p;
  uint64_t bytes;
  bool written;
  const char* what;
};

template <size_t N>
hkv_status check_overlap(const Buffer (&b)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = i + 1; j < N; ++j) {
      if (!b[i].p || !b[j].p || !b[i].bytes || !b[j].bytes) continue;
      if (!b[i].written && !b[j].written) continue;
      const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p);
      const uintptr_t y = reinterpret_cast<uintptr_t>(b[j].p);
      if (x < y + b[j].bytes && y < x + b[i].bytes)
        return set_error(HKV_E_ALIAS, std::string(b[i].what) + " overlaps " + b[j].what);
    }
  return HKV_OK;
}

// Elements from a strided array's first to its last, plus one; -1 if that
// overflows.  Strides are >= 0, counts >= 1.
inline int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
  int64_t a = 0, b = 0, r = 0;
  if (__builtin_mul_overflow(n0 - 1, s0, &a) || __builtin_mul_overflow(n1 - 1, s1, &b) ||
      __builtin_add_overflow(a, b, &r) || __builtin_add_overflow(r, inner, &r) ||
      r > (int64_t(1) << 58))
    return -1;
  return r;
}

// Whether rows of `inner` elements at i0 * s0 + i1 * s1 are disjoint: the
// smaller stride steps over a row, the larger over all rows of the smaller.
inline bool rows_disjoint(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
  if (n0 <= 1 && n1 <= 1) return true;
  if (n0 <= 1) return s1 >= inner;
  if (n1 <= 1) return s0 >= inner;
  if (s0 > s1) {
    std::swap(s0, s1);
    std::swap(n0, n1);
  }
  return s0 >= inner && s1 >= extent(n0, s0, 1, 0, inner);
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline hkv_status layer_of(const Plan& p, int32_t layer, bool mla, const LayerPlacement** out) {
  if (layer < 0 || layer >= (int32_t)p.layers.size())
    return set_error(HKV_E_ARG, "layer index out of range");
  if ((p.layers[layer].is_mla != 0) != mla)
    return set_error(HKV_E_ARG, std::string("layer ") + std::to_string(layer) + " is not " +
                                    (mla ? "an MLA" : "a KDA") + " layer");
  *out = &p.layers[layer];
  return HKV_OK;
}

// The block table's shape and the pool's row geometry, as every MLA operator
// needs them.
inline hkv_status check_table(const Plan& p, int32_t n_seqs, int32_t max_blocks,
                       int64_t table_stride) {
  if (n_seqs < 0 || n_seqs > 65535) return set_error(HKV_E_ARG, "n_seqs must be in [0, 65535]");
  if (max_blocks < 1) return set_error(HKV_E_ARG, "max_blocks must be >= 1");
  if ((uint64_t)max_blocks * (uint64_t)p.block_size > 0x7FFFFFFFull)
    return set_error(HKV_E_ARG, "max_blocks x N exceeds 2^31 - 1 tokens");
  if (table_stride < 0) return set_error(HKV_E_ARG, "table_stride must be >= 0");
  return HKV_OK;
}

}  // namespace hkv
