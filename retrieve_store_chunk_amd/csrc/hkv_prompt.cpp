// C ABI of the operators that bring new tokens into the pool (declared in
// include/hkv.h): appending MLA rows and the KDA prefill.  Every call checks
// its arguments on the host, then enqueues kernel launches on the caller's
// stream; none allocates or synchronises.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <string>

#include "hkv.h"
#include "hkv_checks.hpp"
#include "hkv_handle.hpp"
#include "hkv_ops.hpp"

using hkv::aligned16;
using hkv::aligned_to;
using hkv::Buffer;
using hkv::check_overlap;
using hkv::check_table;
using hkv::DeviceScope;
using hkv::extent;
using hkv::guarded;
using hkv::hip_error;
using hkv::layer_of;
using hkv::rows_disjoint;
using hkv::set_error;
using hkv::stream_device;
using hkv::trace_on;

namespace {

hkv_status check_tokens(int32_t n_tokens) {
  if (n_tokens < 0 || n_tokens > hkv::kPromptMaxTokens)
    return set_error(HKV_E_ARG, "n_tokens must be in [0, 2^20]");
  return HKV_OK;
}

// ---------------------------------------------------------------- append
hkv_status append(const hkv_layout* layout, void* pool, const hkv_mla_append_args* a,
                  void* stream) {
  if (!layout || !a) return set_error(HKV_E_ARG, "layout and args must not be NULL");
  const hkv::Plan& p = layout->plan;
  const hkv::LayerPlacement* L = nullptr;
  hkv_status st = layer_of(p, a->layer, true, &L);
  if (st != HKV_OK) return st;
  const int64_t width = p.shapes[6], bytes = p.shapes[7];
  if (bytes != 1 && bytes != 2)
    return set_error(HKV_E_ARG, "the append needs mla_bytes 1 (e4m3) or 2 (bf16, fp16)");
  if (width % 16 != 0 || width > (int64_t)hkv::kAppendMaxWidth)
    return set_error(HKV_E_ARG, "the append needs an mla_width that is a multiple of 16 and at "
                                "most 1024");
  st = check_table(p, a->n_seqs, a->max_blocks, a->table_stride);
  if (st != HKV_OK) return st;
  st = check_tokens(a->n_tokens);
  if (st != HKV_OK) return st;
  if (!a->seq_starts && a->n_tokens != a->n_seqs)
    return set_error(HKV_E_ARG, "without seq_starts n_tokens must be n_seqs");
  if (a->n_heads < 0 || a->n_heads > 128)
    return set_error(HKV_E_ARG, "n_heads must be in [0, 128]");
  if (a->dtype != HKV_BF16 && a->dtype != HKV_FP16)
    return set_error(HKV_E_ARG, "dtype must be HKV_BF16 or HKV_FP16");
  if (a->cache_dtype != (bytes == 1 ? HKV_E4M3 : a->dtype))
    return set_error(HKV_E_ARG, bytes == 1 ? "a cache of 1-byte values must be HKV_E4M3"
                                           : "a cache of 2-byte values must be of kv's type");
  if (a->rotary_dim < 0 || a->rotary_dim % 16 != 0 || a->rotary_dim > width)
    return set_error(HKV_E_ARG, "rotary_dim must be a multiple of 16 in [0, mla_width]");
  if (a->latent_width < 0 || a->latent_width % 8 != 0 || a->latent_width > width - a->rotary_dim)
    return set_error(HKV_E_ARG, "latent_width must be a multiple of 8 in [0, mla_width - "
                                "rotary_dim]");
  if (a->rotary_halves != 0 && a->rotary_halves != 1)
    return set_error(HKV_E_ARG, "rotary_halves must be 0 or 1");
  if (a->n_positions < 0) return set_error(HKV_E_ARG, "n_positions must be >= 0");
  if (!std::isfinite(a->eps) || a->eps < 0)
    return set_error(HKV_E_ARG, "eps must be finite and >= 0");
  if (!std::isfinite(a->cache_scale) || !(a->cache_scale > 0))
    return set_error(HKV_E_ARG, "cache_scale must be finite and > 0");
  if (a->n_seqs == 0 || a->n_tokens == 0) return HKV_OK;
  const bool turns = a->rotary_dim > 0, queries = turns && a->n_heads > 0;
  if (!pool || !a->kv || !a->seq_lens || !a->block_table)
    return set_error(HKV_E_ARG, "pool, kv, seq_lens and block_table must not be NULL");
  if (turns && (!a->cos_sin || !a->positions))
    return set_error(HKV_E_ARG, "a rotation needs cos_sin and positions");
  if (queries && (!a->q_in || !a->q_out))
    return set_error(HKV_E_ARG, "q_in and q_out must not be NULL where n_heads > 0");
  if (a->kv_stride < 0 || a->q_in_token_stride < 0 || a->q_in_head_stride < 0 ||
      a->q_out_token_stride < 0 || a->q_out_head_stride < 0)
    return set_error(HKV_E_ARG, "strides must be >= 0");
  const int64_t n = a->n_seqs, T = a->n_tokens, H = a->n_heads, r = a->rotary_dim;
  if (queries && !rows_disjoint(T, a->q_out_token_stride, H, a->q_out_head_stride, r))
    return set_error(HKV_E_ALIAS, "the strides make rows of q_out overlap");
  const int64_t kv_ext = extent(T, a->kv_stride, 1, 0, width);
  const int64_t t_ext = extent(n, a->table_stride, 1, 0, a->max_blocks);
  const int64_t qi_ext = queries ? extent(T, a->q_in_token_stride, H, a->q_in_head_stride, r) : 0;
  const int64_t qo_ext = queries ? extent(T, a->q_out_token_stride, H, a->q_out_head_stride, r) : 0;
  if (kv_ext < 0 || t_ext < 0 || qi_ext < 0 || qo_ext < 0)
    return set_error(HKV_E_ARG, "strides are too large");
  if (!aligned16(pool) || !aligned16(a->kv) || !aligned16(a->norm_weight) ||
      (turns && !aligned16(a->cos_sin)) || (queries && (!aligned16(a->q_in) || !aligned16(a->q_out))))
    return set_error(HKV_E_ALIGN, "pool, kv, norm_weight, cos_sin, q_in and q_out must be 16-byte "
                                  "aligned");
  if (a->kv_stride % 8 != 0 ||
      (queries && (a->q_in_token_stride | a->q_in_head_stride | a->q_out_token_stride |
                   a->q_out_head_stride) % 8 != 0))
    return set_error(HKV_E_ALIGN, "strides of kv and the queries must be multiples of 8 elements");
  if (L->pool_offset % 16 != 0 || L->stride % 16 != 0)
    return set_error(HKV_E_ALIGN, "the layer's pages are not 16-byte aligned in this layout");
  if (!aligned_to(a->positions, 4) || !aligned_to(a->seq_starts, 4) ||
      !aligned_to(a->seq_lens, 4) || !aligned_to(a->block_table, 4))
    return set_error(HKV_E_ALIGN, "positions, seq_starts, seq_lens and block_table must be 4-byte "
                                  "aligned");
  const bool in_place = a->q_out == a->q_in && a->q_out_token_stride == a->q_in_token_stride &&
                        a->q_out_head_stride == a->q_in_head_stride;
  const Buffer buffers[] = {
      {pool, p.pool_used, true, "the pool"},
      {a->kv, (uint64_t)kv_ext * 2, false, "kv"},
      {a->norm_weight, (uint64_t)a->latent_width * 2, false, "norm_weight"},
      {turns ? a->cos_sin : nullptr, (uint64_t)a->n_positions * (uint64_t)r * 4, false, "cos_sin"},
      {turns ? a->positions : nullptr, (uint64_t)T * 4, false, "positions"},
      {a->seq_starts, (uint64_t)(n + 1) * 4, false, "seq_starts"},
      {a->seq_lens, (uint64_t)n * 4, false, "seq_lens"},
      {a->block_table, (uint64_t)t_ext * 4, false, "block_table"},
      {queries && !in_place ? a->q_in : nullptr, (uint64_t)qi_ext * 2, false, "q_in"},
      {queries ? a->q_out : nullptr, (uint64_t)qo_ext * 2, true, "q_out"},
  };
  st = check_overlap(buffers);
  if (st != HKV_OK) return st;

  hkv::AppendArgs k{};
  k.pages = static_cast<uint8_t*>(pool) + L->pool_offset;
  k.stride = L->stride;
  k.kv = a->kv;
  k.kv_stride = a->kv_stride;
  k.norm = a->norm_weight;
  k.cos_sin = a->cos_sin;
  k.positions = a->positions;
  k.starts = a->seq_starts;
  k.lens = a->seq_lens;
  k.table = a->block_table;
  k.table_stride = a->table_stride;
  k.q_in = a->q_in;
  k.q_in_token = a->q_in_token_stride;
  k.q_in_head = a->q_in_head_stride;
  k.q_out = a->q_out;
  k.q_out_token = a->q_out_token_stride;
  k.q_out_head = a->q_out_head_stride;
  k.eps = a->eps;
  k.cache_scale = a->cache_scale;
  k.num_blocks = (uint32_t)p.num_blocks;
  k.block_tokens = (uint32_t)p.block_size;
  k.max_blocks = (uint32_t)a->max_blocks;
  k.n_seqs = (uint32_t)n;
  k.n_tokens = (uint32_t)T;
  k.n_positions = (uint32_t)a->n_positions;
  k.n_heads = queries ? (uint32_t)H : 0;
  k.width = (uint32_t)width;
  k.latent = (uint32_t)a->latent_width;
  k.rotary = (uint32_t)r;
  k.halves = (uint32_t)a->rotary_halves;
  k.cache_bytes = (uint32_t)bytes;
  int dev = 0;
  st = stream_device(reinterpret_cast<hipStream_t>(stream), &dev);
  if (st != HKV_OK) return st;
  DeviceScope scope(dev);
  if (scope.err != hipSuccess) return hip_error(scope.err, "selecting the stream's device");
  const int e = hkv::launch_append(k, a->dtype, stream);
  if (e != 0) return hip_error((hipError_t)e, "launching the append");
  if (trace_on())
    std::fprintf(stderr, "[hkv] hkv_mla_append: layer %d, %d sequences, up to %d tokens, %d "
                 "heads\n", a->layer, a->n_seqs, a->n_tokens, a->n_heads);
  return HKV_OK;
}

// ---------------------------------------------------------------- KDA prefill
hkv_status plan_prefill(const hkv_layout* layout, const hkv_kda_prefill_args* a,
                        hkv::PrefillArgs* k, hkv::PrefillWorkspace* w) {
  const hkv::Plan& p = layout->plan;
  const int64_t heads = p.shapes[0], d = p.shapes[1], conv_dim = p.shapes[3], taps = p.shapes[4];
  const int64_t es = p.shapes[5];
  if (p.shapes[2] != 4) return set_error(HKV_E_ARG, "the prefill needs kda_state_bytes 4 (fp32)");
  if (d != 16 && d != 32 && d != 64 && d != 128 && d != 256)
    return set_error(HKV_E_ARG, "the prefill needs kda_head_dim 16, 32, 64, 128 or 256");
  if (heads > 65535) return set_error(HKV_E_ARG, "more than 65535 heads");
  if (conv_dim != 3 * heads * d)
    return set_error(HKV_E_ARG, "the prefill needs conv_dim = 3 x heads x head_dim");
  if (taps > (int64_t)hkv::kKdaMaxKernel)
    return set_error(HKV_E_ARG, "the prefill needs a conv_kernel of at most 8");
  if (!((es == 2 && (a->dtype == HKV_BF16 || a->dtype == HKV_FP16)) ||
        (es == 4 && a->dtype == HKV_FP32)))
    return set_error(HKV_E_ARG, "dtype must be HKV_BF16 or HKV_FP16 for conv_bytes 2, HKV_FP32 "
                                "for conv_bytes 4");
  hkv_status st = check_table(p, a->n_seqs, a->max_blocks, a->table_stride);
  if (st != HKV_OK) return st;
  if (a->n_seqs > (int32_t)hkv::kKdaMaxSeqs)
    return set_error(HKV_E_ARG, "n_seqs must be in [0, 4096]");
  st = check_tokens(a->n_tokens);
  if (st != HKV_OK) return st;
  if (a->max_seq_tokens < 0) return set_error(HKV_E_ARG, "max_seq_tokens must be >= 0");
  *k = hkv::PrefillArgs{};
  k->num_blocks = (uint32_t)p.num_blocks;
  k->block_tokens = (uint32_t)p.block_size;
  k->max_blocks = (uint32_t)a->max_blocks;
  k->n_seqs = (uint32_t)a->n_seqs;
  k->n_tokens = (uint32_t)a->n_tokens;
  k->max_seq_tokens = (uint32_t)std::min(a->max_seq_tokens, a->n_tokens);
  k->heads = (uint32_t)heads;
  k->head_dim = (uint32_t)d;
  k->taps = (uint32_t)taps;
  // In chunks where that pays (and is built): not for runs of a few tokens.
  k->short_tokens = k->n_seqs > 1 ? hkv::kPrefillShort : 0;
  k->chunked = d == (int64_t)hkv::kPrefillChunkDim && taps == 4 && es == 2 &&
               k->max_seq_tokens > (k->n_seqs > 1 ? hkv::kPrefillTokens
                                                  : hkv::kPrefillTokensOne);
  k->counted = k->n_tokens / k->block_tokens > hkv::kPrefillPairBlocks;
  k->planned = k->chunked || k->counted || k->n_seqs > hkv::kPrefillLookThrough;
  // A sequence's blocks are cut each on its own: the last chunk of the first, of
  // the last and of every whole block may be short.
  if (k->chunked)
    k->max_chunks = k->n_tokens / hkv::kPrefillChunk + k->n_tokens / k->block_tokens + 2 * k->n_seqs;
  // A launch has at most 2^32 threads: 512 for a chunk and head, 8 x 256 for a sequence
  // and head.
  if ((uint64_t)k->max_chunks * k->heads > (1u << 23) - 1 ||
      (uint64_t)k->n_seqs * k->heads > (1u << 20))
    return set_error(HKV_E_ARG, "too many heads for so many tokens or sequences; split the batch");
  const uint32_t pairs = k->n_seqs * k->heads;
  // 16 columns a scanning workgroup while each has a CU to itself, else 32, which read a
  // record half as often (us in all, 16 and 32 columns: 1887 tokens, 16 heads 83, 102; 20011
  // tokens, 32 heads 1167, 1266; 4 prompts and 24 single tokens, 32 heads 308, 262; 16
  // prompts, 32 heads 1055, 901).  All sequences count, short ones too: 20011 tokens beside
  // one single token, 32 heads, go by 32 columns, 1274 for 1159 alone.
  k->column_tiles = pairs * 8 > 256 ? 2 : 1;
  k->parts = 1;
  const uint32_t fit = 256 / (pairs * 8 > 0 ? pairs * 8 : 1) + 1;  // one workgroup a CU
  if (k->chunked && fit >= 4 && k->max_seq_tokens >= hkv::kPrefillPartTokens)
    k->parts = std::min<uint32_t>(fit, 8);
  *w = hkv::prefill_workspace(k->n_seqs, k->max_chunks, k->heads, k->parts,
                              k->counted ? k->num_blocks : 0);
  return HKV_OK;
}

hkv_status prefill(const hkv_layout* layout, void* pool, const hkv_kda_prefill_args* a, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!layout || !a) return set_error(HKV_E_ARG, "layout and args must not be NULL");
  const hkv::Plan& p = layout->plan;
  const hkv::LayerPlacement* L = nullptr;
  hkv_status st = layer_of(p, a->layer, false, &L);
  if (st != HKV_OK) return st;
  hkv::PrefillArgs k;
  hkv::PrefillWorkspace w;
  st = plan_prefill(layout, a, &k, &w);
  if (st != HKV_OK) return st;
  if (!std::isfinite(a->scale) || !std::isfinite(a->eps) || a->eps < 0)
    return set_error(HKV_E_ARG, "scale and eps must be finite, eps >= 0");
  if (a->n_seqs == 0 || a->n_tokens == 0) return HKV_OK;
  if (!pool || !a->x || !a->conv_weight || !a->log_decay || !a->beta || !a->seq_starts ||
      !a->positions || !a->src_blocks || !a->block_table || !a->out)
    return set_error(HKV_E_ARG, "no pointer may be NULL");
  if (a->x_stride < 0 || a->decay_stride < 0 || a->beta_stride < 0)
    return set_error(HKV_E_ARG, "strides must be >= 0");
  const int64_t n = a->n_seqs, T = a->n_tokens, heads = k.heads, hd = heads * k.head_dim;
  const int64_t conv_dim = 3 * hd, es = p.shapes[5];
  if (T > 1 && a->out_stride < hd)
    return set_error(HKV_E_ALIAS, "out_stride makes rows of out overlap");
  const int64_t x_ext = extent(T, a->x_stride, 1, 0, conv_dim);
  const int64_t g_ext = extent(T, a->decay_stride, 1, 0, hd);
  const int64_t b_ext = extent(T, a->beta_stride, 1, 0, heads);
  const int64_t o_ext = extent(T, std::max<int64_t>(a->out_stride, 0), 1, 0, hd);
  const int64_t t_ext = extent(n, a->table_stride, 1, 0, a->max_blocks);
  if (x_ext < 0 || g_ext < 0 || b_ext < 0 || o_ext < 0 || t_ext < 0)
    return set_error(HKV_E_ARG, "strides are too large");
  if (!ws || ws_bytes < w.total)
    return set_error(HKV_E_WORKSPACE, "workspace needs " + std::to_string(w.total) + " bytes");
  if (!aligned16(pool) || !aligned16(a->out) || !aligned16(ws))
    return set_error(HKV_E_ALIGN, "pool, out and workspace must be 16-byte aligned");
  if (T > 1 && a->out_stride % 4 != 0)
    return set_error(HKV_E_ALIGN, "out_stride must be a multiple of 4 elements");
  if (p.conv_part % 16 != 0 || L->pool_offset % 16 != 0 || L->stride % 16 != 0)
    return set_error(HKV_E_ALIGN, "the layer's recurrent states are not 16-byte aligned in this "
                                  "layout");
  if (!aligned_to(a->x, (uintptr_t)es) || !aligned_to(a->conv_weight, (uintptr_t)es))
    return set_error(HKV_E_ALIGN, "x or conv_weight is not aligned to its element");
  const void* words[] = {a->log_decay, a->beta, a->seq_starts, a->positions, a->src_blocks,
                         a->block_table};
  for (const void* v : words)
    if (!aligned_to(v, 4)) return set_error(HKV_E_ALIGN, "an array is not 4-byte aligned");
  const Buffer buffers[] = {
      {pool, p.pool_used, true, "the pool"},
      {a->x, (uint64_t)(x_ext * es), false, "x"},
      {a->conv_weight, (uint64_t)(conv_dim * k.taps * es), false, "conv_weight"},
      {a->log_decay, (uint64_t)g_ext * 4, false, "log_decay"},
      {a->beta, (uint64_t)b_ext * 4, false, "beta"},
      {a->seq_starts, (uint64_t)(n + 1) * 4, false, "seq_starts"},
      {a->positions, (uint64_t)n * 4, false, "positions"},
      {a->src_blocks, (uint64_t)n * 4, false, "src_blocks"},
      {a->block_table, (uint64_t)t_ext * 4, false, "block_table"},
      {a->out, (uint64_t)(o_ext * es), true, "out"},
      {ws, w.total, true, "the workspace"},
  };
  st = check_overlap(buffers);
  if (st != HKV_OK) return st;

  k.pages = static_cast<uint8_t*>(pool) + L->pool_offset;
  k.stride = L->stride;
  k.conv_bytes = p.conv_part;
  k.x = a->x;
  k.x_stride = a->x_stride;
  k.conv_weight = a->conv_weight;
  k.log_decay = a->log_decay;
  k.decay_stride = a->decay_stride;
  k.beta = a->beta;
  k.beta_stride = a->beta_stride;
  k.starts = a->seq_starts;
  k.positions = a->positions;
  k.src = a->src_blocks;
  k.table = a->block_table;
  k.table_stride = a->table_stride;
  k.out = a->out;
  k.out_stride = a->out_stride;
  k.scale = a->scale;
  k.eps = a->eps;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  k.status = reinterpret_cast<int32_t*>(wsb + w.status);
  k.uses = reinterpret_cast<uint32_t*>(wsb + w.uses);
  k.first_chunk = reinterpret_cast<int32_t*>(wsb + w.first_chunk);
  k.chunks = reinterpret_cast<hkv::PrefillChunk*>(wsb + w.chunks);
  k.records = wsb + w.records;
  k.made = reinterpret_cast<float*>(wsb + w.made);
  int dev = 0;
  st = stream_device(reinterpret_cast<hipStream_t>(stream), &dev);
  if (st != HKV_OK) return st;
  DeviceScope scope(dev);
  if (scope.err != hipSuccess) return hip_error(scope.err, "selecting the stream's device");
  const int e = hkv::launch_prefill(k, a->dtype, stream);
  if (e != 0) return hip_error((hipError_t)e, "launching the KDA prefill");
  if (trace_on())
    std::fprintf(stderr, "[hkv] hkv_kda_prefill: layer %d, %d sequences, up to %d tokens, %lld "
                 "heads of %u\n", a->layer, a->n_seqs, a->n_tokens, (long long)heads, k.head_dim);
  return HKV_OK;
}

}  // namespace

extern "C" {

hkv_status hkv_mla_append(const hkv_layout* layout, void* pool, const hkv_mla_append_args* args,
                          void* stream) {
  return guarded([&] { return append(layout, pool, args, stream); });
}

hkv_status hkv_kda_prefill_workspace(const hkv_layout* layout, const hkv_kda_prefill_args* args,
                                     size_t* bytes) {
  return guarded([&]() -> hkv_status {
    if (!layout || !args || !bytes)
      return set_error(HKV_E_ARG, "layout, args and bytes must not be NULL");
    hkv::PrefillArgs k;
    hkv::PrefillWorkspace w;
    const hkv_status st = plan_prefill(layout, args, &k, &w);
    if (st == HKV_OK) *bytes = (size_t)w.total;
    return st;
  });
}

hkv_status hkv_kda_prefill(const hkv_layout* layout, void* pool, const hkv_kda_prefill_args* args,
                           void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] { return prefill(layout, pool, args, workspace, ws_bytes, stream); });
}

}  // extern "C"
