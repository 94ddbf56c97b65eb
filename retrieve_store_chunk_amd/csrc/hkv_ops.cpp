// C ABI of the operators that read and update the pool in place (declared in
// include/hkv.h): MLA attention, eviction, the KDA step.  Every call checks its arguments on the
// host, then enqueues kernel launches on the caller's stream; none allocates
// or synchronises.
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

// ---------------------------------------------------------------- attention
// One workgroup (9 to 12 waves, 116 to 132 KB of LDS) fits a CU.  The head tiles
// of a batch run at once, those of one run of tokens on the same XCD (a
// multiple of 8 apart, but in calls of fewer tiles than workers), so that only
// the first reads from HBM.
hkv_status plan_attend(const hkv_layout* layout, const hkv_mla_attend_args* a, bool weights,
                       hkv::AttendArgs* k, hkv::AttendWorkspace* ws) {
  const hkv::Plan& p = layout->plan;
  const int64_t width = p.shapes[6], bytes = p.shapes[7];
  if (bytes != 1 && bytes != 2)
    return set_error(HKV_E_ARG, "attention needs mla_bytes 1 (e4m3) or 2 (bf16, fp16)");
  if (width % 32 != 0 || width > hkv::kAttendMaxWidth)
    return set_error(HKV_E_ARG, "attention needs an mla_width that is a multiple of 32 and at "
                                "most " + std::to_string(hkv::kAttendMaxWidth));
  hkv_status st = check_table(p, a->n_seqs, a->max_blocks, a->table_stride);
  if (st != HKV_OK) return st;
  if (a->n_heads < 1 || a->n_heads > 128)
    return set_error(HKV_E_ARG, "n_heads must be in [1, 128]");
  if (a->value_width < 16 || a->value_width % 16 != 0 ||
      a->value_width > (int32_t)hkv::kAttendMaxValues || a->value_width > width)
    return set_error(HKV_E_ARG, "value_width must be a multiple of 16, at most 512 and at most "
                                "mla_width");
  *k = hkv::AttendArgs{};
  k->num_blocks = (uint32_t)p.num_blocks;
  k->block_tokens = (uint32_t)p.block_size;
  k->row_bytes = (uint32_t)(width * bytes);
  k->width = (uint32_t)width;
  k->values = (uint32_t)a->value_width;
  k->n_seqs = (uint32_t)a->n_seqs;
  k->n_heads = (uint32_t)a->n_heads;
  k->max_blocks = (uint32_t)a->max_blocks;
  const uint64_t tokens = (uint64_t)a->max_blocks * (uint64_t)p.block_size;
  k->max_tiles = (uint32_t)((tokens + hkv::kAttendTile - 1) / hkv::kAttendTile);
  const uint64_t tiles = (uint64_t)k->n_seqs * k->max_tiles;
  if (tiles > 0x7FFFFFFFull)
    return set_error(HKV_E_ARG, "n_seqs x max_blocks x N exceeds 2^36 tokens; split the batch");
  k->head_tile = hkv::attend_head_tile(k->n_heads, tiles * ((k->n_heads + 15) / 16), bytes == 1);
  k->head_tiles = (k->n_heads + k->head_tile - 1) / k->head_tile;
  const uint64_t fit = hkv::kAttendMaxWorkers / k->head_tiles / 8 * 8;
  k->workers = (uint32_t)std::max<uint64_t>(1, std::min(fit, tiles));
  k->streams = tiles * hkv::kAttendTile * k->row_bytes > hkv::kAttendStreamBytes;
  // 512, 128 or 64 columns a joining workgroup: few (sequence, head) pairs are
  // spread over more workgroups, many need no more (in us, with 64, 128 and 512:
  // 1 sequence of 16000 tokens, 16 heads 18.8, 21.4, 38.6; 22 of 2011, 16 heads
  // 23.9, 22.5, 23.7; 64 of 500, 64 heads 66.5, 50.2, 39.3).
  const uint64_t pairs = (uint64_t)k->n_seqs * k->n_heads;
  k->join_shift = pairs >= 1024 ? 7 : pairs >= 256 ? 5 : 4;
  *ws = hkv::attend_workspace(k->workers, k->head_tiles, k->head_tile, k->values, k->n_seqs,
                              k->n_heads, k->max_tiles, weights);
  return HKV_OK;
}

hkv_status attend(const hkv_layout* layout, const void* pool, const hkv_mla_attend_args* a,
                  void* ws, size_t ws_bytes, void* stream) {
  if (!layout || !a) return set_error(HKV_E_ARG, "layout and args must not be NULL");
  const hkv::Plan& p = layout->plan;
  const hkv::LayerPlacement* L = nullptr;
  hkv_status st = layer_of(p, a->layer, true, &L);
  if (st != HKV_OK) return st;
  hkv::AttendArgs k;
  hkv::AttendWorkspace w;
  st = plan_attend(layout, a, a->weights != nullptr, &k, &w);
  if (st != HKV_OK) return st;
  const int64_t width = p.shapes[6], bytes = p.shapes[7];
  if (a->dtype != HKV_BF16 && a->dtype != HKV_FP16)
    return set_error(HKV_E_ARG, "dtype must be HKV_BF16 or HKV_FP16");
  if (a->cache_dtype != (bytes == 1 ? HKV_E4M3 : a->dtype))
    return set_error(HKV_E_ARG, bytes == 1 ? "a cache of 1-byte values must be HKV_E4M3"
                                           : "a cache of 2-byte values must be of q's type");
  if (!std::isfinite(a->scale) || !std::isfinite(a->cache_scale) ||
      !std::isfinite(a->scale * a->cache_scale))
    return set_error(HKV_E_ARG, "scale, cache_scale and their product must be finite");
  if (a->n_seqs == 0) return HKV_OK;
  if (!pool || !a->q || !a->block_table || !a->seq_lens || !a->out)
    return set_error(HKV_E_ARG, "pool, q, block_table, seq_lens and out must not be NULL");
  if (a->q_seq_stride < 0 || a->q_head_stride < 0 || a->out_seq_stride < 0 ||
      a->out_head_stride < 0)
    return set_error(HKV_E_ARG, "strides must be >= 0");
  const int64_t n = a->n_seqs, H = a->n_heads;
  if (!rows_disjoint(n, a->out_seq_stride, H, a->out_head_stride, a->value_width))
    return set_error(HKV_E_ALIAS, "the strides make rows of out overlap");
  const int64_t tokens = (int64_t)a->max_blocks * p.block_size;
  if (a->weights && a->weights_stride < tokens)
    return set_error(HKV_E_ARG, "weights_stride must be >= max_blocks x N");
  const int64_t q_ext = extent(n, a->q_seq_stride, H, a->q_head_stride, width);
  const int64_t o_ext = extent(n, a->out_seq_stride, H, a->out_head_stride, a->value_width);
  const int64_t t_ext = extent(n, a->table_stride, 1, 0, a->max_blocks);
  const int64_t w_ext = extent(n, a->weights_stride, 1, 0, tokens);
  if (q_ext < 0 || o_ext < 0 || t_ext < 0 || (a->weights && w_ext < 0))
    return set_error(HKV_E_ARG, "strides are too large");
  if (!ws || ws_bytes < w.total)
    return set_error(HKV_E_WORKSPACE, "workspace needs " + std::to_string(w.total) + " bytes");
  if (!aligned16(pool) || !aligned16(a->q) || !aligned16(a->out) || !aligned16(ws))
    return set_error(HKV_E_ALIGN, "pool, q, out and workspace must be 16-byte aligned");
  if ((a->q_seq_stride | a->q_head_stride | a->out_seq_stride | a->out_head_stride) % 8 != 0)
    return set_error(HKV_E_ALIGN, "strides of q and out must be multiples of 8 elements");
  if (L->pool_offset % 16 != 0 || L->stride % 16 != 0)
    return set_error(HKV_E_ALIGN, "the layer's pages are not 16-byte aligned in this layout");
  if (!aligned_to(a->block_table, 4) || !aligned_to(a->seq_lens, 4) || !aligned_to(a->lse, 4) ||
      !aligned_to(a->weights, 4))
    return set_error(HKV_E_ALIGN, "block_table, seq_lens, lse and weights must be 4-byte aligned");
  const Buffer buffers[] = {
      {pool, p.pool_used, false, "the pool"},
      {a->q, (uint64_t)q_ext * 2, false, "q"},
      {a->block_table, (uint64_t)t_ext * 4, false, "block_table"},
      {a->seq_lens, (uint64_t)n * 4, false, "seq_lens"},
      {a->out, (uint64_t)o_ext * 2, true, "out"},
      {a->lse, (uint64_t)(n * H) * 4, true, "lse"},
      {a->weights, a->weights ? (uint64_t)w_ext * 4 : 0, true, "weights"},
      {ws, w.total, true, "the workspace"},
  };
  st = check_overlap(buffers);
  if (st != HKV_OK) return st;

  k.pages = static_cast<const uint8_t*>(pool) + L->pool_offset;
  k.stride = L->stride;
  k.q = a->q;
  k.q_seq_stride = a->q_seq_stride;
  k.q_head_stride = a->q_head_stride;
  k.table = a->block_table;
  k.table_stride = a->table_stride;
  k.lens = a->seq_lens;
  k.out = a->out;
  k.out_seq_stride = a->out_seq_stride;
  k.out_head_stride = a->out_head_stride;
  k.lse = a->lse;
  k.weights = a->weights;
  k.weights_stride = a->weights_stride;
  k.scale = a->scale * a->cache_scale;
  k.cache_scale = a->cache_scale;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  k.part_o = reinterpret_cast<float*>(wsb + w.part_o);
  k.part_ml = reinterpret_cast<float*>(wsb + w.part_ml);
  k.spans = reinterpret_cast<int32_t*>(wsb + w.spans);
  if (a->weights) {
    k.norm = reinterpret_cast<float*>(wsb + w.norm);
    k.logits = reinterpret_cast<float*>(wsb + w.logits);
  }
  int dev = 0;
  st = stream_device(reinterpret_cast<hipStream_t>(stream), &dev);
  if (st != HKV_OK) return st;
  DeviceScope scope(dev);
  if (scope.err != hipSuccess) return hip_error(scope.err, "selecting the stream's device");
  const int e = hkv::launch_attend(k, a->dtype, a->cache_dtype, stream);
  if (e != 0) return hip_error((hipError_t)e, "launching the attention kernels");
  if (trace_on())
    std::fprintf(stderr, "[hkv] hkv_mla_attend: layer %d, %d sequences of up to %lld tokens, "
                 "%d heads, %u workers\n", a->layer, a->n_seqs, (long long)tokens, a->n_heads,
                 k.workers);
  return HKV_OK;
}

// ---------------------------------------------------------------- eviction
hkv_status plan_evict(const hkv_layout* layout, const hkv_mla_evict_args* a, hkv::EvictArgs* k,
                      hkv::EvictWorkspace* w) {
  const hkv::Plan& p = layout->plan;
  if (a->n_layers < 1 || a->n_layers > (int32_t)hkv::kEvictMaxLayers)
    return set_error(HKV_E_ARG, "n_layers must be in [1, 64]");
  hkv_status st = check_table(p, a->n_seqs, a->max_blocks, a->table_stride);
  if (st != HKV_OK) return st;
  if (a->budget < 1) return set_error(HKV_E_ARG, "budget must be >= 1");
  if ((int64_t)a->n_layers * a->n_seqs > 65535)
    return set_error(HKV_E_ARG, "n_layers x n_seqs exceeds 65535; split the batch");
  if ((uint64_t)a->max_blocks * (uint64_t)p.block_size > (1ull << 28))
    return set_error(HKV_E_ARG, "eviction takes tables of at most 2^28 tokens");
  *k = hkv::EvictArgs{};
  k->num_blocks = (uint32_t)p.num_blocks;
  k->block_tokens = (uint32_t)p.block_size;
  k->row_bytes = (uint32_t)(p.shapes[6] * p.shapes[7]);
  k->n_layers = (uint32_t)a->n_layers;
  k->n_seqs = (uint32_t)a->n_seqs;
  k->max_blocks = (uint32_t)a->max_blocks;
  k->budget = (uint32_t)a->budget;
  const uint64_t slots = (uint64_t)a->max_blocks * (uint64_t)p.block_size;
  k->max_moves =
      slots > k->budget ? (uint32_t)std::min<uint64_t>(k->budget, slots - k->budget) : 0u;
  // Chunks of [0, budget) and of the slots after it.
  auto chunks = [](uint64_t n) { return (n + hkv::kEvictChunkSlots - 1) / hkv::kEvictChunkSlots; };
  if (slots > hkv::kEvictSelectSlots)
    k->chunks = (uint32_t)(chunks(std::min<uint64_t>(k->budget, slots)) +
                           chunks(slots > k->budget ? slots - k->budget : 0));
  k->by_pairs = k->max_blocks <= hkv::kEvictPairBlocks &&
                (uint64_t)k->n_seqs * k->max_blocks * k->max_blocks <= hkv::kEvictPairs;
  *w = hkv::evict_workspace(k->num_blocks, k->n_seqs, (uint64_t)k->n_layers * k->n_seqs,
                            k->max_moves, k->chunks, k->by_pairs != 0);
  return HKV_OK;
}

hkv_status evict(const hkv_layout* layout, void* pool, const hkv_mla_evict_args* a, void* ws,
                 size_t ws_bytes, void* stream) {
  if (!layout || !a) return set_error(HKV_E_ARG, "layout and args must not be NULL");
  const hkv::Plan& p = layout->plan;
  hkv::EvictArgs k;
  hkv::EvictWorkspace w;
  hkv_status st = plan_evict(layout, a, &k, &w);
  if (st != HKV_OK) return st;
  if (!a->layers) return set_error(HKV_E_ARG, "layers must not be NULL");
  for (int32_t i = 0; i < a->n_layers; ++i) {
    const hkv::LayerPlacement* L = nullptr;
    st = layer_of(p, a->layers[i], true, &L);
    if (st != HKV_OK) return st;
    if (L->kv_group != p.layers[a->layers[0]].kv_group)
      return set_error(HKV_E_ARG, "the layers of one call must be of one KV group");
    for (int32_t j = 0; j < i; ++j)
      if (a->layers[j] == a->layers[i])
        return set_error(HKV_E_ALIAS, "layer " + std::to_string(a->layers[i]) +
                                          " is given twice");
    k.page_of[i] = L->pool_offset;
    k.stride = L->stride;
  }
  if (a->sinks < 0 || a->recent < 0 || (int64_t)a->sinks + a->recent > a->budget)
    return set_error(HKV_E_ARG, "sinks and recent must be >= 0, their sum at most budget");
  if (a->n_seqs == 0) return HKV_OK;
  if (!pool || !a->block_table || !a->seq_lens || !a->next_positions || !a->weights ||
      !a->positions || !a->weights_out || !a->positions_out)
    return set_error(HKV_E_ARG, "only new_lens may be NULL");
  if (a->layer_stride < 0 || a->seq_stride < 0)
    return set_error(HKV_E_ARG, "strides must be >= 0");
  const int64_t n = a->n_seqs, nl = a->n_layers, slots = (int64_t)a->max_blocks * p.block_size;
  if (!rows_disjoint(nl, a->layer_stride, n, a->seq_stride, slots))
    return set_error(HKV_E_ALIAS, "the strides make rows of weights overlap");
  const int64_t m_ext = extent(nl, a->layer_stride, n, a->seq_stride, slots);
  const int64_t t_ext = extent(n, a->table_stride, 1, 0, a->max_blocks);
  if (m_ext < 0 || t_ext < 0) return set_error(HKV_E_ARG, "strides are too large");
  if (!ws || ws_bytes < w.total)
    return set_error(HKV_E_WORKSPACE, "workspace needs " + std::to_string(w.total) + " bytes");
  if (!aligned16(pool) || !aligned16(ws))
    return set_error(HKV_E_ALIGN, "pool and workspace must be 16-byte aligned");
  const void* words[] = {a->block_table, a->seq_lens, a->next_positions, a->weights,
                         a->positions, a->weights_out, a->positions_out, a->new_lens};
  for (const void* x : words)
    if (!aligned_to(x, 4)) return set_error(HKV_E_ALIGN, "an array is not 4-byte aligned");
  const uint64_t m_bytes = (uint64_t)m_ext * 4;
  const bool w_in = a->weights_out == a->weights, p_in = a->positions_out == a->positions;
  const Buffer buffers[] = {
      {pool, p.pool_used, true, "the pool"},
      {a->block_table, (uint64_t)t_ext * 4, false, "block_table"},
      {a->seq_lens, (uint64_t)n * 4, false, "seq_lens"},
      {a->next_positions, (uint64_t)n * 4, false, "next_positions"},
      {a->weights, w_in ? 0 : m_bytes, false, "weights"},
      {a->positions, p_in ? 0 : m_bytes, false, "positions"},
      {a->weights_out, m_bytes, true, "weights_out"},
      {a->positions_out, m_bytes, true, "positions_out"},
      {a->new_lens, (uint64_t)n * 4, true, "new_lens"},
      {ws, w.total, true, "the workspace"},
  };
  st = check_overlap(buffers);
  if (st != HKV_OK) return st;

  k.pool = static_cast<uint8_t*>(pool);
  k.table = a->block_table;
  k.table_stride = a->table_stride;
  k.lens = a->seq_lens;
  k.next = a->next_positions;
  k.weights = a->weights;
  k.positions = a->positions;
  k.weights_out = a->weights_out;
  k.positions_out = a->positions_out;
  k.layer_stride = a->layer_stride;
  k.seq_stride = a->seq_stride;
  k.new_lens = a->new_lens;
  k.sinks = (uint32_t)a->sinks;
  k.recent = (uint32_t)a->recent;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  k.claims = reinterpret_cast<int32_t*>(wsb + w.claims);
  k.ok = reinterpret_cast<int32_t*>(wsb + w.ok);
  k.moves = reinterpret_cast<uint32_t*>(wsb + w.moves);
  k.lists = reinterpret_cast<uint32_t*>(wsb + w.lists);
  k.hist = reinterpret_cast<uint32_t*>(wsb + w.hist);
  k.totals = reinterpret_cast<uint32_t*>(wsb + w.totals);
  k.least = reinterpret_cast<uint32_t*>(wsb + w.least);
  int dev = 0;
  st = stream_device(reinterpret_cast<hipStream_t>(stream), &dev);
  if (st != HKV_OK) return st;
  DeviceScope scope(dev);
  if (scope.err != hipSuccess) return hip_error(scope.err, "selecting the stream's device");
  const int e = hkv::launch_evict(k, stream);
  if (e != 0) return hip_error((hipError_t)e, "launching the eviction kernels");
  if (trace_on())
    std::fprintf(stderr, "[hkv] hkv_mla_evict: %d layers, %d sequences of up to %lld tokens, "
                 "budget %d\n", a->n_layers, a->n_seqs, (long long)slots, a->budget);
  return HKV_OK;
}

// ---------------------------------------------------------------- KDA step
hkv_status kda_step(const hkv_layout* layout, void* pool, const hkv_kda_step_args* a,
                    void* stream) {
  if (!layout || !a) return set_error(HKV_E_ARG, "layout and args must not be NULL");
  const hkv::Plan& p = layout->plan;
  const hkv::LayerPlacement* L = nullptr;
  hkv_status st = layer_of(p, a->layer, false, &L);
  if (st != HKV_OK) return st;
  const int64_t heads = p.shapes[0], d = p.shapes[1], conv_dim = p.shapes[3], taps = p.shapes[4];
  const int64_t es = p.shapes[5];
  if (p.shapes[2] != 4) return set_error(HKV_E_ARG, "the step needs kda_state_bytes 4 (fp32)");
  if (d != 16 && d != 32 && d != 64 && d != 128 && d != 256)
    return set_error(HKV_E_ARG, "the step needs kda_head_dim 16, 32, 64, 128 or 256");
  if (heads > 65535) return set_error(HKV_E_ARG, "more than 65535 heads");
  if (conv_dim != 3 * heads * d)
    return set_error(HKV_E_ARG, "the step needs conv_dim = 3 x heads x head_dim");
  if (taps > (int64_t)hkv::kKdaMaxKernel)
    return set_error(HKV_E_ARG, "the step needs a conv_kernel of at most 8");
  if (!((es == 2 && (a->dtype == HKV_BF16 || a->dtype == HKV_FP16)) ||
        (es == 4 && a->dtype == HKV_FP32)))
    return set_error(HKV_E_ARG, "dtype must be HKV_BF16 or HKV_FP16 for conv_bytes 2, HKV_FP32 "
                                "for conv_bytes 4");
  if (a->n_seqs < 0 || a->n_seqs > (int32_t)hkv::kKdaMaxSeqs)
    return set_error(HKV_E_ARG, "n_seqs must be in [0, 4096]");
  if (!std::isfinite(a->scale) || !std::isfinite(a->eps) || a->eps < 0)
    return set_error(HKV_E_ARG, "scale and eps must be finite, eps >= 0");
  if (a->n_seqs == 0) return HKV_OK;
  if (!pool || !a->x || !a->conv_weight || !a->log_decay || !a->beta || !a->src_blocks ||
      !a->dst_blocks || !a->out)
    return set_error(HKV_E_ARG, "no pointer may be NULL");
  if (a->x_stride < 0 || a->decay_stride < 0 || a->beta_stride < 0)
    return set_error(HKV_E_ARG, "strides must be >= 0");
  const int64_t n = a->n_seqs;
  if (n > 1 && a->out_stride < heads * d)
    return set_error(HKV_E_ALIAS, "out_stride makes rows of out overlap");
  const int64_t x_ext = extent(n, a->x_stride, 1, 0, conv_dim);
  const int64_t g_ext = extent(n, a->decay_stride, 1, 0, heads * d);
  const int64_t b_ext = extent(n, a->beta_stride, 1, 0, heads);
  const int64_t o_ext = extent(n, std::max<int64_t>(a->out_stride, 0), 1, 0, heads * d);
  if (x_ext < 0 || g_ext < 0 || b_ext < 0 || o_ext < 0)
    return set_error(HKV_E_ARG, "strides are too large");
  if (!aligned16(pool) || !aligned16(a->out))
    return set_error(HKV_E_ALIGN, "pool and out must be 16-byte aligned");
  if (n > 1 && a->out_stride % 4 != 0)
    return set_error(HKV_E_ALIGN, "out_stride must be a multiple of 4 elements");
  if (p.conv_part % 16 != 0 || L->pool_offset % 16 != 0 || L->stride % 16 != 0)
    return set_error(HKV_E_ALIGN, "the layer's recurrent states are not 16-byte aligned in this "
                                  "layout");
  if (!aligned_to(a->x, (uintptr_t)es) || !aligned_to(a->conv_weight, (uintptr_t)es) ||
      !aligned_to(a->log_decay, 4) || !aligned_to(a->beta, 4) || !aligned_to(a->src_blocks, 4) ||
      !aligned_to(a->dst_blocks, 4))
    return set_error(HKV_E_ALIGN, "an array is not aligned to its element");
  const Buffer buffers[] = {
      {pool, p.pool_used, true, "the pool"},
      {a->x, (uint64_t)(x_ext * es), false, "x"},
      {a->conv_weight, (uint64_t)(conv_dim * taps * es), false, "conv_weight"},
      {a->log_decay, (uint64_t)g_ext * 4, false, "log_decay"},
      {a->beta, (uint64_t)b_ext * 4, false, "beta"},
      {a->src_blocks, (uint64_t)n * 4, false, "src_blocks"},
      {a->dst_blocks, (uint64_t)n * 4, false, "dst_blocks"},
      {a->out, (uint64_t)(o_ext * es), true, "out"},
  };
  st = check_overlap(buffers);
  if (st != HKV_OK) return st;

  hkv::KdaArgs k{};
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
  k.src = a->src_blocks;
  k.dst = a->dst_blocks;
  k.out = a->out;
  k.out_stride = a->out_stride;
  k.scale = a->scale;
  k.eps = a->eps;
  k.num_blocks = (uint32_t)p.num_blocks;
  k.n_seqs = (uint32_t)n;
  k.heads = (uint32_t)heads;
  k.head_dim = (uint32_t)d;
  k.taps = (uint32_t)taps;
  int dev = 0;
  st = stream_device(reinterpret_cast<hipStream_t>(stream), &dev);
  if (st != HKV_OK) return st;
  DeviceScope scope(dev);
  if (scope.err != hipSuccess) return hip_error(scope.err, "selecting the stream's device");
  const int e = hkv::launch_kda(k, a->dtype, stream);
  if (e != 0) return hip_error((hipError_t)e, "launching the KDA step");
  if (trace_on())
    std::fprintf(stderr, "[hkv] hkv_kda_step: layer %d, %d sequences, %lld heads of %lld\n",
                 a->layer, a->n_seqs, (long long)heads, (long long)d);
  return HKV_OK;
}

}  // namespace

extern "C" {

hkv_status hkv_mla_attend_workspace(const hkv_layout* layout, const hkv_mla_attend_args* args,
                                    size_t* bytes) {
  return guarded([&]() -> hkv_status {
    if (!layout || !args || !bytes)
      return set_error(HKV_E_ARG, "layout, args and bytes must not be NULL");
    hkv::AttendArgs k;
    hkv::AttendWorkspace w;
    const hkv_status st = plan_attend(layout, args, args->weights != nullptr, &k, &w);
    if (st == HKV_OK) *bytes = (size_t)w.total;
    return st;
  });
}

hkv_status hkv_mla_attend(const hkv_layout* layout, const void* pool,
                          const hkv_mla_attend_args* args, void* workspace, size_t ws_bytes,
                          void* stream) {
  return guarded([&] { return attend(layout, pool, args, workspace, ws_bytes, stream); });
}

hkv_status hkv_mla_evict_workspace(const hkv_layout* layout, const hkv_mla_evict_args* args,
                                   size_t* bytes) {
  return guarded([&]() -> hkv_status {
    if (!layout || !args || !bytes)
      return set_error(HKV_E_ARG, "layout, args and bytes must not be NULL");
    hkv::EvictArgs k;
    hkv::EvictWorkspace w;
    const hkv_status st = plan_evict(layout, args, &k, &w);
    if (st == HKV_OK) *bytes = (size_t)w.total;
    return st;
  });
}

hkv_status hkv_mla_evict(const hkv_layout* layout, void* pool, const hkv_mla_evict_args* args,
                         void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] { return evict(layout, pool, args, workspace, ws_bytes, stream); });
}

hkv_status hkv_kda_step(const hkv_layout* layout, void* pool, const hkv_kda_step_args* args,
                        void* stream) {
  return guarded([&] { return kda_step(layout, pool, args, stream); });
}

}  // extern "C"
