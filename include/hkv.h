/*
 * hkv.h — chunk store/retrieve for hybrid KDA+MLA model caches on MI355X.
 *
 * The library moves a hybrid model's cache between a paged GPU pool (the
 * layout vLLM gives a model whose KDA linear-attention layers keep a
 * recurrent state and whose MLA layers keep per-token latent KV) and
 * contiguous chunk objects, one object per (chunk, object group):
 *
 *   store    : block-table gather, pool pages -> chunk objects;
 *   retrieve : scatter of chunk objects into newly allocated block ids.
 *
 * and runs the operators of a decode step that read and update the pool's
 * pages in place: MLA attention, eviction by attention weight, the KDA step.
 *
 * To the copies pages are opaque bytes: the KDA state (recurrent heads x d x d
 * plus conv (conv_dim, kernel-1)) is one opaque page, as LMCache treats it
 * ("Kimi-Linear" and "Kimi K3" recipes, introduction; "Hybrid Attention
 * Models", Mamba / Linear-Attention Hybrids), so they are exact byte copies.
 *
 * Conventions for every call:
 *   - returns hkv_status: HKV_OK (0) or a negative error code; nothing aborts
 *     or throws; hkv_last_error() gives a message for the calling thread;
 *   - all validation happens on the host, synchronously, before any work is
 *     enqueued (but of the DEVICE tables that the decode step's operators
 *     take, see there); a call that returns an error has enqueued nothing
 *     (except HKV_E_HIP, which reports a failure of the HIP runtime itself);
 *   - "HOST" arrays are read only during the call; "DEVICE" buffers must stay
 *     allocated until the stream has passed the enqueued work;
 *   - work is enqueued on the caller's stream, which is never synchronised.
 *
 * Sizes are bytes unless stated; block ids are int32 in [0, num_blocks).
 */
#ifndef HKV_H
#define HKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t hkv_status;

#define HKV_OK 0
#define HKV_E_ARG (-1)       /* malformed argument (NULL, negative count, bad enum) */
#define HKV_E_COVER (-2)     /* given N is not a multiple of 16 tokens or its MLA page
                                does not cover the KDA state page */
#define HKV_E_CHUNK (-3)     /* strict mode and the chunk minimum is not a multiple of N */
#define HKV_E_BATCH (-4)     /* max_num_batched_tokens outside the allowed range */
#define HKV_E_POOL (-5)      /* the pool holds no whole block (or more than INT32_MAX) */
#define HKV_E_RANGE (-6)     /* a block id outside [0, num_blocks) */
#define HKV_E_ALIAS (-7)     /* a retrieve target id repeated in one call, or two buffers
                                of one call overlap */
#define HKV_E_ALIGN (-8)     /* pool, object or workspace pointer not 16-byte aligned */
#define HKV_E_WORKSPACE (-9) /* workspace NULL or smaller than hkv_workspace_size() */
#define HKV_E_HIP (-10)      /* the HIP runtime reported an error (see hkv_last_error) */
#define HKV_E_CAPTURE (-11)  /* the stream is capturing and the call cannot be captured
                                (see hkv_store_chunks) */

/* One rank's model shapes.  KDA state shapes are PER RANK: heads and conv_dim
 * are already divided by the TP degree, because the KDA state is sharded
 * across TP ranks while the MLA cache is replicated ("Kimi-Linear" recipe,
 * Note; vLLM hybrid KV-cache blog, section 2.1 gives the two state shapes). */
typedef struct hkv_model {
  int32_t n_layers;        /* number of decoder layers, >= 1 */
  const uint8_t* is_mla;   /* HOST [n_layers], model order: 1 = MLA layer, 0 = KDA layer */
  int32_t kda_heads;       /* recurrent state heads per rank */
  int32_t kda_head_dim;    /* d: the recurrent state is heads x d x d */
  int32_t kda_state_bytes; /* bytes per recurrent-state element (4 = fp32) */
  int32_t conv_dim;        /* conv state rows per rank */
  int32_t conv_kernel;     /* conv kernel size; the state keeps kernel-1 columns */
  int32_t conv_bytes;      /* bytes per conv-state element (2 = bf16) */
  int32_t mla_width;       /* values per token per MLA layer (kv_lora_rank + rope dim, 576) */
  int32_t mla_bytes;       /* bytes per MLA value (2 = bf16, 1 = fp8 e4m3) */
} hkv_model;

/* Unified block size N: the smallest multiple of 16 tokens whose MLA page
 * (N x mla_width x mla_bytes) is at least one rank's KDA state page
 * (heads x d x d x state_bytes + conv_dim x (conv_kernel-1) x conv_bytes).
 * Defined in "Hybrid Attention Models", Mamba / Linear-Attention Hybrids,
 * Step 1 (vLLM forces one block size across groups so the attention page
 * covers the state page) and the "Kimi-Linear" recipe, Note (N follows the
 * per-rank state).  A model without KDA layers gets N = 16.
 * align_tokens must be 16 (the only step this library supports; 0 = 16).
 * Errors: HKV_E_ARG (NULL pointers, non-positive shapes, align != 16). */
hkv_status hkv_unified_block_size(const hkv_model* model, int32_t align_tokens,
                                  int64_t* n_out);

/* Everything a layout needs. */
typedef struct hkv_layout_desc {
  hkv_model model;
  int64_t block_size;         /* N in tokens; 0 = derive with the rule above; nonzero
                                 must be a multiple of 16 covering the KDA page
                                 (else HKV_E_COVER) */
  int64_t chunk_min_tokens;   /* >= 1: the chunk size is the smallest multiple of N at or
                                 above it ("Kimi K3" recipe, Why these settings) */
  int32_t strict_chunk_multiple; /* 1: HKV_E_CHUNK unless chunk_min_tokens % N == 0 (the
                                 older rule, "Kimi-Linear" recipe, Why these settings) */
  int32_t path;               /* 0 = path A, shared tensors with the unified padded page
                                 (vLLM hybrid KV-cache blog, section 3.1);
                                 1 = path B, packed per-layer offset + block stride
                                 (same blog, section 3.2) */
  int32_t separate_object_groups; /* 1: KDA and MLA layers go to different objects;
                                 0: one object holds every layer ("Hybrid Attention
                                 Models", Object-group separation) */
  const int32_t* kv_group_of_layer; /* HOST [n_layers] KV-cache group of each layer, ids
                                 0..G-1 all used; NULL = default: the MLA layers form one
                                 group, the KDA layers in model order form
                                 ceil(n_kda/n_mla) contiguous groups of sizes differing
                                 by at most one, larger first (Mooncake K3 blog, "Flat
                                 KV"); KDA groups are numbered before the MLA group */
  uint64_t pool_bytes;        /* bytes of the pool the layout may use */
  int64_t max_num_batched_tokens; /* 0 = skip; else must be >= N, and < 2N unless
                                 object groups are separated (HKV_E_BATCH) ("Kimi-Linear"
                                 recipe, Why these settings; "Hybrid Attention Models",
                                 Step 2) */
  uint64_t tile_bytes;        /* 0 = default (4 KiB); else the largest span one
                                 workgroup copies: a multiple of 4096 up to 1 GiB.  A
                                 tuning knob: results do not depend on it */
  uint32_t max_workgroups;    /* 0 = one workgroup per tile; else the grid is capped at
                                 this many workgroups, each looping over tiles.  A
                                 tuning knob: results do not depend on it */
  int32_t kda_codec;          /* 0 = KDA pages are stored as opaque bytes (default);
                                 1 = INT8 codec of the recurrent state in objects, for
                                 inactive checkpoints (Mooncake K3 blog, Compressed
                                 Checkpoint Storage: per-channel INT8 for the recurrent
                                 state, the conv window at full precision).  A KDA page
                                 is read as the conv state (conv_dim x (kernel-1) x
                                 conv_bytes, a multiple of 16 bytes) followed by the fp32
                                 recurrent state (heads x d x d, d in {16, 32, 64, 128,
                                 256}); in an object it becomes the conv bytes verbatim,
                                 then int8 codes of every row of d values, then one fp32
                                 scale per row.  Per row: s = (largest finite |x|) / 127;
                                 q = round-half-even(x / s) clamped to [-127, 127], and 0
                                 for non-finite x or s == 0 (x / s an IEEE fp32 division);
                                 retrieve writes q * s in fp32, a NaN product (only from an
                                 object the encoder did not write) as 0x7FC00000.  Lossy:
                                 |x - q s| <= s / 2 for finite x.  Else HKV_E_ARG */
} hkv_layout_desc;

typedef struct hkv_layout hkv_layout; /* opaque; its plan is immutable after init; may be
                                         shared by threads.  The first store or retrieve
                                         on a device copies the plan's constant tables
                                         (layer placements and per-chunk work items, about
                                         115 KB at the Kimi-Linear shapes) into that
                                         device's memory, synchronously; they stay there
                                         until hkv_layout_destroy. */

/* Plans a layout.  Path A: every layer uses the unified page P = the largest
 * real page (the MLA page), smaller KDA pages are padded to it; slab s holds
 * the s-th layer of every KV group, pool_offset = s x num_blocks x P,
 * stride P, num_blocks = pool_bytes / (slabs x P).  Path B: inside a group
 * the layers' real pages are packed in model order (running offset), the
 * block stride is the largest group total, num_blocks = pool_bytes /
 * stride.  Object layout: layer-major in model order, then the k blocks of
 * the chunk, real page bytes only, no header; for MLA layers this is an
 * [L_obj][chunk_tokens][mla_width] array.
 * Defined by: the block size N ("Hybrid Attention Models", Mamba /
 * Linear-Attention Hybrids, Step 1; "Kimi-Linear" recipe, Note), the chunk
 * size rule ("Kimi K3" recipe, Why these settings), one block table per KV
 * group (vLLM hybrid KV-cache blog, section 2.2), the two pool layouts (same
 * blog, sections 3.1 and 3.2), the balanced KDA groups (Mooncake K3 blog,
 * "Flat KV") and the separate object groups ("Hybrid Attention Models",
 * Object-group separation).
 * Errors: HKV_E_ARG, HKV_E_COVER, HKV_E_CHUNK, HKV_E_BATCH, HKV_E_POOL.
 * On success *out owns heap memory released by hkv_layout_destroy. */
hkv_status hkv_layout_init(const hkv_layout_desc* desc, hkv_layout** out);

/* Releases a layout and its tables in device memory.  NULL is ignored.  The
 * caller must not destroy a layout while a call that uses it is running on
 * another thread or while work it enqueued has not finished. */
void hkv_layout_destroy(hkv_layout* layout);

typedef struct hkv_layout_info {
  int64_t block_size;        /* N (tokens) */
  int64_t chunk_tokens;      /* C (tokens), a multiple of N */
  int32_t blocks_per_chunk;  /* k = C / N */
  int32_t n_layers;
  int32_t n_kv_groups;       /* G */
  int32_t n_obj_groups;      /* O: 1 or 2 */
  int64_t num_blocks;        /* valid block ids are [0, num_blocks) */
  int32_t path;              /* 0 = A, 1 = B */
  int32_t n_slabs;           /* path A: tensors = largest group size; path B: 0 */
  uint64_t unified_page_bytes; /* path A: P; path B: 0 */
  uint64_t block_stride;     /* bytes between consecutive block ids of one layer */
  uint64_t pool_bytes_used;  /* bytes of the pool the layout addresses */
  uint64_t obj_bytes[2];     /* bytes of one chunk's object of each object group (0 if
                                unused) */
  uint64_t chunk_payload_bytes; /* obj_bytes[0] + obj_bytes[1]: bytes moved per chunk */
  int32_t kda_codec;         /* as in hkv_layout_desc */
} hkv_layout_info;

/* Copies the layout's summary.  Errors: HKV_E_ARG. */
hkv_status hkv_layout_info_get(const hkv_layout* layout, hkv_layout_info* out);

typedef struct hkv_layer_info {
  int32_t is_mla;
  int32_t kv_group;          /* index into the block table's group axis */
  int32_t obj_group;         /* which object of the chunk holds this layer */
  int32_t slot;              /* position inside its KV group (path A: its slab) */
  uint64_t page_bytes;       /* real bytes of one page (copied) */
  uint64_t reserved_bytes;   /* bytes reserved per block (path A: P, padding included) */
  uint64_t pool_offset;      /* byte offset of block 0's page in the pool */
  uint64_t stride;           /* bytes between the pages of consecutive block ids */
  uint64_t obj_offset;       /* byte offset of block j=0's page inside its object; block j
                                sits at obj_offset + j * obj_page_bytes */
  uint64_t obj_page_bytes;   /* bytes one page takes in an object: page_bytes, or the INT8
                                form of a KDA page under the codec */
} hkv_layer_info;

/* Copies one layer's placement.  Errors: HKV_E_ARG (bad layer index). */
hkv_status hkv_layer_info_get(const hkv_layout* layout, int32_t layer, hkv_layer_info* out);

/* A block-table entry that names no page.  With a token budget of 2N or
 * more a scheduler step spans several blocks and only its last block gets a
 * KDA snapshot ("Kimi-Linear" recipe, Why these settings), so a KDA group's
 * table can have holes; an MLA block past a partial chunk's last token has
 * no page either.  Store writes zeros in a null page's place in the object (a
 * missing state reads as zero, as the engine zeroes the initial state of a
 * miss: vLLM hybrid KV-cache blog, section 5.3); retrieve writes nothing for
 * it.  Null ids may repeat within a call. */
#define HKV_NULL_BLOCK (-1)

/* One call's chunks. */
typedef struct hkv_chunk_batch {
  int32_t n_chunks;          /* >= 0; 0 is a no-op */
  const int32_t* block_ids;  /* HOST [n_chunks][G][k]: chunk c's block ids in each KV
                                group (one block table per group, vLLM hybrid KV-cache
                                blog, section 2.2), or HKV_NULL_BLOCK */
  void* const* objects;      /* HOST [n_chunks][O] pointers the GPU can address (device
                                memory, or pinned host memory from hipHostMalloc), each
                                to obj_bytes[o] bytes, 16-byte aligned, pairwise disjoint
                                and disjoint from the pool */
  const int32_t* chunk_tokens; /* HOST [n_chunks] valid tokens per chunk (0..C), or NULL
                                when every chunk is whole.  A partial chunk (a tail
                                registered at a fine boundary: vLLM hybrid KV-cache blog,
                                section 6.3; Mooncake K3 blog, fine-grained partial hits)
                                carries in MLA page j the token rows [j*N, min(t,
                                (j+1)*N)) only; store zeroes the rest of that page's
                                object bytes and retrieve writes only those rows.  KDA
                                pages are whole or null. */
  int32_t engine;            /* HKV_ENGINE_KERNEL (0): the gather/scatter kernels.
                                HKV_ENGINE_DMA (1), retrieve only: the pages go by DMA
                                copies on the stream (hipMemcpyAsync), one per run of
                                pages that are contiguous in both the object and the pool
                                (a path B KV group's pages of one block are one run).
                                For chunk objects in pinned host memory this leaves the
                                host link's other direction and the compute units to a
                                concurrent store (LMCache keeps objects in a pinned host
                                L1: "Kimi-Linear" and "Kimi K3" recipes).  Not for INT8
                                layouts (the codec decodes in the scatter kernel) or
                                stores (they zero-fill object bytes): HKV_E_ARG. */
} hkv_chunk_batch;

#define HKV_ENGINE_KERNEL 0
#define HKV_ENGINE_DMA 1

/* Device workspace bytes needed by a call with up to max_chunks chunks: the
 * call's tables (layer placements, work items, block ids, object addresses,
 * token counts), with room for up to 8 per-class item lists.  A retrieve
 * with null ids or partial chunks whose chunks fall into at most 8 classes
 * (same null entries, same token count) launches once per class over only
 * the work items that write something.  Errors: HKV_E_ARG. */
hkv_status hkv_workspace_size(const hkv_layout* layout, int32_t max_chunks, size_t* bytes);

/* Store (gather): for every chunk c, layer l and block j < k, copies the
 * page_bytes(l) bytes at pool + pool_offset(l) + block_ids[c][g(l)][j] x
 * stride(l) to objects[c][o(l)] + obj_offset(l) + j x obj_page_bytes(l).
 * The source address is the page of a block id in the layer's pool view
 * (vLLM hybrid KV-cache blog, sections 3.1 and 3.2: a layer's pages sit at
 * its offset plus block id times its stride); the destination bytes are the
 * opaque pages of the chunk's object of that layer's object group ("Hybrid
 * Attention Models", Object-group separation; "Kimi-Linear" recipe: the KDA
 * state is one opaque page per block).
 * (obj_page_bytes = page_bytes, except KDA pages under kda_codec = 1, which
 * are written in their INT8 form).  Padding and group slack are never read.
 * The pool is not modified.  Under kda_codec = 1 the first object pointer's
 * memory type (hipPointerGetAttributes) picks the gather: pinned host memory
 * takes a form that writes each row's codes as one run, which the host link
 * carries better; the bytes written are the same either way.
 * pool: DEVICE, 16-byte aligned, pool_bytes_used long.  workspace: DEVICE,
 * 16-byte aligned, ws_bytes >= hkv_workspace_size(n_chunks); it is
 * overwritten and must not be used by another call until the stream passes
 * this one.  stream: a hipStream_t (NULL = the default stream).
 * The call's block ids, object addresses and token counts travel in the
 * kernel arguments when they fit in 3 KiB (up to 96 chunks at the
 * Kimi-Linear shapes), so such a call is a single kernel launch; a larger
 * call first copies them into the workspace from pinned staging on the
 * same stream.
 * Repeated source ids are allowed.  Null ids and partial chunks: see
 * HKV_NULL_BLOCK and hkv_chunk_batch.chunk_tokens.
 * Graph capture: while `stream` is capturing (hipStreamBeginCapture), a call
 * whose tables travel in the kernel arguments is captured as its single
 * launch, and a DMA retrieve as its copies; a replay moves the bytes the
 * buffers hold at replay time.  Any other call returns HKV_E_CAPTURE and
 * enqueues nothing: a larger call (its staged table copy would replay
 * whatever the staging slot holds later), and a layout's first call on a
 * device (it uploads the layout's tables synchronously).  Null ids and
 * partial chunks are then served by one launch over all work items.
 * Errors: HKV_E_ARG (also a chunk_tokens entry outside [0, C]), HKV_E_RANGE
 * (an id neither HKV_NULL_BLOCK nor in [0, num_blocks)), HKV_E_ALIAS (objects
 * overlap each other, the pool or the workspace), HKV_E_ALIGN,
 * HKV_E_WORKSPACE, HKV_E_CAPTURE, HKV_E_HIP (a HIP call failed;
 * hkv_last_error names it). */
hkv_status hkv_store_chunks(const hkv_layout* layout, const void* pool,
                            const hkv_chunk_batch* batch, void* workspace, size_t ws_bytes,
                            void* stream);

/* Retrieve (scatter): the inverse copy, objects -> pages of the given,
 * newly allocated block ids (the engine hands the connector fresh block ids
 * to load a hit into: "Kimi K3" recipe, AMD MI355X notes; the loaded state
 * becomes the request's initial state: vLLM hybrid KV-cache blog, section
 * 5.3; page addresses as for hkv_store_chunks, sections 3.1 and 3.2).  Writes exactly the real page bytes of the
 * addressed pages and nothing else (KDA padding, group slack and every other
 * block are left as they were; a null id writes nothing, and a partial chunk
 * writes only its valid MLA token rows).  Because all groups share one
 * block-id space, every non-null id of the call must be distinct
 * (HKV_E_ALIAS otherwise).
 * Same buffer and capture rules as hkv_store_chunks; objects are not
 * modified.
 * Errors: HKV_E_ARG, HKV_E_RANGE, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_WORKSPACE,
 * HKV_E_CAPTURE, HKV_E_HIP. */
hkv_status hkv_retrieve_chunks(const hkv_layout* layout, void* pool,
                               const hkv_chunk_batch* batch, void* workspace,
                               size_t ws_bytes, void* stream);

#define HKV_OP_STORE 0
#define HKV_OP_RETRIEVE 1

/* For callers that cannot allocate memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): hkv_store_chunks
 * (op = HKV_OP_STORE) or hkv_retrieve_chunks (op = HKV_OP_RETRIEVE) with the
 * same kernels and the same bytes in the pool and objects, but no workspace
 * and no allocation.  It calls no hipMalloc, hipFree, hipHostMalloc or other
 * allocating routine, and uses none of the library's pinned staging.
 *   - The layout's constant tables live in a static device array of the
 *     library, 4 MiB per device (held from the first such call on a device
 *     until the process ends); a layout whose tables are larger (more than
 *     about 500,000 work items per chunk) gets HKV_E_WORKSPACE.
 *   - The array holds several layouts' tables at once, each in a range of
 *     its own (about 117 KB at the Kimi-Linear shapes, so some 35 such
 *     layouts).  A call whose layout's tables are not there copies them in
 *     from the layout's host memory (hipMemcpyAsync from pageable memory,
 *     which the HIP runtime moves through its own staging) and waits for
 *     `stream` to finish; later calls with that layout on that device
 *     enqueue without waiting.  When the array is full, the layout used
 *     least recently is dropped to make room, except layouts that a captured
 *     call has used.  hkv_layout_destroy frees the layout's ranges.
 *   - While `stream` is capturing, a copy-in is refused (HKV_E_CAPTURE,
 *     nothing enqueued): make one call with each layout on the device before
 *     capturing.  A captured call reads its layout's tables when the graph
 *     replays, so that layout stays in the array until it is destroyed (do
 *     not replay the graph after that); when such layouts fill the array, a
 *     call that needs room gets HKV_E_WORKSPACE.
 *   - The call's block ids, object addresses and token counts travel in
 *     kernel arguments: one launch per run of chunks that fits (up to 96
 *     chunks at the Kimi-Linear shapes), so a large call is several launches.
 *   - Every call on a device shares that device's array.  Calls that
 *     overlap on one device (other streams, other threads) race only when
 *     one of them copies a layout in over the range of a layout that the
 *     other is using (an eviction, with more layouts than fit): order such
 *     calls.
 *   - A retrieve with null ids or partial chunks runs one launch over every
 *     work item per run of chunks (no per-class launches); the bytes written
 *     are the same.
 * pool: DEVICE as for hkv_store_chunks (written only by a retrieve).
 * batch: as for hkv_store_chunks; engine must be HKV_ENGINE_KERNEL.
 * Host-side checks keep per-thread buffers between calls, so a call no
 * larger than the thread's earlier ones does not allocate host memory either.
 * Errors: HKV_E_ARG (also a bad op, the DMA engine, or a chunk whose ids and
 * object addresses alone exceed the kernel-argument block), HKV_E_RANGE,
 * HKV_E_ALIAS (objects overlap each other or the pool; repeated retrieve
 * ids), HKV_E_ALIGN, HKV_E_WORKSPACE (tables larger than the static array, or
 * no room beside the layouts that captured calls use), HKV_E_CAPTURE,
 * HKV_E_HIP. */
hkv_status hkv_move_chunks_noalloc(const hkv_layout* layout, int32_t op, void* pool,
                                   const hkv_chunk_batch* batch, void* stream);

/* ------------------------------------------------------------------------
 * The decode step over the pool: operators that read and update the pages
 * in place, for one new token per sequence.
 *
 * Unlike the copies above, their block tables, block ids and lengths are
 * DEVICE arrays, as a decode loop keeps them, so a captured call follows them
 * from replay to replay.  Their contents therefore cannot be checked on the
 * host: a kernel never reads or writes through an id outside the pool or past
 * a table's end, and each call says what becomes of a sequence with such a
 * value.  Everything else is checked on the host before anything is enqueued.
 * The calls allocate nothing, synchronise nothing, enqueue only kernel
 * launches on the caller's stream and may all be captured into a HIP graph.
 * A workspace may be shared by calls and by captured graphs that the stream
 * runs one after another, not by ones that may run at once; nothing in it
 * has to be kept or cleared between calls.  No array of a call may be written
 * by anything else while the call runs.
 * A table holds at most 2^31 - 1 tokens (max_blocks x N; 2^28 for an eviction)
 * and a layer's pages start on 16-byte boundaries (HKV_E_ALIGN for a packed
 * layout where they do not; an eviction takes those too).  What the host plans
 * and the workspaces follow max_blocks, since it does not know the lengths:
 * tables not much wider than the sequences are faster.
 * ------------------------------------------------------------------------ */

#define HKV_BF16 0
#define HKV_FP16 1
#define HKV_FP32 2
#define HKV_E4M3 3 /* OCP fp8 e4m3 (no infinities) */

/* MLA attention of one new token per sequence over one layer's paged latent
 * cache.  A cached row k_t has mla_width values of which the first
 * value_width are also its value v_t (an MLA layer caches the latent and the
 * rotary part as one row: vLLM hybrid KV-cache blog, section 4.2, the
 * (num_blocks, N, 576) view); the query is already multiplied into the
 * latent space, so every head reads the same rows:
 *   s_ht = scale x cache_scale x sum_w q_hw k_tw          (fp32)
 *   lse_h = ln sum_t exp(s_ht),  p_ht = exp(s_ht - lse_h)
 *   out_hv = cache_scale x sum_t p_ht k_tv, v < value_width
 * over the tokens t < seq_lens[s] whose block is not HKV_NULL_BLOCK.  Token t
 * is row t % N of block block_table[s][t / N].  The new token's own row must
 * be in the cache already (seq_lens counts it).
 * A sequence with no such token gets zeros and lse = -infinity. */
typedef struct hkv_mla_attend_args {
  int32_t layer;             /* an MLA layer */
  int32_t n_seqs;            /* 0..65535; 0 is a no-op */
  int32_t n_heads;           /* 1..128 query heads */
  int32_t value_width;       /* a multiple of 16, at most 512 and at most mla_width */
  int32_t dtype;             /* of q and out: HKV_BF16 or HKV_FP16 */
  int32_t cache_dtype;       /* mla_bytes = 2: the same as dtype; 1: HKV_E4M3 */
  int32_t max_blocks;        /* entries of a block_table row, >= 1; n_seqs x max_blocks x N at
                                most 2^36 - 32 tokens */
  float scale;               /* softmax scale */
  float cache_scale;         /* what a cached 1.0 stands for (1 unless e4m3); both and their
                                product are finite */
  const void* q;             /* DEVICE [n_seqs][n_heads][mla_width] */
  int64_t q_seq_stride;      /* elements; multiples of 8, >= 0 */
  int64_t q_head_stride;
  const int32_t* block_table; /* DEVICE [n_seqs][max_blocks] block ids of the layer's KV
                                group, or HKV_NULL_BLOCK; entries past a sequence's end are
                                not read.  A block may appear in several sequences */
  int64_t table_stride;      /* elements between its rows, >= 0 */
  const int32_t* seq_lens;   /* DEVICE [n_seqs] tokens, 0..max_blocks x N */
  void* out;                 /* DEVICE [n_seqs][n_heads][value_width]; rows must not overlap */
  int64_t out_seq_stride;    /* elements; multiples of 8 */
  int64_t out_head_stride;
  float* lse;                /* DEVICE [n_seqs][n_heads], or NULL */
  float* weights;            /* DEVICE [n_seqs][weights_stride], or NULL: weights[s][t] +=
                                sum_h p_ht for t < seq_lens[s] (what hkv_mla_evict reads);
                                other entries are left as they were */
  int64_t weights_stride;    /* elements, >= max_blocks x N */
} hkv_mla_attend_args;

/* Device workspace bytes of a call with these shapes (n_seqs, n_heads,
 * value_width, max_blocks and whether weights is given; pointers are not
 * read).  With weights it holds one fp32 per head and token of the table.
 * Errors: HKV_E_ARG. */
hkv_status hkv_mla_attend_workspace(const hkv_layout* layout, const hkv_mla_attend_args* args,
                                    size_t* bytes);

/* Enqueues the attention (see above).  pool: DEVICE as for hkv_store_chunks,
 * only read.  Needs mla_width a multiple of 32 of at most 576 and mla_bytes 1
 * or 2.  q, out and the workspace are 16-byte aligned, the other arrays by
 * their element; out, lse, weights and the workspace must not overlap any
 * other buffer of the call.  The result of a call depends on its inputs alone
 * (no atomics).  A sequence that names a live block id outside [0,
 * num_blocks) gets NaN in out, lse and its weights; one whose length is
 * outside [0, max_blocks x N] gets NaN in out and lse, and its weights are
 * left as they were.
 * Errors: HKV_E_ARG, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_WORKSPACE, HKV_E_HIP. */
hkv_status hkv_mla_attend(const hkv_layout* layout, const void* pool,
                          const hkv_mla_attend_args* args, void* workspace, size_t ws_bytes,
                          void* stream);

/* Eviction from the MLA cache by accumulated attention weight: cuts every
 * sequence longer than `budget` down to `budget` tokens, in each of the given
 * layers by that layer's own weights, and closes the gaps in place, so that
 * the sequence's first ceil(budget / N) blocks hold what is kept and its other
 * blocks are free.
 * Per layer i and sequence s, of the slots t < seq_lens[s]:
 *   kept:  slots whose position is below `sinks` or at least
 *          next_positions[s] - recent, then those of the largest weights
 *          (NaN counts as the least, below -infinity); ties go to the lowest
 *          slot;
 *   moved: the kept slots t >= budget, in order, into the dropped slots
 *          t < budget, in order: row, weight and position.  No other row
 *          moves, so after a first eviction slots are not ordered by
 *          position; the attention does not depend on the order of its rows.
 * weights_out and positions_out get the kept slots' values for t < budget, and
 * 0 and -1 for budget <= t < seq_lens[s] (a token that is appended there later
 * starts with no weight); shorter sequences' are copied.  Entries past
 * seq_lens[s] are left as they were.  The arrays may be the inputs themselves;
 * where they are not, the same call can be repeated: it finds its inputs
 * unchanged and moves the same rows to the same places.
 * The blocks of a sequence that was cut no longer hold the tokens, or the
 * order, that its prefix hashes and hkv_chunk_keys name.  Store them under keys
 * of their own, never under the prefix's, and give an eviction no block that a
 * prefix cache or another sequence still reads. */
typedef struct hkv_mla_evict_args {
  int32_t n_layers;          /* 1..64 */
  const int32_t* layers;     /* HOST [n_layers] distinct MLA layers of one KV group (they
                                share the block table) */
  int32_t n_seqs;            /* 0..65535, n_layers x n_seqs too; 0 is a no-op */
  int32_t max_blocks;        /* entries of a block_table row, >= 1 */
  int32_t budget;            /* tokens to keep, >= 1 */
  int32_t sinks;             /* >= 0, sinks + recent <= budget */
  int32_t recent;            /* >= 0 */
  const int32_t* block_table; /* DEVICE [n_seqs][max_blocks], as for hkv_mla_attend; the
                                blocks of a sequence belong to it alone */
  int64_t table_stride;      /* elements, >= 0 */
  const int32_t* seq_lens;   /* DEVICE [n_seqs] tokens in the cache, 0..max_blocks x N */
  const int32_t* next_positions; /* DEVICE [n_seqs] position the sequence's next token gets */
  const float* weights;      /* DEVICE [n_layers][n_seqs][max_blocks x N] accumulated weights */
  const int32_t* positions;  /* DEVICE, same shape: the position each slot's token had */
  float* weights_out;        /* DEVICE, same shape and strides: == weights, or disjoint */
  int32_t* positions_out;    /* DEVICE, same shape and strides: == positions, or disjoint */
  int64_t layer_stride;      /* elements between layers and sequences of these four; rows */
  int64_t seq_stride;        /*   must not overlap */
  int32_t* new_lens;         /* DEVICE [n_seqs] or NULL: min(seq_lens[s], budget), or -1 for
                                a sequence that was left as it was (below) */
} hkv_mla_evict_args;

/* Device workspace bytes of a call with these shapes (n_layers, n_seqs,
 * max_blocks, budget; pointers are not read).  Errors: HKV_E_ARG. */
hkv_status hkv_mla_evict_workspace(const hkv_layout* layout, const hkv_mla_evict_args* args,
                                   size_t* bytes);

/* Enqueues the eviction (see above).  Works on rows of any width as opaque
 * bytes.  pool: DEVICE as for hkv_store_chunks; pool and workspace 16-byte
 * aligned.  A sequence whose length is outside [0, max_blocks x N], or whose
 * table holds HKV_NULL_BLOCK, an id outside [0, num_blocks) or a block that
 * the call's tables name twice before its end, keeps its rows where they are:
 * its weights and positions are copied unchanged (as far as its length is
 * valid) and its new_lens entry is -1.
 * Errors: HKV_E_ARG, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_WORKSPACE, HKV_E_HIP. */
hkv_status hkv_mla_evict(const hkv_layout* layout, void* pool, const hkv_mla_evict_args* args,
                         void* workspace, size_t ws_bytes, void* stream);

/* One token's step of a KDA layer, from the state page of block src_blocks[s]
 * to that of dst_blocks[s] (vLLM hybrid KV-cache blog, section 5.3: the
 * retrieved state is the initial state; at a block boundary the next state
 * goes to a new block, so the finished block's page stays as a snapshot).  A
 * page is the conv state (conv_dim, kernel-1), oldest tap first, then the
 * fp32 recurrent state S (heads, d, d), rows = key channels.  conv_dim is
 * 3 x heads x d: the q, k and v channels of every head, in this order.
 *   y      = silu(sum_j conv_weight_cj tap_cj + conv_weight_c,kernel-1 x_c)
 *   q, k   = y's q and k parts over sqrt(sum of squares + eps) per head; q x scale
 *   S'     = diag(exp(log_decay)) S
 *   u      = beta (v - S'^T k)
 *   S      = S' + k u^T,  out = S^T q
 * in fp32; x becomes the conv state's newest tap.
 * A source of HKV_NULL_BLOCK is a state of zeros (a request without a cached
 * prefix); a destination of HKV_NULL_BLOCK is not written.  Source and
 * destination may be the same block. */
typedef struct hkv_kda_step_args {
  int32_t layer;             /* a KDA layer */
  int32_t n_seqs;            /* 0..4096; 0 is a no-op */
  int32_t dtype;             /* of x, conv_weight and out, and the conv state's type:
                                HKV_BF16 or HKV_FP16 (conv_bytes 2), HKV_FP32 (conv_bytes 4) */
  float scale;               /* of q, e.g. d^-1/2 */
  float eps;                 /* >= 0 */
  const void* x;             /* DEVICE [n_seqs][conv_dim] */
  int64_t x_stride;          /* elements, >= 0 */
  const void* conv_weight;   /* DEVICE [conv_dim][conv_kernel] */
  const float* log_decay;    /* DEVICE [n_seqs][heads x d] natural logs (<= 0 to decay) */
  int64_t decay_stride;      /* elements, >= 0 */
  const float* beta;         /* DEVICE [n_seqs][heads] */
  int64_t beta_stride;       /* elements, >= 0 */
  const int32_t* src_blocks; /* DEVICE [n_seqs] */
  const int32_t* dst_blocks; /* DEVICE [n_seqs], may be src_blocks */
  void* out;                 /* DEVICE [n_seqs][heads x d] */
  int64_t out_stride;        /* elements, a multiple of 4, >= heads x d */
} hkv_kda_step_args;

/* Enqueues the step as one kernel, without a workspace (see above).  Needs
 * kda_state_bytes 4, kda_head_dim 16, 32, 64, 128 or 256, conv_kernel 1..8,
 * conv_dim = 3 x heads x d and a conv state of whole 16-byte units (the pages
 * hold plain fp32 states in the pool whether or not kda_codec is set).  pool
 * and out are 16-byte aligned, the other arrays by their element.
 * A sequence with a block id that is neither HKV_NULL_BLOCK nor in [0,
 * num_blocks), or whose destination another sequence of the call reads or
 * writes, gets NaN in out and writes no page.
 * Errors: HKV_E_ARG, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_HIP. */
hkv_status hkv_kda_step(const hkv_layout* layout, void* pool, const hkv_kda_step_args* args,
                        void* stream);

/* ------------------------------------------------------------------------
 * New tokens into the pool: what fills the pages that the decode step reads.
 * A prompt (or what is left of it after a retrieve) runs through
 * hkv_mla_append and hkv_kda_prefill layer by layer; the pages that they leave
 * are what hkv_mla_attend and hkv_kda_step go on from and hkv_store_chunks
 * stores.  The rules of the decode step hold here too: tables, ids and lengths
 * are DEVICE arrays, everything else is checked on the host, the calls only
 * enqueue kernel launches and may be captured.
 *
 * The tokens of a call's sequences lie one after another in its rows:
 * sequence s has rows seq_starts[s] .. seq_starts[s+1] - 1.  The starts must
 * not decrease.  Rows before the first sequence and behind the last (a padded
 * batch) are not written, and what they hold does not matter.
 * ------------------------------------------------------------------------ */

/* Appends tokens to one layer's paged latent cache, and rotates their queries.
 * Of a token's new row c (mla_width values, an MLA layer's joint projection of
 * latent and rotary part):
 *   columns w < latent_width:  c_w / sqrt(mean_{w < latent_width} c_w^2 + eps)
 *                              x norm_weight_w   (norm_weight NULL: c_w itself)
 *   the last rotary_dim columns, by pairs (a, b):  (a cos - b sin, a sin + b cos)
 *   columns between them: c_w itself
 * in fp32, each divided by cache_scale and rounded once to the cache's type.
 * Pair j is columns (2j, 2j+1) of the rotary part, or (j, j + rotary_dim/2)
 * with rotary_halves; its cos and sin are cos_sin[position][j] and
 * cos_sin[position][rotary_dim/2 + j].  Token i of sequence s, counted from 0,
 * goes to slot t = seq_lens[s] - (its new tokens) + i, i.e. row t % N of block
 * block_table[s][t / N], where hkv_mla_attend reads it; its position is its own
 * (after an eviction slots and positions differ).  A token whose block is
 * HKV_NULL_BLOCK is not stored.
 * Queries: the rotary parts q_in go to q_out (fp32, rounded once to dtype),
 * which may be q_in itself or the last columns of hkv_mla_attend's q. */
typedef struct hkv_mla_append_args {
  int32_t layer;             /* an MLA layer */
  int32_t n_seqs;            /* 0..65535; 0 is a no-op */
  int32_t n_tokens;          /* rows of kv, 0..2^20 */
  int32_t n_heads;           /* 0..128 query heads; 0: no queries */
  int32_t dtype;             /* of kv, norm_weight and the queries: HKV_BF16 or HKV_FP16 */
  int32_t cache_dtype;       /* mla_bytes = 2: the same as dtype; 1: HKV_E4M3 */
  int32_t latent_width;      /* a multiple of 8, 0..mla_width - rotary_dim */
  int32_t rotary_dim;        /* a multiple of 16, 0..mla_width; 0: no rotation */
  int32_t rotary_halves;     /* 0 or 1: which columns are pairs (above) */
  int32_t n_positions;       /* rows of cos_sin */
  int32_t max_blocks;        /* entries of a block_table row, >= 1 */
  float eps;                 /* >= 0 */
  float cache_scale;         /* what a cached 1.0 stands for (1 unless e4m3); finite, > 0 */
  const void* kv;            /* DEVICE [n_tokens][mla_width] */
  int64_t kv_stride;         /* elements, a multiple of 8, >= 0 */
  const void* norm_weight;   /* DEVICE [latent_width], or NULL */
  const float* cos_sin;      /* DEVICE [n_positions][rotary_dim] */
  const int32_t* positions;  /* DEVICE [n_tokens] (may be NULL without rotation) */
  const int32_t* seq_starts; /* DEVICE [n_seqs + 1], or NULL: one token per sequence
                                (n_tokens = n_seqs) */
  const int32_t* seq_lens;   /* DEVICE [n_seqs] tokens in the cache, the new ones counted */
  const int32_t* block_table; /* DEVICE [n_seqs][max_blocks], as for hkv_mla_attend; only the
                                entries of the new tokens are read */
  int64_t table_stride;      /* elements, >= 0 */
  const void* q_in;          /* DEVICE [n_tokens][n_heads][rotary_dim] */
  int64_t q_in_token_stride; /* elements, multiples of 8, >= 0, as the next three */
  int64_t q_in_head_stride;
  void* q_out;               /* DEVICE, same shape; == q_in with its strides, or disjoint */
  int64_t q_out_token_stride;
  int64_t q_out_head_stride;
} hkv_mla_append_args;

/* Enqueues the append as one kernel, without a workspace (see above).  pool:
 * DEVICE as for hkv_store_chunks.  Needs mla_width a multiple of 16 of at most
 * 1024 and mla_bytes 1 or 2.  pool, kv, norm_weight, cos_sin, q_in and q_out are
 * 16-byte aligned, the other arrays by their element.  In an e4m3 cache a value
 * beyond +-448 x cache_scale becomes +-448, NaN stays NaN.
 * A token whose sequence's length is outside [its new tokens, max_blocks x N],
 * or whose block id is not in [0, num_blocks), is not stored; one whose position
 * is outside [0, n_positions) gets NaN in its rotary columns and queries.  No
 * slot of the pool may be named by two tokens of a call: it would hold parts of
 * either.
 * Errors: HKV_E_ARG, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_HIP. */
hkv_status hkv_mla_append(const hkv_layout* layout, void* pool, const hkv_mla_append_args* args,
                          void* stream);

/* hkv_kda_step for many tokens of each sequence: the same conv, norms and
 * recurrence (above), token after token, from the state page of block
 * src_blocks[s], which covers the sequence's first positions[s] tokens, to the
 * pages of the sequence's own blocks: the state after a token of position p goes
 * to block block_table[s][p / N] if p is the last position of its block
 * ((p + 1) % N = 0, a snapshot of the block boundary as a store wants it: vLLM
 * hybrid KV-cache blog, section 7, mamba_cache_mode=align) or the sequence's
 * last new token.  A source of HKV_NULL_BLOCK is a state of zeros; an entry of
 * HKV_NULL_BLOCK is not written (snapshots that are not kept).  The source may
 * be one of the sequence's own blocks.  A sequence without new tokens reads and
 * writes nothing.
 * Sums, norms, decays and states are fp32, with the hardware's exponential and
 * reciprocals in SiLU, decays and norms: a decay of e^-x is off by up to about
 * 6e-8 (1 + x) of itself.  Longer runs of heads of 128 with conv_kernel 4 in bf16
 * or fp16 are computed in chunks of up to 64 tokens, whose products take each
 * operand as two fp16 terms (22 bits): a chunk adds to a column of the state an
 * error of up to about 1e-6 of the largest value that it, or the values v that it
 * takes in, had in the chunk and the one before, which fades as the state does.
 * The bound is the column's: rows far below its largest value (those of key
 * channels near zero) keep fewer bits of their own.  In chunks a NaN or an
 * infinity may also reach outputs of its head up to 63 rows before it. */
typedef struct hkv_kda_prefill_args {
  int32_t layer;             /* a KDA layer */
  int32_t n_seqs;            /* 0..4096; 0 is a no-op */
  int32_t n_tokens;          /* rows of x and out, 0..2^20 */
  int32_t max_seq_tokens;    /* no sequence has more new tokens; plans the call */
  int32_t max_blocks;        /* entries of a block_table row, >= 1 */
  int32_t dtype;             /* as for hkv_kda_step */
  float scale;               /* of q, e.g. d^-1/2 */
  float eps;                 /* >= 0 */
  const void* x;             /* DEVICE [n_tokens][conv_dim] */
  int64_t x_stride;          /* elements, >= 0 */
  const void* conv_weight;   /* DEVICE [conv_dim][conv_kernel] */
  const float* log_decay;    /* DEVICE [n_tokens][heads x d] natural logs, <= 0 (a positive one
                                counts as 0); -infinity forgets */
  int64_t decay_stride;      /* elements, >= 0 */
  const float* beta;         /* DEVICE [n_tokens][heads], in [0, 2] */
  int64_t beta_stride;       /* elements, >= 0 */
  const int32_t* seq_starts; /* DEVICE [n_seqs + 1] */
  const int32_t* positions;  /* DEVICE [n_seqs] position of the sequence's first new token */
  const int32_t* src_blocks; /* DEVICE [n_seqs] */
  const int32_t* block_table; /* DEVICE [n_seqs][max_blocks] block ids of the layer's KV group;
                                only the entries of the new tokens are read */
  int64_t table_stride;      /* elements, >= 0 */
  void* out;                 /* DEVICE [n_tokens][heads x d] */
  int64_t out_stride;        /* elements, a multiple of 4, >= heads x d */
} hkv_kda_prefill_args;

/* Device workspace bytes of a call with these shapes (n_seqs, max_blocks,
 * table_stride, n_tokens, max_seq_tokens, dtype; pointers are not read).  In chunks
 * it is mostly 141 KiB for each head of each of the C = n_tokens / 64 + n_tokens / N +
 * 2 n_seqs chunks that there may be (N: tokens of a block), about 2.2 KB a token and
 * head for long runs; 8 bytes for each of the pool's blocks where n_tokens / N is over 24.
 * Errors: HKV_E_ARG (also where C x heads is over 2^23 - 1 in chunks, or n_seqs x heads
 * over 2^20). */
hkv_status hkv_kda_prefill_workspace(const hkv_layout* layout, const hkv_kda_prefill_args* args,
                                     size_t* bytes);

/* Enqueues the prefill (see above).  Needs of the layout what hkv_kda_step
 * needs; pool, out and workspace are 16-byte aligned, the other arrays by their
 * element.  The result of a call depends on its inputs alone (no atomics but
 * on integers, whose order does not matter).
 * A sequence whose position is negative, that has more tokens than
 * max_seq_tokens or than its table's max_blocks x N - positions[s], that names
 * a block id which is neither HKV_NULL_BLOCK nor in [0, num_blocks), or a block
 * to be written that its table names twice or another sequence of the call
 * reads or writes, gets NaN in its rows of out and writes no page.  One whose
 * starts decrease or leave [0, n_tokens] is left as it was.
 * Errors: HKV_E_ARG, HKV_E_ALIAS, HKV_E_ALIGN, HKV_E_WORKSPACE, HKV_E_HIP. */
hkv_status hkv_kda_prefill(const hkv_layout* layout, void* pool, const hkv_kda_prefill_args* args,
                           void* workspace, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Object identity.  Cached pages are byte-opaque, so an entry must never be
 * read back by an engine whose object format differs: other attention
 * backends or kernel block sizes ("Kimi-Linear", "Kimi K3" recipes and
 * "Hybrid Attention Models", Caveats).  Objects are told apart by cache
 * group, prefix hash and parallel configuration (Mooncake K3 blog, vLLM x
 * Mooncake: hybrid cache reuse across instances).
 *
 * All hashing uses mix64, the output function of SplitMix64 (Steele, Lea and
 * Flood, OOPSLA 2014):
 *   mix64(z): z ^= z >> 30; z *= 0xBF58476D1CE4E5B9; z ^= z >> 27;
 *             z *= 0x94D049BB133111EB; z ^= z >> 31.
 * and GAMMA = 0x9E3779B97F4A7C15.  All arithmetic is modulo 2^64.
 * ------------------------------------------------------------------------ */

/* 64-bit fingerprint of the chunk-object format: it changes whenever the
 * bytes of an object would mean something else, and only then.  It folds,
 * with f = mix64(f ^ w) from f = GAMMA, the words: 1 (format version), N,
 * k, n_layers, kda_heads, kda_head_dim, kda_state_bytes, conv_dim,
 * conv_kernel, conv_bytes, mla_width, mla_bytes, n_obj_groups, kda_codec, and
 * per layer in model order is_mla | obj_group << 1 | obj_page_bytes << 8.  The pool path,
 * pool size, KV grouping and tuning knobs do not enter it: they do not change
 * object bytes, so objects stored from a path A pool can be retrieved into a
 * path B pool of the same model.  Errors: HKV_E_ARG. */
hkv_status hkv_layout_fingerprint(const hkv_layout* layout, uint64_t* out);

/* Chained prefix hashes and object keys for one request (vLLM hybrid
 * KV-cache blog, section 6.3: hashes are computed per hash block and each
 * folds in the previous one, so the i-th hash fingerprints the whole prefix;
 * a coarse block's hash is the hash of its last fine sub-block).
 *
 *   tokens            HOST [n_tokens] token ids of the request, in order;
 *   hash_block_tokens h: a divisor of N (0 = N);
 *   root              H_0, e.g. 0 or the hash a parent prefix ended on;
 *   rank_tag          the caller's parallel configuration (e.g. tp_size << 32
 *                     | tp_rank), mixed into every key;
 *   prefix_hashes_out HOST [n_tokens / h] or NULL: H_1 .. H_(n_tokens/h);
 *   keys_out          HOST [n_chunks][O] or NULL; n_chunks = n_tokens / C
 *                     (whole chunks only; a trailing partial chunk has none),
 *                     at most max_chunks are written;
 *   n_chunks_out      the number of whole chunks (may exceed max_chunks).
 *
 * Definitions (t_j = tokens[(i-1)*h + j], j = 0..h-1, as uint32):
 *   content_i = fold of c = mix64(c ^ (t_j | j << 32)) over j from c = GAMMA
 *   H_i       = mix64((H_{i-1} ^ content_i) + GAMMA)
 *   prefix(c) = H_{(c+1) C / h}                       (the chunk's last fine block)
 *   key(c, o) = mix64(mix64(fingerprint ^ rank_tag) ^ (prefix(c) + (o+1) GAMMA))
 * Errors: HKV_E_ARG (NULL tokens with n_tokens > 0, h not dividing N,
 * negative counts). */
hkv_status hkv_chunk_keys(const hkv_layout* layout, const int32_t* tokens, int64_t n_tokens,
                          int32_t hash_block_tokens, uint64_t root, uint64_t rank_tag,
                          uint64_t* prefix_hashes_out, uint64_t* keys_out, int32_t max_chunks,
                          int64_t* n_chunks_out);

/* Message for the calling thread's last non-OK status ("" if none).  The
 * pointer stays valid until the thread's next hkv_* call. */
const char* hkv_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* HKV_H */
