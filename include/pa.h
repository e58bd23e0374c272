/*
 * pa.h — C ABI of libpa, the hot path of a paged-KV-cache attention engine
 * for one NVIDIA GB300 (sm_103a).
 *
 * Source pages (cited by title and section throughout this library):
 *   [vLLM-wiki] itwiki.kr, "vLLM"
 *   [MRV2]      llm-wiki.hwlabs.dev, "vLLM 0.25 Model Runner V2: 비동기 추론 경로의
 *               재설계와 마이그레이션"
 *   [V1-blog]   techknowgenie.com, "vLLM V1 코어 리팩토링 아키텍처: Zero-overhead C++
 *               스케줄러와 Dynamic Chunked Prefill, PagedAttention v3 심층 분석"
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Ownership: every buffer is allocated and owned by the caller. The library
 *    never allocates, frees or keeps a pointer after the call returns, except
 *    through work that it has enqueued on `stream`.
 *  - Execution: every call enqueues kernels on `stream` (a cudaStream_t passed
 *    as void*; NULL is the legacy default stream) and returns without waiting.
 *    Only pa_get_error() synchronises.
 *  - Host-side argument errors (NULL pointers, negative sizes, misaligned
 *    pointers, inconsistent host mirrors) return PA_ERR_INVALID before any
 *    launch; unsupported shapes return PA_ERR_UNSUPPORTED. A failed launch
 *    returns PA_ERR_CUDA.
 *  - Device-side range errors (a block id, slot or table row that points
 *    outside its buffer) never fault: the kernel skips or clamps the offending
 *    access and sets a sticky bit in a per-device error word, which
 *    pa_get_error() reports and clears. Outputs of a call that raised a device
 *    error are unspecified.
 *  - All pointers marked "dev" are device pointers on the current device; "host"
 *    pointers are read synchronously during the call only.
 *  - The library looks up the device addresses of its own device variables
 *    (the error word, the scratch array of pa_forward_noalloc) once per device,
 *    on first use, and keeps them for the life of the process. They do not
 *    survive cudaDeviceReset: after a reset of a device, make no further call
 *    of this library on that device in the same process.
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* pa_stream_t; /* a cudaStream_t */

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID = 1,       /* bad argument, detected on the host before launch   */
  PA_ERR_UNSUPPORTED = 2,   /* shape or dtype outside the supported set           */
  PA_ERR_CUDA = 3,          /* a CUDA runtime call failed                         */
  PA_ERR_DEVICE_BOUNDS = 4, /* a kernel met an out-of-range index (pa_get_error)  */
  PA_ERR_TIMEOUT = 5        /* a bounded device-side wait gave up (pa_get_error)  */
} pa_status;

typedef enum pa_kv_dtype {
  PA_KV_BF16 = 0,     /* K/V stored as bfloat16                                  */
  PA_KV_FP8_E4M3 = 1  /* K/V stored as OCP FP8 E4M3 codes with per-tensor scales */
} pa_kv_dtype;

/*
 * The physical KV block pool.
 * [vLLM-wiki, "블록 테이블"]: device memory is split ahead of time into equal-size
 * physical blocks of `block_size` tokens; a request's logical blocks map to
 * physical blocks that need not be contiguous.
 *
 * Layout (caller-owned device memory, 16-byte aligned), for K and V separately:
 *     pool[num_blocks][num_kv_heads][block_size][head_dim]
 * so the `block_size` tokens of one (block, kv-head) pair are one contiguous
 * chunk of block_size*head_dim elements. Element type is bf16 (2 bytes) or an
 * E4M3 code (1 byte) according to `dtype`.
 *
 * FP8 [vLLM-wiki, "엔진 구조와 주요 기능", quantisation bullet; V1-blog, "FP8 KV 캐시
 * 양자화의 네이티브 통합"]: a stored code c represents decode(c) * k_scale (or
 * v_scale). Scales are ignored for bf16 pools.
 *
 * Supported: head_dim in {64, 128}; block_size in {16, 32, 64}.
 */
typedef struct pa_kv_pool {
  void* k_pool;          /* dev */
  void* v_pool;          /* dev */
  int32_t num_blocks;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;         /* pa_kv_dtype */
  float k_scale;
  float v_scale;
} pa_kv_pool;

/*
 * pa_write_kv — scatter this step's new keys and values into the pool.
 * [vLLM-wiki, "블록 테이블"] (slot = physical_block * block_size + offset) and
 * [MRV2, "재설계 4"] (slot_mapping is prepared per token before the forward).
 *
 *   k_new, v_new   dev bf16 [T][num_kv_heads][head_dim], 16-byte aligned
 *   slot_mapping   dev int64 [T]; slot < 0 marks a padding token (skipped)
 *   T              number of tokens (0 is a no-op)
 *
 * For token t with s = slot_mapping[t] >= 0: blk = s / block_size,
 * off = s % block_size, and for every kv head h and dim d
 *     K[blk][h][off][d] = k_new[t][h][d]   (and the same for V).
 * bf16 pools copy the bits. FP8 pools store e4m3(float(x) / scale), the
 * quotient correctly rounded in fp32, then rounded to nearest-even with
 * saturation to +-448; NaN stores 0x7F.
 * A slot >= num_blocks*block_size sets PA_ERR_DEVICE_BOUNDS and is skipped.
 * Duplicate slots within one call: which token wins is unspecified.
 */
pa_status pa_write_kv(const pa_kv_pool* pool, const void* k_new, const void* v_new,
                      const int64_t* slot_mapping, int32_t T, pa_stream_t stream);

/*
 * pa_forward_workspace_size — bytes of optional scratch that lets pa_forward
 * split long decode requests across CTAs (split-KV, merged by log-sum-exp).
 * `max_splits` is the largest number of splits the caller wants per request.
 * pa_forward works with any workspace size, including 0 (then each decode
 * request is handled by one CTA per kv head).
 */
size_t pa_forward_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t head_dim,
                                 int32_t max_splits);

/*
 * pa_forward — paged attention over a mixed batch of decode tokens and prefill
 * chunks.
 * [vLLM-wiki, "블록 단위 어텐션 계산", equation for A_ij and o_i]: the softmax runs
 * across every visible key of every block of the request; the result equals
 * ordinary attention, only the memory layout differs.
 * [V1-blog, "고정 예산 기반 청크 분할 알고리즘"] and [vLLM-wiki, "엔진 구조와 주요 기능"
 * unified-scheduler bullet]: one step packs one token per running decode next to
 * prefill chunks.
 * [MRV2, "재설계 4"]: query_start_loc and seq_lens describe the batch.
 *
 *   q                 dev bf16 [T][num_q_heads][head_dim], 16-byte aligned
 *   out               dev bf16 [T][num_q_heads][head_dim], 16-byte aligned
 *   query_start_loc   dev int32 [R+1], qsl[0]=0, non-decreasing, qsl[R]=T
 *   seq_lens          dev int32 [R], all tokens of request r including this
 *                     step's query tokens (whose K/V must already be written)
 *   qsl_host, seq_lens_host
 *                     host mirrors of the two arrays above (same values); used
 *                     to plan grids without a device sync
 *   block_tables      dev int32 [R][max_blocks]: physical block of logical
 *                     block i of request r; entries past ceil(seq_len/B) unread
 *   num_q_heads       Hq; must be a multiple of pool->num_kv_heads. Query head
 *                     h reads kv head h / (Hq / Hkv) (contiguous GQA groups).
 *   scale             softmax scale (e.g. 1/sqrt(head_dim))
 *   causal            1: query j of request r (absolute position
 *                     p = seq_len - q_len + j) sees keys 0..p. 0: every query
 *                     sees keys 0..seq_len-1. A decode query (q_len == 1)
 *                     sees all seq_len keys either way.
 *   workspace         dev scratch of workspace_bytes (may be NULL/0)
 *
 * out[t][h][:] = sum_n softmax_n(scale * q[t][h] . k_n) v_n over the visible
 * keys, computed in fp32 and rounded to bf16 (nearest-even). Rows of requests
 * with q_len == 0 are not touched. Requests may appear in any order.
 * Host checks: qsl_host must be non-decreasing with qsl_host[R] == T, and
 * 1 <= q_len <= seq_len <= max_blocks * block_size for every request with
 * q_len > 0, and a pool with at least one block when any request has
 * q_len > 0; otherwise PA_ERR_INVALID.
 * Device checks: the grids are planned from the host mirrors. A device
 * query_start_loc or seq_lens that disagrees with them so that a request's
 * rows would leave [0, T), or its keys or query tiles would need more CTAs
 * or workspace slots than were planned, sets PA_ERR_DEVICE_BOUNDS; nothing is
 * read or written outside q, out, the pool and the workspace.
 */
pa_status pa_forward(const void* q, void* out, const int32_t* query_start_loc,
                     const int32_t* seq_lens, const int32_t* qsl_host,
                     const int32_t* seq_lens_host, const int32_t* block_tables,
                     int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                     int32_t num_q_heads, const pa_kv_pool* pool, float scale,
                     int32_t causal, void* workspace, size_t workspace_bytes,
                     pa_stream_t stream);

/*
 * pa_forward_shared_prefix — pa_forward for a batch in which groups of decode
 * requests share the physical blocks of a common prefix (parallel sampling,
 * beam candidates, a shared system prompt).
 * [vLLM-wiki, "블록 공유와 쓰기 시 복사"]:
 * the samples of one prompt map the prompt's logical blocks to the same
 * physical blocks (reference-counted, copied on write); only the tails differ.
 * The result is the attention pa_forward computes (the same bounds against
 * exact arithmetic; the fp32 summation order differs): the softmax over the
 * union of the prefix keys and the tail keys is taken in parts, the prefix
 * pieces and the tail splits, merged by log-sum-exp. Each group's prefix K/V
 * is read once for every 64 of its (member, GQA head) rows (four warps share
 * each staged K/V chunk) instead of once per member; any GQA width.
 *
 * Arguments as pa_forward, plus:
 *   num_groups          G, 0 <= G <= 64 (more: PA_ERR_UNSUPPORTED). G == 0
 *                       behaves as pa_forward.
 *   group_first_host    host int32 [G]: group k is the group_size_host[k]
 *   group_size_host     host int32 [G]  consecutive requests from
 *                       group_first_host[k]; groups in increasing order and
 *                       disjoint, within [0, num_reqs); other requests may sit
 *                       before, between and after them
 *   prefix_blocks_host  host int32 [G]: the first prefix_blocks_host[k]
 *                       entries of every member's block-table row are the
 *                       same physical blocks (the caller's contract: the
 *                       prefix is read through the first member's row)
 *   workspace           required: at least pa_forward_workspace_size(R, Hq,
 *                       head_dim, 2) bytes (one prefix piece and one tail
 *                       split per member); more lets the call cut prefixes and
 *                       tails into more pieces that run in parallel
 *
 * Host checks (PA_ERR_INVALID): every member is a decode request (q_len 1)
 * with seq_len > prefix_blocks * block_size, 1 <= prefix_blocks <=
 * max_blocks, groups non-empty and in range, workspace large enough.
 * Requests outside every group, and prefill chunks, are handled exactly as by
 * pa_forward. If members' rows differ on the prefix, the result is
 * unspecified but every block id read is still bounds-checked.
 */
pa_status pa_forward_shared_prefix(const void* q, void* out, const int32_t* query_start_loc,
                                   const int32_t* seq_lens, const int32_t* qsl_host,
                                   const int32_t* seq_lens_host, const int32_t* block_tables,
                                   int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                                   int32_t num_q_heads, const pa_kv_pool* pool, float scale,
                                   int32_t causal, int32_t num_groups,
                                   const int32_t* group_first_host,
                                   const int32_t* group_size_host,
                                   const int32_t* prefix_blocks_host, void* workspace,
                                   size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_prepare_inputs — one step's attention inputs built on the device from
 * per-slot state, so that the host sends only (slot, token count) per request
 * and the block-table diffs.
 * [MRV2, "재설계 1"]: a live request keeps a fixed persistent slot; entry i of
 * the step is slot idx_mapping[i]. [MRV2, "재설계 4"]: query_start_loc,
 * positions, seq_lens and the slot mapping are prepared on the GPU.
 * [vLLM-wiki, "블록 테이블"]: position p lives in logical block p / B at offset
 * p % B; its pool slot is physical_block * B + offset.
 *
 *   num_computed     dev int32 [max_reqs]: tokens of each slot whose K/V are
 *                    stored; read, then advanced by the step's counts
 *   table            dev int32 [max_reqs][max_blocks]: the persistent block
 *                    table (after pa_apply_staged_writes)
 *   idx_mapping      dev int32 [R]: slot of entry i (each slot at most once)
 *   num_scheduled    dev int32 [R]: tokens of entry i this step (>= 0);
 *                    NULL: one token per entry (a decode step)
 *   token_capacity   entries of positions / slot_mapping
 *   query_start_loc  dev int32 [R+1]  out: running sum of num_scheduled
 *   seq_lens         dev int32 [R]    out: num_computed[slot] + num_scheduled
 *   positions        dev int32 [T]    out: the tokens' positions
 *   slot_mapping     dev int64 [T]    out: the tokens' pool slots (input of
 *                                     pa_write_kv)
 *
 * One launch on `stream`. Integer work: exactly the definition above. A slot
 * outside [0, max_reqs), a negative count, a total above token_capacity, a
 * position past the table row or a block outside [0, num_blocks) sets
 * PA_ERR_DEVICE_BOUNDS (read by pa_get_error); such slots are written as -1
 * (pa_write_kv skips them) and nothing is written outside the buffers. A slot
 * listed twice gives unspecified counts. Host checks: PA_ERR_INVALID for
 * negative sizes or NULL buffers that the sizes require.
 */
pa_status pa_prepare_inputs(int32_t* num_computed, int32_t max_reqs, const int32_t* table,
                            int32_t max_blocks, int32_t block_size, int32_t num_blocks,
                            const int32_t* idx_mapping, const int32_t* num_scheduled,
                            int32_t num_reqs, int32_t token_capacity, int32_t* query_start_loc,
                            int32_t* seq_lens, int32_t* positions, int64_t* slot_mapping,
                            pa_stream_t stream);

/*
 * pa_decode_graph_* — several decode steps of the same requests captured once
 * into a CUDA graph and replayed with one launch.
 * [V1-blog, "PagedAttention V3 커널 아키텍처와 하드웨어 레벨 메모리 정렬",
 * multi-step scheduling bullet]: N decode steps (4 to 8, say) run from a CUDA
 * graph without a host round trip per token. [MRV2, "재설계 4"]: graphs are
 * managed explicitly; each captured shape costs capture time and memory.
 *
 * Step s of the graph (s = 0 .. num_steps-1) is exactly this eager sequence:
 *   pa_prepare_inputs(num_computed, ..., idx_mapping, NULL (one token each),
 *                     num_reqs, num_reqs, query_start_loc, seq_lens, positions,
 *                     slot_mapping)
 *   pa_write_kv(pool, k_new + s * R*Hkv*D, v_new + s * R*Hkv*D, slot_mapping, R)
 *   pa_forward(q + s * R*Hq*D, out + s * R*Hq*D, query_start_loc, seq_lens,
 *              {0, 1, .., R}, seq_len_bound_host, block_tables, max_blocks, R, R,
 *              num_q_heads, pool, scale, 1, workspace, workspace_bytes)
 * so every output equals that of the eager calls made with the same bound.
 * The forward plan is fixed at creation from seq_len_bound_host; every launch
 * should keep each request's sequence length (num_computed + 1 at each step)
 * at or below its bound. A length past its bound is either still covered by
 * the plan, with exact results (the persistent GQA decode of pa_forward cuts
 * the device-side lengths into its CTA ranges at every launch, within the
 * workspace's split slots), or refused with PA_ERR_DEVICE_BOUNDS; nothing is
 * ever read out of range. The table must already hold the blocks of every
 * position the steps write; block_tables holds the rows table[idx_mapping[i]].
 *
 * The pool struct, pointers and sizes are read at creation and baked into the
 * graph: the buffers must stay allocated and in place until destroy. The
 * graph object is created (host and driver memory) by create and released by
 * destroy; the library allocates no device memory. Launches of one graph must
 * not overlap (they share the scratch buffers); launch returns without
 * waiting. Errors: PA_ERR_INVALID (NULL or non-positive sizes), the status of
 * the first captured call that fails, PA_ERR_CUDA if capture or instantiation
 * fails.
 */
typedef struct pa_decode_graph pa_decode_graph;

typedef struct {
  const pa_kv_pool* pool;
  float scale;
  int32_t num_q_heads;
  int32_t num_reqs;                    /* R: decode requests, one token per step  */
  int32_t num_steps;                   /* N                                        */
  int32_t* num_computed;               /* dev int32 [max_reqs] (advanced N / launch) */
  int32_t max_reqs;
  const int32_t* table;                /* dev int32 [max_reqs][max_blocks]         */
  int32_t max_blocks;
  const int32_t* idx_mapping;          /* dev int32 [R]                            */
  const int32_t* block_tables;         /* dev int32 [R][max_blocks]                */
  const int32_t* seq_len_bound_host;   /* host int32 [R]                           */
  const void* q;                       /* dev bf16 [N][R][Hq][D]                   */
  const void* k_new;                   /* dev bf16 [N][R][Hkv][D]                  */
  const void* v_new;                   /* dev bf16 [N][R][Hkv][D]                  */
  void* out;                           /* dev bf16 [N][R][Hq][D]                   */
  int32_t* query_start_loc;            /* dev scratch int32 [R+1]                  */
  int32_t* seq_lens;                   /* dev scratch int32 [R]                    */
  int32_t* positions;                  /* dev scratch int32 [R]                    */
  int64_t* slot_mapping;               /* dev scratch int64 [R]                    */
  void* workspace;                     /* as pa_forward (may be NULL / 0)          */
  size_t workspace_bytes;
} pa_decode_graph_desc;

pa_status pa_decode_graph_create(const pa_decode_graph_desc* desc, pa_decode_graph** graph);
pa_status pa_decode_graph_launch(pa_decode_graph* graph, pa_stream_t stream);
void pa_decode_graph_destroy(pa_decode_graph* graph);
/* Kernel launches one pa_decode_graph_launch performs (0 for NULL). */
uint32_t pa_decode_graph_kernels(const pa_decode_graph* graph);

/*
 * pa_apply_staged_writes — apply packed block-table diffs, then gather the
 * rows of this step.
 * [MRV2, "재설계 3: 큰 block table은 staged diff만 보낸다"]: the device copy of the
 * block table is the reference copy; the host records (row, start, values)
 * diffs, uploads them in one small staging buffer, and one kernel applies them;
 * the rows needed this step are then gathered by idx_mapping.
 * [MRV2, "재설계 1"]: a request keeps a fixed persistent slot (row) while live;
 * idx_mapping[i] is the slot of the i-th request of this batch.
 * [MRV2, "재설계 2"]: the staging buffers must not be modified by the caller until
 * the stream has consumed them.
 *
 *   table          dev int32 [max_reqs][max_blocks], updated in place
 *   rows, starts   dev int32 [W]
 *   val_offsets    dev int32 [W+1], non-decreasing from val_offsets[0] >= 0;
 *                  diff w writes len_w = val_offsets[w+1] - val_offsets[w]
 *                  values
 *   vals           dev int32 [val_offsets[W]]
 *   idx_mapping    dev int32 [R]
 *   gathered       dev int32 [R][max_blocks]
 *
 * For w = 0..W-1 in record order: table[rows[w]][starts[w] + k] =
 * vals[val_offsets[w] + k], k < len_w (a later diff overwrites an earlier one
 * on the same cell: last writer wins). Then gathered[i][c] =
 * table[idx_mapping[i]][c] for every c < max_blocks. A diff whose row or
 * column range leaves the table, whose value run leaves [0, val_offsets[W]),
 * or an idx_mapping entry outside
 * [0, max_reqs), sets PA_ERR_DEVICE_BOUNDS and is skipped (gathered row left
 * untouched). W == 0 performs only the gather; R == 0 only the writes.
 */
pa_status pa_apply_staged_writes(int32_t* table, int32_t max_reqs, int32_t max_blocks,
                                 const int32_t* rows, const int32_t* starts,
                                 const int32_t* val_offsets, const int32_t* vals,
                                 int32_t W, const int32_t* idx_mapping, int32_t R,
                                 int32_t* gathered, pa_stream_t stream);

/*
 * pa_copy_blocks — copy whole physical blocks (K and V, every kv head), the
 * device half of copy-on-write.
 * [vLLM-wiki, "블록 공유와 쓰기 시 복사"]: a block shared by several sequences is
 * copied only when one of them must write a new token into it.
 *
 *   src, dst   dev int32 [n]; block src[i] is copied to block dst[i]
 * The dst blocks must be distinct from each other and from every src block
 * (then the copies are order-independent). An id outside [0, num_blocks) sets
 * PA_ERR_DEVICE_BOUNDS and that pair is skipped.
 */
pa_status pa_copy_blocks(const pa_kv_pool* pool, const int32_t* src, const int32_t* dst,
                         int32_t n, pa_stream_t stream);

/*
 * pa_gather_rows — dst row i = src row rows[i], for i < n: the rows a step
 * hands on (each request's last query token, whose output the sampler
 * needs) gathered by index, as [MRV2, "재설계 1"] gathers the persistent
 * batch's rows by idx_mapping.
 *
 *   src        dev, src_rows rows of row_bytes bytes (16-byte aligned)
 *   row_bytes  a positive multiple of 16
 *   rows       dev int32 [n]
 *   dst        dev, n rows of row_bytes bytes (16-byte aligned), not
 *              overlapping src
 * A row index outside [0, src_rows) sets PA_ERR_DEVICE_BOUNDS and that dst
 * row is left unchanged. n == 0 is a no-op. Argument errors: PA_ERR_INVALID.
 */
pa_status pa_gather_rows(const void* src, int64_t src_rows, int64_t row_bytes,
                         const int32_t* rows, int32_t n, void* dst, pa_stream_t stream);

/*
 * The latent path: layers that cache one shared latent vector per token.
 *
 * Such a layer keeps, per token, a latent row c [latent_dim] and one rotary
 * key row k_r [rope_dim]; the key and the value of head h are products of c,
 *     k[h] = [ W_k[h] c ; k_r ],    v[h] = W_v[h] c.
 * Scores and outputs can be taken in two forms that give the same result:
 *   expanded   k and v of every head are made and attended to as usual
 *              (pa_latent_prefill; fewest operations for long chunks);
 *   absorbed   W_k[h]^T moves into the query and W_v[h] behind the output,
 *              so that every head attends straight to the cache, with key
 *              [c ; k_r] and value c (pa_latent_forward; a token's cache is
 *              read once for all heads).
 * The products with W are the caller's. pa_rope turns the queries' rotary
 * part, pa_write_latent turns and stores a step's new rows, pa_read_latent
 * fetches cached rows back for the expanded form.
 */

/*
 * pa_rope — rotary positions. The first rot_dim dims of every head of every
 * token are turned in pairs: pair i of token t by the angle
 * positions[t] * inv_freq[i] (radians),
 *     (x, y) -> factor * (x cos - y sin, y cos + x sin);
 * the dims past rot_dim are copied unchanged.
 *
 *   x, out          dev bf16 [T][num_heads][head_dim], innermost dims
 *                   contiguous, the token and head strides given in elements
 *                   (0 .. 2^38 - 1; x may repeat rows with stride 0, rows of out must
 *                   not overlap). out may be x itself, with the same strides
 *                   (then turned in place); otherwise the two must not overlap.
 *                   A rotary part at the end of a wider head is reached by
 *                   pointing at it.
 *   positions       dev int32 [T], any value
 *   inv_freq        dev fp32 [rot_dim / 2]
 *   rot_dim         even, 0 .. min(head_dim, 256)
 *   layout          PA_ROPE_HALF: pair i is dims (i, i + rot_dim / 2);
 *                   PA_ROPE_INTERLEAVED: dims (2i, 2i + 1)
 *   factor          finite and positive (long-context scalings change inv_freq and this factor)
 *
 * Angles are off by less than 2^-25 of a turn at any position, for frequencies
 * of magnitude up to 256; fp32 arithmetic, one rounding to bf16 (nearest-even). The inverse turn is the same call with
 * negated positions and 1 / factor. Errors: PA_ERR_INVALID (sizes, strides,
 * NULL or misaligned pointers), PA_ERR_UNSUPPORTED (odd rot_dim or above 256,
 * head_dim above 32768, num_heads * head_dim above 2^31).
 */
typedef enum pa_rope_layout { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;

pa_status pa_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                  int64_t out_token_stride, int64_t out_head_stride, const int32_t* positions,
                  int32_t T, int32_t num_heads, int32_t head_dim, const float* inv_freq,
                  int32_t rot_dim, int32_t layout, float factor, pa_stream_t stream);

/*
 * The latent block pool (caller-owned device memory, 16-byte aligned). Blocks,
 * block tables and slots are those of pa_kv_pool; a cell is one token:
 *     latent[num_blocks][block_size][latent_dim]   bf16, or E4M3 codes
 *     rope  [num_blocks][block_size][rope_dim]     bf16
 *     scales[num_blocks][block_size]               fp32, E4M3 pools only
 * A code of token n stands for decode(code) * scales[n]. pa_write_latent stores
 * powers of two, 2^-60 and more; attention takes any scale from 2^-90 to 2^100.
 *
 * Supported: latent_dim in {256, 512}; rope_dim 64; block_size in {16, 32, 64}.
 */
typedef struct pa_latent_pool {
  void* latent;          /* dev */
  void* rope;            /* dev */
  float* scales;         /* dev; NULL for bf16 pools */
  int32_t num_blocks;
  int32_t block_size;
  int32_t latent_dim;
  int32_t rope_dim;
  int32_t dtype;         /* pa_kv_dtype */
} pa_latent_pool;

/*
 * pa_write_latent — scatter this step's latent rows and rotary keys into the
 * pool by slot, as pa_write_kv does for keys and values.
 *
 *   latent        dev bf16 [T][latent_dim], token stride latent_stride
 *                 (elements, a multiple of 8), 16-byte aligned
 *   k_rope        dev bf16 [T][rope_dim], token stride rope_stride
 *   positions     dev int32 [T], inv_freq dev fp32 [rope_dim / 2], layout and
 *                 factor: k_rope is turned as pa_rope does before it is
 *                 stored. Both NULL: stored as it comes.
 *   slot_mapping  dev int64 [T]; slot < 0 marks a padding token (skipped)
 *
 * bf16 pools copy latent's bits. E4M3 pools store, per token,
 *   scale = 2^e, the smallest with max |latent| <= 448 * 2^e over the finite
 *           elements (e >= -60; 1 for a row of zeros),
 *   code  = e4m3(latent / scale), nearest-even, saturating; NaN stores 0x7F,
 * so that decode(code) * scale is exact in bf16 (up to bf16's range).
 * A slot >= num_blocks*block_size sets PA_ERR_DEVICE_BOUNDS and is skipped.
 * Duplicate slots within one call leave the cell unspecified.
 */
pa_status pa_write_latent(const pa_latent_pool* pool, const void* latent, int64_t latent_stride,
                          const void* k_rope, int64_t rope_stride, const int32_t* positions,
                          const float* inv_freq, int32_t layout, float factor,
                          const int64_t* slot_mapping, int32_t T, pa_stream_t stream);

/*
 * pa_read_latent — cached rows of a batch of requests, gathered through their
 * block tables into one ragged array and widened to bf16 (the input of the
 * products that make the expanded keys and values of a context).
 *
 *   block_tables  dev int32 [num_reqs][max_blocks]
 *   kv_start_loc  dev int32 [num_reqs+1], from 0, non-decreasing: request r's
 *                 tokens are rows kv_start_loc[r] .. kv_start_loc[r+1]-1
 *   first         dev int32 [num_reqs]: position of the request's first token
 *                 that is read (NULL: 0), for contexts read in windows
 *   num_tokens    rows of the outputs; rows past kv_start_loc[num_reqs] are
 *                 left as they are
 *   latent_out    dev bf16 [num_tokens][latent_dim], stride latent_stride
 *                 (a multiple of 8), 16-byte aligned
 *   rope_out      dev bf16 [num_tokens][rope_dim], stride rope_stride (even),
 *                 4-byte aligned
 *
 * A position outside the table, a block outside the pool, kv_start_loc[0] != 0
 * or more rows than num_tokens set PA_ERR_DEVICE_BOUNDS; such rows are skipped.
 */
pa_status pa_read_latent(const pa_latent_pool* pool, const int32_t* block_tables,
                         int32_t max_blocks, const int32_t* kv_start_loc, const int32_t* first,
                         int32_t num_reqs, int32_t num_tokens, void* latent_out,
                         int64_t latent_stride, void* rope_out, int64_t rope_stride,
                         pa_stream_t stream);

/*
 * pa_copy_latent_blocks — pa_copy_blocks for a latent pool (latents, rotary
 * parts and scales); the same rules for src and dst.
 */
pa_status pa_copy_latent_blocks(const pa_latent_pool* pool, const int32_t* src,
                                const int32_t* dst, int32_t n, pa_stream_t stream);

/*
 * pa_latent_forward — attention in the absorbed form over the paged latent
 * cache, for a mixed batch of decode tokens and chunks, as pa_forward:
 *   s[t][h][n] = scale * q[t][h] . [c_n ; k_r_n],
 *   out[t][h]  = sum_n softmax_n(s[t][h]) c_n    over the visible keys.
 *
 *   q            dev bf16 [T][num_q_heads][latent_dim + rope_dim], 16-byte
 *                aligned: the absorbed query, then its turned rotary part
 *   out          dev bf16 [T][num_q_heads][latent_dim], 16-byte aligned
 *   query_start_loc, seq_lens, qsl_host, seq_lens_host, block_tables,
 *   max_blocks, num_reqs, num_tokens, causal
 *                as pa_forward (the step's own rows are already written)
 *   num_q_heads  any positive number (all heads read the same cache)
 *   workspace    dev scratch, required: pa_latent_workspace_size bytes serve
 *                every batch; 16-byte aligned. Calls that may run at the same
 *                time (other streams, captured graphs that overlap) need
 *                workspaces of their own.
 *
 * Computed in fp32 and rounded once to bf16; the softmax weights enter the
 * second product rounded to bf16. On E4M3 pools the codes are multiplied as
 * they are: the latent part of a query is taken to 2^-17 of its row's largest
 * element (if that is 2^-119 at least), and a weight times its cell's scale to 2^-9 of itself or 2^-24 of
 * the row's largest such product. Rows of requests with q_len == 0 and rows
 * past query_start_loc[num_reqs] are not touched.
 * Cells past a request's seq_len may hold anything. A NaN or an infinity in a
 * query stays in its own row of out; one in a cell reaches the rows that see it
 * and no others. A cell that a row scores -inf weighs 0 there, which its elements
 * are still multiplied by (NaN where they are not finite); a row that scores
 * every visible cell so is NaN.
 * The work is divided from the device arrays at every launch; the host mirrors
 * only size the launch. A captured call therefore follows device lengths that
 * change between replays, with exact results, as long as query_start_loc
 * stays within num_tokens and each seq_len within max_blocks * block_size.
 * Host checks as pa_forward, PA_ERR_INVALID for a workspace too small, and
 * PA_ERR_UNSUPPORTED for shapes outside pa_latent_pool's and for batches past
 * 32-bit bookkeeping: num_tokens * num_q_heads > 2^31 - 65, or
 * (num_tokens * num_q_heads / 16 + num_reqs) * max_blocks * block_size / 32
 * near 2^31.
 * Device checks: a request whose device entries leave those bounds (or with
 * q_len > seq_len) sets PA_ERR_DEVICE_BOUNDS and is skipped; where the others
 * claim more work than the bound above (a query_start_loc that goes back and
 * forth), all are; a block id outside the pool sets it too. Nothing is read or written outside the
 * buffers.
 */
size_t pa_latent_workspace_size(int32_t num_q_heads, int32_t latent_dim);

pa_status pa_latent_forward(const void* q, void* out, const int32_t* query_start_loc,
                            const int32_t* seq_lens, const int32_t* qsl_host,
                            const int32_t* seq_lens_host, const int32_t* block_tables,
                            int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                            int32_t num_q_heads, const pa_latent_pool* pool, float scale,
                            int32_t causal, void* workspace, size_t workspace_bytes,
                            pa_stream_t stream);

/*
 * pa_latent_prefill — attention in the expanded form: ragged query chunks
 * against keys and values that the caller has made from the latents of each
 * request's whole context (cached tokens, from pa_read_latent, and the
 * chunk's own):
 *   s[i][h][n] = scale * (q[i][h][:nope_dim] . k_nope[n][h]
 *                         + q[i][h][nope_dim:] . k_rope[n]),
 *   out[i][h]  = sum_n softmax_n(s[i][h]) v[n][h]   over the visible keys.
 *
 *   q        dev bf16 [num_tokens][num_heads][nope_dim + rope_dim]
 *   k_nope   dev bf16 [num_kv_tokens][num_heads][nope_dim]
 *   k_rope   dev bf16 [num_kv_tokens][rope_dim], shared by the heads
 *   v        dev bf16 [num_kv_tokens][num_heads][v_dim]
 *            16-byte aligned, innermost dims contiguous, token and head
 *            strides in elements, positive multiples of 8 (k_nope and v may
 *            be the two parts of one projection's output)
 *   out      dev bf16 [num_tokens][num_heads][v_dim], contiguous, 16-byte aligned
 *   query_start_loc, kv_start_loc
 *            dev int32 [num_reqs+1], from 0, non-decreasing; qsl_host and
 *            ksl_host their host mirrors (same values)
 *   causal   1: query j of a request sees keys 0 .. k_len - q_len + j; 0: all
 *            k_len keys. A row without a visible key is zero.
 *
 * Computed in fp32 (the softmax weights enter the second product rounded to
 * bf16), rounded once to bf16. Rows past query_start_loc[num_reqs] are not
 * touched; rows past kv_start_loc[num_reqs] may hold anything. A NaN or an
 * infinity in a query or in a key (and its value) reaches the rows that see it and
 * no others; one in a value whose key is finite reaches those too and may, as
 * NaN (0 times it), reach every row of its request and head. A key that a row
 * scores -inf weighs 0 there, which its value is still multiplied by; a row that
 * scores every visible key so is NaN. Supported: nope_dim 128, rope_dim 64,
 * v_dim 128. Needs no workspace.
 * Host checks: PA_ERR_INVALID (sizes, mirrors that do not end at num_tokens
 * and num_kv_tokens, strides, pointers), PA_ERR_UNSUPPORTED (other dims, more
 * than 32767 requests). Device checks: start arrays that leave the buffers or
 * need more query tiles than the mirrors set PA_ERR_DEVICE_BOUNDS; nothing
 * outside the buffers is read or written.
 */
pa_status pa_latent_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const void* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                            const void* k_rope, int64_t rope_token_stride, const void* v,
                            int64_t v_token_stride, int64_t v_head_stride, void* out,
                            const int32_t* query_start_loc, const int32_t* kv_start_loc,
                            const int32_t* qsl_host, const int32_t* ksl_host, int32_t num_reqs,
                            int32_t num_tokens, int32_t num_kv_tokens, int32_t num_heads,
                            int32_t nope_dim, int32_t rope_dim, int32_t v_dim, float scale,
                            int32_t causal, pa_stream_t stream);

/*
 * pa_get_error — synchronise `stream`, then return and clear the sticky
 * device error word of the current device: PA_ERR_TIMEOUT if a bounded wait
 * gave up, else PA_ERR_DEVICE_BOUNDS if an index was out of range, else
 * PA_OK. Returns PA_ERR_CUDA if the synchronisation itself failed.
 * The word is read and cleared in one atomic exchange (a one-thread kernel on
 * `stream`, counted by pa_kernel_launches), so a bit that a kernel on another
 * stream sets meanwhile is returned by this call or by the next one, never
 * cleared unseen. Not callable during stream capture (it synchronises).
 */
pa_status pa_get_error(pa_stream_t stream);

/* pa_status_string — a static, human-readable name for a status code. */
const char* pa_status_string(pa_status status);

/*
 * pa_forward_noalloc — pa_forward for callers that cannot allocate device
 * memory. The pages have no counterpart of this call.
 *
 * Some callers may not call cudaMalloc (or any allocator) where they run
 * attention: a plugin inside a host runtime that has reserved the device
 * memory through its own pool and gives plugins no allocator, or a serving
 * loop that forbids allocation after start-up because cudaMalloc can
 * synchronise the device. This call takes the same arguments as pa_forward
 * except the workspace: its split-KV scratch comes from a fixed array that
 * the library keeps in device memory, PA_NOALLOC_SCRATCH_BYTES on every GPU
 * that loads the library, held until the process exits.
 *
 *   max_splits   as in pa_forward_workspace_size; the scratch it needs,
 *                pa_forward_workspace_size(num_reqs, num_q_heads, head_dim,
 *                max_splits), must not exceed PA_NOALLOC_SCRATCH_BYTES, else
 *                the call returns PA_ERR_UNSUPPORTED before any launch.
 *                0 uses no scratch (one split per decode request).
 *
 * The call allocates nothing and frees nothing. The first call on each device
 * looks up the array's device address (cudaGetSymbolAddress) and caches it;
 * make that first call before any stream capture. The cached address does not
 * survive cudaDeviceReset (see the conventions above). Every call shares the same
 * array: calls that may run at the same time on the GPU (different streams,
 * or several host threads) race on it and must be serialised by the caller.
 * The array keeps the previous call's contents; nothing needs clearing,
 * because every cell a call reads is written earlier in that call.
 */
#define PA_NOALLOC_SCRATCH_BYTES (16u << 20)

pa_status pa_forward_noalloc(const void* q, void* out, const int32_t* query_start_loc,
                             const int32_t* seq_lens, const int32_t* qsl_host,
                             const int32_t* seq_lens_host, const int32_t* block_tables,
                             int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                             int32_t num_q_heads, const pa_kv_pool* pool, float scale,
                             int32_t causal, int32_t max_splits, pa_stream_t stream);

/*
 * pa_selftest_wait_timeout — diagnostics, not part of the method on the pages.
 * Launches one small kernel that waits on a device barrier which nothing will
 * complete, through the same bounded waits that the kernels of this library
 * use, one after the other. Each gives up after its limit (2 seconds, so about
 * 4 in all), the last records the timeout in the error word, and the kernel
 * returns: afterwards pa_get_error() reports
 * PA_ERR_TIMEOUT. Lets callers and tests check the no-hang error path.
 */
pa_status pa_selftest_wait_timeout(pa_stream_t stream);

/*
 * pa_kernel_launches — number of CUDA kernels this library has launched in
 * this process (all devices, all streams), for launch accounting in
 * benchmarks and tests. Not part of the method on the pages; never fails.
 */
uint64_t pa_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */
