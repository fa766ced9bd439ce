/*
 * pkv_decode.h -- paged decode attention over a block-pool KV cache (GB300, sm_103a).
 *
 * What the library computes
 * -------------------------
 * Single-step and few-query decode attention over a paged KV cache, the read
 * described on the mlx-bun pages ("@mlx-bun/inference 0.0.0-stage -> 1.0.0",
 * package/src/kernels/attention/paged.ts: ``paged_attention_partial``,
 * ``paged_attention_affine_partial`` and ``paged_attention_merge`` behind
 * ``pagedAttentionView(...).attend(q, scale, mask)``; the 4-bit decode of
 * kernels/attention/kvq4-decode.ts; the few-query causal rule of
 * kernels/attention/multi-query.ts). For sequence b, query row i < N and query
 * head h:
 *
 *     kv    = h / (HQ / HK)                      consecutive heads share a KV head
 *     key t is visible iff t <= len_b - N + i    (len_b counts the N new rows)
 *                     and, with a sliding window W, t > len_b - N + i - W
 *     K[t]  = k_pool[block_tables[b][t / BS]][kv][t % BS][:]
 *     affine pages: K[t][d] = scale[t][d/64] * code[t][d] + bias[t][d/64]
 *     e4m3 pages:   K[t][d] = scale[block of t][kv] * code[t][d]
 *     out[b][h][i] = softmax_t(scale * <q, K[t]>) . V[t]       rounded to bf16
 *
 * The work is split along the sequence into partitions; each partition keeps an
 * f32 online-softmax state (running max, normaliser, unnormalised output) and
 * a merge pass combines partitions by log-sum-exp. Each K/V row is read from
 * HBM once and serves every query head of its KV head (GQA reuse).
 *
 * Data layout (row-major, all device memory unless stated otherwise)
 * -----------------------------------------------------------------
 *   q             bf16  [num_seqs, num_q_heads, n_query, head_dim]
 *   k_pool,v_pool bits=16: bf16 [num_blocks, num_kv_heads, block_size, W]
 *                 bits=4/8: uint32 words [num_blocks, num_kv_heads, block_size,
 *                 W*bits/32]; code d of a row sits in word d/(32/bits) at
 *                 bit offset (d % (32/bits))*bits (lowest bits first).
 *                 W is head_dim for K and v_head_dim for V.
 *   k_scales, k_biases, v_scales, v_biases
 *                 bf16 [num_blocks, num_kv_heads, block_size, W/64]
 *                 (affine pages only; NULL for bf16 pages). Dim d uses group d/64.
 *                 These are the layouts of the pages' BlockPool
 *                 (state/paged/cache.ts): every plane [numBlocks, H, blockSize, width].
 *   e4m3 pages    (bits = 8, group_size = PKV_GROUP_BLOCK) k_pool, v_pool: one byte per
 *                 value, an e4m3 code (4 exponent and 3 fraction bits, bias 7, largest
 *                 448, no infinities) [num_blocks, num_kv_heads, block_size, W];
 *                 k_scales, v_scales: f32 [num_blocks, num_kv_heads], >= 0 and finite, one
 *                 for the block's rows of a KV head; k_biases, v_biases unused (NULL).
 *                 A row at or past seq_len may hold any byte. No page of the reference
 *                 has this format; it is the 8-bit float cache of other servers.
 *   block_tables  int32 [num_seqs, max_blocks_per_seq]: logical page -> physical block.
 *   seq_lens      int32 [num_seqs]: cached rows per sequence, including the n_query
 *                 new ones.
 *   out           bf16  [num_seqs, num_q_heads, n_query, v_head_dim]
 *
 * Ownership: every pointer is borrowed; the library frees nothing and keeps no
 * pointer after a call returns (except a pkv_step handle, which keeps the pointers
 * it was created with until it is destroyed). Calls are asynchronous on the given stream
 * (a cudaStream_t passed as void*; NULL = the legacy default stream) and make
 * no allocation and no host synchronisation, so they can be captured in a
 * CUDA graph. Stream order holds as usual: the partial pass (unless its
 * partitions merge in clusters of several CTAs per SM outside a host-driven step
 * that reads its inputs from host memory) and the merge pass are launched as
 * programmatic dependents of the previous work on the stream (their CTAs may be
 * placed while that work finishes), and they touch no global memory before that
 * work has completed.
 *
 * Errors: host-side argument checks happen before any CUDA call and return a
 * negative PKV_ERR_* code without launching anything. Problems that only the
 * device can see (a block-table entry outside [0, num_blocks), a seq_len
 * below n_query or above max_blocks_per_seq*block_size) never trap: the
 * offending rows are skipped (bad block) or the sequence's outputs are written
 * as zeros (bad length), and a PKV_DEVERR_* bit is OR-ed into *error_flag when
 * error_flag is not NULL. Rows at or past seq_len in a sequence's last page
 * are never used, whatever they hold.
 */
#ifndef PKV_DECODE_H
#define PKV_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side return codes. */
#define PKV_OK 0
#define PKV_ERR_NULL_POINTER (-1)        /* a required pointer is NULL */
#define PKV_ERR_MISALIGNED (-2)          /* a device pointer is not 16-byte aligned */
#define PKV_ERR_BAD_LAYOUT (-3)          /* unsupported bits / group_size / head dims / block_size */
#define PKV_ERR_BAD_PARAMS (-4)          /* bad num_seqs, heads, n_query, table width or partition size */
#define PKV_ERR_UNSUPPORTED_SHAPE (-5)   /* no kernel for these head dims with (num_q_heads/num_kv_heads)*n_query rows */
#define PKV_ERR_WORKSPACE_TOO_SMALL (-6) /* workspace NULL or smaller than pkv_plan.workspace_bytes */
#define PKV_ERR_CUDA (-7)                /* a CUDA runtime or driver call failed */
#define PKV_ERR_SCRATCH_TOO_SMALL (-8)   /* no-alloc entry: partition states larger than its static scratch */

/* Size of the static device scratch behind pkv_paged_decode_attention_no_alloc. */
#define PKV_STATIC_SCRATCH_BYTES (16u << 20)

/* Device-side error bits, OR-ed into *error_flag. */
#define PKV_DEVERR_BAD_BLOCK 1   /* a referenced block id outside [0, num_blocks): its rows were skipped */
#define PKV_DEVERR_BAD_SEQ_LEN 2 /* seq_len < n_query or > max_blocks_per_seq*block_size: outputs zeroed */
#define PKV_DEVERR_TIMEOUT 4     /* an internal pipeline wait gave up (after about a second by
                                    default, see pkv_set_wait_limit_ns); the outputs of that call
                                    are then unspecified */

/* pkv_pool_layout.group_size of e4m3 pages (with bits = 8): one f32 scale per block and KV head. */
#define PKV_GROUP_BLOCK (-1)

/* Pool layout descriptor (the pages' PagedAttentionStorage: blockSize, headDim,
 * vHeadDim, quantization {bits, groupSize}).
 * Head dims with a kernel (key/value; the host rejects the rest), each with up to 64
 * query rows per KV head ((num_q_heads / num_kv_heads) * n_query, the pages' limit for
 * the few-query kernel, kernels/attention/multi-query.ts):
 *   equal dims: 64, 128, 256 (bf16) and 128, 256 (affine);
 *   bf16 192/128, 256/128 and 128/256; affine 256/128 and 128/256;
 *   e4m3 pages: every pair of the bf16 ones. */
typedef struct pkv_pool_layout {
  int32_t num_blocks;   /* blocks in the pool, > 0 */
  int32_t num_kv_heads; /* HK, > 0 */
  int32_t block_size;   /* BS: rows per block; a multiple of the chunk the kernels stage (16 rows
                           bf16, 32 affine and e4m3), or 8 (bf16) / 8 or 16 (others) rows, a chunk then
                           spanning several blocks: such pools run partitions (not the balanced
                           schedule), and neither the CUDA-core contraction nor the fused
                           append-and-attend call takes them (PKV_ERR_UNSUPPORTED_SHAPE) */
  int32_t head_dim;     /* D: key (and query) head dim */
  int32_t bits;         /* 16 = bf16 pages; 4 or 8 = affine codes; 8 = e4m3 codes with group_size -1 */
  int32_t group_size;   /* affine group: 64; PKV_GROUP_BLOCK (-1) with bits = 8: e4m3 pages
                           (ignored for bf16) */
  int32_t v_head_dim;   /* Dv: value (and output) head dim; 0 = head_dim */
} pkv_pool_layout;

/* Per-call decode parameters. */
typedef struct pkv_decode_params {
  int32_t num_seqs;           /* B, > 0 */
  int32_t num_q_heads;        /* HQ, a multiple of num_kv_heads; num_seqs * HQ * n_query < 2^31 */
  int32_t n_query;            /* N >= 1 new query rows per sequence */
  int32_t max_blocks_per_seq; /* row stride of block_tables, > 0 */
  int32_t partition_tokens;   /* rows per partition: 0 = chosen from lengths and SM count;
                                 otherwise rounded up to the chunk rows (16 bf16, 32 affine).
                                 A value >= max_blocks_per_seq*block_size gives one partition. */
  int32_t window;             /* sliding window W in rows, 0 = none: query i then sees only keys
                                 t with len-N+i-W < t <= len-N+i (the W most recent positions,
                                 its own included), as the pages' causal mask with a window
                                 size (kernels/attention/masks.ts, createCausalMask). Reads
                                 start at the 32-row boundary at or below the lowest visible
                                 row, so up to 31 rows below the window are read and masked:
                                 their block-table entries must be valid and their values
                                 finite, as for any row below len; rows further below are
                                 never read */
  int32_t contraction;        /* how the dot products and the weighted value sums run:
                                 PKV_CONTRACTION_AUTO (0, the library's choice per shape),
                                 PKV_CONTRACTION_TENSOR (1, warp-level tensor-core MMA) or
                                 PKV_CONTRACTION_CUDA_CORE (2, per-lane f32 FMAs with warp-shuffle
                                 reductions, the form of the pages' direct paged kernel,
                                 kernels/attention/paged.ts; bf16 pages with equal key/value head
                                 dims and at most 4 query rows per KV head, else
                                 PKV_ERR_UNSUPPORTED_SHAPE) */
  int32_t schedule;           /* how the rows are split over the CTAs, when partition_tokens = 0:
                                 PKV_SCHEDULE_AUTO (0): balanced for 4-bit pages, and for e4m3
                                 pages with more than 8 query rows per KV head, rows *
                                 (head_dim + v_head_dim) > 2048, a table of more than
                                 8192 cache rows and enough sequences and heads that
                                 each has few of the GPU's runs, where the plan
                                 would otherwise write partition states to the workspace, else
                                 partitions;
                                 PKV_SCHEDULE_PARTITIONS (1): fixed-size partitions of every
                                 (sequence, KV head);
                                 PKV_SCHEDULE_BALANCED (2): balanced wherever it is available.
                                 Balanced: one wave of CTAs, each of whose page groups reads an
                                 equal run of the list of all (sequence, KV head, chunk)
                                 triples, whatever the lengths; a run's state per (sequence, KV
                                 head) goes to the workspace and the merge pass combines them.
                                 Available for up to 256 sequences, the tensor-core contraction
                                 and the unfused entry points (the fused append-and-attend call
                                 runs partitions). Ignored when partition_tokens > 0. */
} pkv_decode_params;

#define PKV_CONTRACTION_AUTO 0
#define PKV_CONTRACTION_TENSOR 1
#define PKV_CONTRACTION_CUDA_CORE 2

#define PKV_SCHEDULE_AUTO 0
#define PKV_SCHEDULE_PARTITIONS 1
#define PKV_SCHEDULE_BALANCED 2

/* How a call will be carried out. */
typedef struct pkv_plan {
  int32_t partition_tokens; /* resolved rows per partition */
  int32_t max_partitions;   /* partitions per (sequence, KV head) in the grid and the workspace: those
                               of the longest admissible sequence, or with a window those that tile
                               window + n_query - 1 rows from a base rounded down to a multiple of 32
                               rows (at most window + n_query + 30 rows) */
  int32_t chunk_rows;       /* rows staged per pipeline step */
  int32_t sm_count;         /* SM count the plan was made for */
  int32_t threads_per_cta;  /* partial-kernel CTA size */
  int32_t smem_bytes;       /* partial-kernel dynamic shared memory */
  int32_t merge_in_cluster; /* 1: the partitions of each (sequence, KV head) form one thread-block
                               cluster and merge through distributed shared memory inside the
                               partial kernel (2..16 partitions on a grid of at most one wave) */
  int32_t contraction;      /* the contraction the call runs: PKV_CONTRACTION_TENSOR or
                               PKV_CONTRACTION_CUDA_CORE */
  size_t workspace_bytes;   /* device scratch for the partition states; 0 with one partition
                               or with merge_in_cluster; with balanced = 1, enough for either
                               schedule (the fused call runs partitions) */
  int32_t balanced;         /* 1: the balanced schedule (pkv_decode_params.schedule); then
                               partition_tokens, max_partitions and merge_in_cluster describe the
                               partitions the fused call would run */
} pkv_plan;

/* Makes the plan for (layout, params) on a GPU with sm_count SMs. Pure host
 * code, no CUDA call. Returns PKV_OK or a PKV_ERR_* code. */
int pkv_make_plan(const pkv_pool_layout* layout, const pkv_decode_params* params, int32_t sm_count,
                  pkv_plan* plan);

/* pkv_make_plan for the current CUDA device (reads its SM count). */
int pkv_plan_for_current_device(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                pkv_plan* plan);

/* Paged decode attention: partial pass (and merge pass when there is more than
 * one partition), asynchronous on `stream`.
 *   scale            softmax scale applied to <q, K> (e.g. 1/sqrt(head_dim))
 *   workspace        device scratch of at least plan.workspace_bytes (may be NULL
 *                    when that is 0); the caller owns it; its contents need no
 *                    initialisation and are overwritten.
 *   error_flag       optional device int32 that receives PKV_DEVERR_* bits; the
 *                    library only ORs into it, the caller clears it.
 * Returns PKV_OK once the kernels are enqueued, or a PKV_ERR_* code. */
int pkv_paged_decode_attention(const pkv_pool_layout* layout, const pkv_decode_params* params,
                               const void* q, const void* k_pool, const void* v_pool,
                               const void* k_scales, const void* k_biases, const void* v_scales,
                               const void* v_biases, const int32_t* block_tables,
                               const int32_t* seq_lens, float scale, void* out, void* workspace,
                               size_t workspace_bytes, int32_t* error_flag, void* stream);

/* The two passes of pkv_paged_decode_attention, for callers that schedule them
 * apart (for example to combine partition states computed elsewhere, or to time
 * the partial pass alone). pkv_paged_decode_partial takes the same arguments
 * and enqueues only the partial pass: with one partition, or when the plan merges
 * in a cluster, it writes the final `out`; otherwise it writes each partition's
 * state (running max in log2 units, normaliser, unnormalised output, all f32)
 * into `workspace`. pkv_merge_partitions then enqueues the log-sum-exp merge of
 * those states into `out` for the same layout and params (it does nothing when
 * the plan needs no merge pass).
 * Returns as pkv_paged_decode_attention. */
int pkv_paged_decode_partial(const pkv_pool_layout* layout, const pkv_decode_params* params, const void* q,
                             const void* k_pool, const void* v_pool, const void* k_scales,
                             const void* k_biases, const void* v_scales, const void* v_biases,
                             const int32_t* block_tables, const int32_t* seq_lens, float scale, void* out,
                             void* workspace, size_t workspace_bytes, int32_t* error_flag, void* stream);

int pkv_merge_partitions(const pkv_pool_layout* layout, const pkv_decode_params* params,
                         const int32_t* seq_lens, const void* workspace, size_t workspace_bytes, void* out,
                         int32_t* error_flag, void* stream);

/* One decode step driven from host memory, as a host-side serving loop runs it
 * (and what the end-to-end figure of bench.py times). The step's inputs (q,
 * seq_lens, changed block tables and, for the fused step, the new K/V rows) sit
 * packed in a host block in_host of in_bytes bytes, laid out as their device
 * counterparts in in_dev; the device pointers q, block_tables, seq_lens, k_new,
 * v_new may point into in_dev. On `stream` the call enqueues the decode
 * (pkv_paged_decode_append_attention when k_new and v_new are given, else
 * pkv_paged_decode_attention, the pools then only read) with the step's data
 * moving as follows:
 *   - in_host page-locked and mapped into the device's address space (the default
 *     for cudaHostAlloc / pinned memory on a GB300), with in_host and in_dev
 *     16-byte aligned: the kernels read every input that lies in in_dev's range
 *     directly from in_host, over NVLink-C2C, and in_dev is not written. The
 *     block must hold the step's final values when the call is made: a grid of
 *     one CTA per SM may read q, seq_lens and the block tables from it before the
 *     previous kernel on the stream has finished;
 *   - otherwise: one cudaMemcpyAsync of the block into in_dev first (synchronised
 *     by the runtime when in_host is pageable); in_bytes = 0 copies nothing;
 *   - out_host such mapped memory (16-byte aligned): the kernels write the bf16
 *     output to it as well as to `out`; other host memory gets a cudaMemcpyAsync
 *     of `out` after the decode; NULL: nothing.
 * The kernels reach mapped host memory with ordinary loads and stores; the
 * copy engine's start-up latency would be far larger than the transfer of a few
 * KB. All other arguments are those of the two decode calls; a failed copy
 * returns PKV_ERR_CUDA. */
int pkv_paged_decode_attention_host(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                    const void* in_host, void* in_dev, size_t in_bytes, void* out_host,
                                    const void* q, const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                    void* k_scales, void* k_biases, void* v_scales, void* v_biases,
                                    const int32_t* block_tables, const int32_t* seq_lens, float scale, void* out,
                                    void* workspace, size_t workspace_bytes, int32_t* error_flag, void* stream);

/* A prepared host-driven step: the arguments of pkv_paged_decode_attention_host
 * checked, planned and resolved into kernel parameters and TMA descriptors once,
 * so that each step costs the host only its launches (and copies, if any). The step keeps
 * every pointer it is given: the buffers must outlive it and stay at their
 * addresses (a resized pool or workspace needs a new step), and the device that
 * was current at creation must be current when it runs. The handle lives in host
 * memory (the one host allocation of this library); no device memory is
 * allocated.
 *   pkv_step_create   arguments as pkv_paged_decode_attention_host, plus the
 *                     handle's address; returns PKV_OK or a PKV_ERR_* code
 *                     (nothing is created then)
 *   pkv_step_run      enqueues the step on the stream given at creation, moving
 *                     its data as pkv_paged_decode_attention_host does
 *   pkv_step_destroy  frees the handle (NULL is allowed); it does not wait for
 *                     work in flight, which keeps using the caller's buffers */
typedef struct pkv_step pkv_step;

int pkv_step_create(const pkv_pool_layout* layout, const pkv_decode_params* params, const void* in_host, void* in_dev,
                    size_t in_bytes, void* out_host, const void* q, const void* k_new, const void* v_new,
                    void* k_pool, void* v_pool, void* k_scales, void* k_biases, void* v_scales, void* v_biases,
                    const int32_t* block_tables, const int32_t* seq_lens, float scale, void* out, void* workspace,
                    size_t workspace_bytes, int32_t* error_flag, void* stream, pkv_step** step);
int pkv_step_run(pkv_step* step);
void pkv_step_destroy(pkv_step* step);

/* pkv_paged_decode_attention for callers that cannot allocate device memory.
 * The pages have no counterpart of this entry point.
 *
 * Some callers cannot call cudaMalloc: runtimes whose device memory is owned by
 * their own allocator, which reserves every byte up front and forbids other
 * allocations, and plugins that are handed only the tensors of one call. They
 * cannot provide the workspace the main entry point needs. This entry point
 * needs none. It keeps the f32 partition states in a file-scope static device
 * array of PKV_STATIC_SCRATCH_BYTES (16 MiB), which every GPU that loads the
 * library holds until the process exits. It calls no cudaMalloc, cudaFree or
 * allocating library routine. The caller still passes every input and `out`.
 *
 * Arguments and results are those of pkv_paged_decode_attention, without the
 * workspace. With partition_tokens = 0 the library picks the partition size as
 * usual and coarsens it until the states fit (one partition needs no scratch).
 * A caller-fixed partition_tokens whose states would exceed the scratch is
 * rejected with PKV_ERR_SCRATCH_TOO_SMALL.
 *
 * Set-up: the first call on each device looks up the scratch's device address
 * (cudaGetSymbolAddress, with that device current) and caches it, keyed on the
 * device's current context; a call after a device reset (which makes a new
 * context and loads the module again) looks it up anew. Make the first call on a
 * device, and the first after a reset, before any stream capture on it.
 *
 * Sharing: every call on a device uses the same scratch, which keeps the last
 * call's contents; nothing in it needs to start at zero. Calls whose kernels
 * overlap on the GPU (different streams, or concurrent host threads) race on
 * the scratch and must be ordered by the caller. */
int pkv_paged_decode_attention_no_alloc(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                        const void* q, const void* k_pool, const void* v_pool,
                                        const void* k_scales, const void* k_biases, const void* v_scales,
                                        const void* v_biases, const int32_t* block_tables,
                                        const int32_t* seq_lens, float scale, void* out, int32_t* error_flag,
                                        void* stream);

/* Write side: appends each sequence's n_new new K and V rows into its pages at
 * cache positions seq_lens[b] .. seq_lens[b] + n_new - 1 (position t goes to block
 * block_tables[b][t / block_size], row t % block_size), the pages'
 * PagedKVCache.append / BlockPool.writeBlock (state/paged/cache.ts). Blocks must
 * already be in the tables; allocating them is the caller's.
 *   k_new, v_new  bf16 [num_seqs, num_kv_heads, n_new, head_dim / v_head_dim],
 *                 16-byte aligned
 *   seq_lens      rows held BEFORE the append (the caller then adds n_new)
 * bf16 pages are copied. Affine pages are quantised per row and 64-dim group
 * (the pages do not give the quantiser's formula; this is the min/max reading,
 * every step in f32):
 *     scale = bf16((max - min) / (2^bits - 1)), bias = bf16(min),
 *     code  = clamp(round_half_even((x - bias) / scale), 0, 2^bits - 1)
 *             (0 when the stored scale is 0),
 * codes packed lowest bits first. Bad block ids skip their row and set
 * PKV_DEVERR_BAD_BLOCK; seq_lens[b] + n_new above max_blocks_per_seq*block_size
 * sets PKV_DEVERR_BAD_SEQ_LEN and writes nothing for that sequence.
 * e4m3 pages: per touched block, KV head and plane, with a the largest magnitude of the
 * block's new rows and s its scale (0 when the block holds no earlier row, whatever the
 * scale plane says there),
 *     s' = max(s, 2^e), e the smallest integer >= -126 with a <= 448 * 2^e (0 if a = 0),
 *     new rows:     code = e4m3(x / s')             nearest even (0 when s' = 0)
 *     earlier rows: code = e4m3(code * (s / s'))    when s' > s
 * and s' is stored. Between powers of two the second line is exact but for values that
 * fall below the type's normal range, so growing a scale costs the earlier rows nothing
 * more. A block that receives rows must belong to one sequence only. Values must be
 * finite.
 * Layouts: every (bits, head dims) pair the decode has a kernel for.
 * Asynchronous on `stream`. */
int pkv_paged_append(const pkv_pool_layout* layout, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t n_new,
                     const void* k_new, const void* v_new, const int32_t* block_tables, const int32_t* seq_lens,
                     void* k_pool, void* v_pool, void* k_scales, void* k_biases, void* v_scales, void* v_biases,
                     int32_t* error_flag, void* stream);

/* One decode step with its write: appends each sequence's N = n_query new K and
 * V rows into their pages, then attends over the cache that holds them, in the
 * same launches as pkv_paged_decode_attention. This is the pages' appendDecode
 * (PagedKVCache.appendDecode: append, then read the paged view of the grown
 * cache, "@mlx-bun/inference 0.0.0-stage -> 1.0.0", state/paged/cache.ts).
 *   k_new, v_new  bf16 [num_seqs, num_kv_heads, n_query, head_dim / v_head_dim], 16-byte
 *                 aligned: the K and V rows of the step's query tokens
 *   seq_lens      rows held AFTER the append, as for pkv_paged_decode_attention:
 *                 the new rows go to cache positions seq_lens[b] - n_query ..
 *                 seq_lens[b] - 1, whose blocks must already be in the tables
 * Every other argument is that of pkv_paged_decode_attention; k_pool, v_pool and,
 * for affine pages, the scale and bias planes are written. The rows written and
 * the output are bit for bit those of pkv_paged_append (with seq_lens - n_query)
 * followed by pkv_paged_decode_attention with the same plan. Each new row is
 * written by the CTA whose partition holds it, before that CTA reads the
 * partition, so no second launch and no re-read of the rows from another CTA is
 * needed. Blocks shared by several sequences must not receive new rows (the
 * caller copies them first). A row whose block id is bad is neither written nor
 * read and sets PKV_DEVERR_BAD_BLOCK.
 * e4m3 pages are refused (PKV_ERR_UNSUPPORTED_SHAPE): a new row may rescale its whole
 * block, which may span chunks that other CTAs read. Call pkv_paged_append, then the decode. */
int pkv_paged_decode_append_attention(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                      const void* q, const void* k_new, const void* v_new, void* k_pool,
                                      void* v_pool, void* k_scales, void* k_biases, void* v_scales,
                                      void* v_biases, const int32_t* block_tables, const int32_t* seq_lens,
                                      float scale, void* out, void* workspace, size_t workspace_bytes,
                                      int32_t* error_flag, void* stream);

/* Sparse decode attention: each (sequence, KV head) attends over top_k blocks of its cache,
 * chosen for the step's queries by a score that reads 4 * head_dim bytes per block instead
 * of the block. The reference has no counterpart of it.
 *
 * Block bounds. k_bounds, bf16 [num_blocks, num_kv_heads, 2, head_dim], 16-byte aligned,
 * holds for each block and KV head the elementwise smallest (row 0) and largest (row 1) of
 * its stored keys, rounded outward to bf16. The caller owns the plane; it needs no initial
 * values, and pkv_update_block_bounds keeps it after each append.
 *
 * Score of block j for the query rows r of a KV head (its REP heads times n_query):
 *     score_j = max_r sum_d max(q_rd * lo_jd, q_rd * hi_jd),
 * the largest product any key of the block could have with any of the rows.
 *
 * Choice. With nb = ceil(len / block_size) blocks held: all of them when nb <= top_k, else
 * the first_blocks first, the last_blocks last and, of those between, the best-scored, in
 * all top_k. Blocks are compared as by exact sums, ties going to the lower block: f32 sums
 * decide where their error cannot matter, sums of 48 bits of exact products elsewhere, so the
 * choice does not depend on the order of a sum (while |q|_1 * max|bound| is within f32's
 * range). A query row whose sum is NaN counts as the lowest, like a sum of -infinity: the
 * other rows score the block.
 *
 * The softmax then runs over the chosen rows alone, the causal rule among the n_query newest
 * rows included. window must be 0 and num_seqs * num_kv_heads at most 65535; the layouts and
 * query-row limits are those of the decode. last_blocks must cover the n_query newest rows
 * however full the last block is: (last_blocks - 1) * block_size >= n_query - 1. */
typedef struct pkv_sparse_params {
  int32_t top_k;        /* blocks per (sequence, KV head), > 0 */
  int32_t first_blocks; /* taken at the start of the sequence, >= 0 */
  int32_t last_blocks;  /* taken at its end, >= 1; first_blocks + last_blocks <= top_k */
} pkv_sparse_params;

typedef struct pkv_sparse_plan {
  pkv_plan attention;     /* of the decode over a choice of top_k blocks: num_seqs * num_kv_heads
                             sequences of one KV head; its workspace_bytes are what
                             pkv_selected_decode_attention needs */
  size_t select_bytes;    /* workspace of pkv_select_blocks (0 when the table holds no more than top_k blocks) */
  size_t workspace_bytes; /* workspace of pkv_sparse_decode_attention, which plans for no more
                             blocks than the table holds */
} pkv_sparse_plan;

/* Plans as pkv_make_plan and pkv_plan_for_current_device do. */
int pkv_make_sparse_plan(const pkv_pool_layout* layout, const pkv_decode_params* params,
                         const pkv_sparse_params* sparse, int32_t sm_count, pkv_sparse_plan* plan);
int pkv_sparse_plan_for_current_device(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                       const pkv_sparse_params* sparse, pkv_sparse_plan* plan);

/* Brings the bounds of each sequence's blocks up to date after an append.
 *   seq_lens  rows held, the new ones included
 *   n_new     the last n_new rows of each sequence are new (all of them where it holds
 *             fewer): blocks whose rows are all new get fresh bounds, a block that held
 *             rows before has its bounds widened by the new ones. e4m3 pages, whose earlier
 *             rows an append may have rescaled, have every touched block read whole.
 * A call with n_new of at least every length rebuilds all bounds. k_scales and k_biases as
 * for the decode. Keys must be finite. Bounds of other blocks stay as they were. Rows that a
 * sequence gives up (its length falls back within a block) stay in that block's bounds, which
 * then bound its keys less tightly, until a rebuild. Bad block
 * ids and lengths (outside [0, max_blocks_per_seq*block_size]) are skipped and flagged as
 * by pkv_paged_append. Blocks that receive rows must belong to one sequence only.
 * Asynchronous on `stream`. */
int pkv_update_block_bounds(const pkv_pool_layout* layout, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t n_new,
                            const void* k_pool, const void* k_scales, const void* k_biases,
                            const int32_t* block_tables, const int32_t* seq_lens, void* k_bounds,
                            int32_t* error_flag, void* stream);

/* The choice alone.
 *   blocks         int32 [num_seqs, num_kv_heads, top_k]: the chosen blocks' places in the
 *                  sequence, ascending, -1 past the last (NULL: not wanted)
 *   chosen_tables  int32 [num_seqs, num_kv_heads, top_k]: block_tables entry * num_kv_heads +
 *                  KV head of each, the block's number in the pool seen as num_blocks *
 *                  num_kv_heads blocks of one head (-1 past the last, and for a bad block id)
 *   chosen_lens    int32 [num_seqs, num_kv_heads]: rows of the chosen blocks (0 for a bad length)
 *   workspace      plan.select_bytes
 * A seq_len below n_query or above the table flags PKV_DEVERR_BAD_SEQ_LEN. A bad block id
 * scores lowest and is flagged. */
int pkv_select_blocks(const pkv_pool_layout* layout, const pkv_decode_params* params, const pkv_sparse_params* sparse,
                      const void* q, const void* k_bounds, const int32_t* block_tables, const int32_t* seq_lens,
                      int32_t* blocks, int32_t* chosen_tables, int32_t* chosen_lens, void* workspace,
                      size_t workspace_bytes, int32_t* error_flag, void* stream);

/* The attention alone, over a choice made by pkv_select_blocks (or one of the caller's own
 * in the same form: any blocks of that KV head, in any order, the same one more than once if
 * wanted; chosen_lens rows of them are read, and the last n_query of those count as the
 * sequence's newest). Workspace: plan.attention.workspace_bytes. Other arguments and errors as
 * pkv_paged_decode_attention. */
int pkv_selected_decode_attention(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                  const pkv_sparse_params* sparse, const void* q, const void* k_pool,
                                  const void* v_pool, const void* k_scales, const void* k_biases,
                                  const void* v_scales, const void* v_biases, const int32_t* chosen_tables,
                                  const int32_t* chosen_lens, float scale, void* out, void* workspace,
                                  size_t workspace_bytes, int32_t* error_flag, void* stream);

/* Choice and attention. `blocks` as pkv_select_blocks (may be NULL). Workspace:
 * plan.workspace_bytes; calls that overlap on the GPU need one each. */
int pkv_sparse_decode_attention(const pkv_pool_layout* layout, const pkv_decode_params* params,
                                const pkv_sparse_params* sparse, const void* q, const void* k_pool,
                                const void* v_pool, const void* k_scales, const void* k_biases, const void* v_scales,
                                const void* v_biases, const void* k_bounds, const int32_t* block_tables,
                                const int32_t* seq_lens, float scale, int32_t* blocks, void* out, void* workspace,
                                size_t workspace_bytes, int32_t* error_flag, void* stream);

/* Norm and rotation: what turns a projection's query and key heads into the ones that
 * attention takes, in one pass over them. The reference's attention takes finished heads;
 * it has no counterpart of these calls. For each row x of D = head_dim values, in f32 with one rounding to
 * bf16 at the end:
 *     y = x / sqrt(mean(x^2) + eps) * (weight + weight_offset)    where the weight is given
 *     (y_a, y_b) -> amplitude * (y_a cos w - y_b sin w, y_b cos w + y_a sin w)
 * for the pairs (a, b) of the first rot_dims dims, w = position * inv_freq[i] for pair i.
 * Dims from rot_dims on do not turn. Angles are reduced exactly: any int32 position, with an
 * error below 2^-21 for |inv_freq| < 2 (finite frequencies; larger ones lose as many bits).
 * The squares of a row must sum within f32's range. */
#define PKV_PAIRS_HALVES 0    /* pair i is (i, i + rot_dims/2) */
#define PKV_PAIRS_ADJACENT 1  /* pair i is (2i, 2i + 1) */

/* Which axis of a position with several (time, height, width, ...) turns which frequency. */
#define PKV_SECTIONS_BLOCKS 0 /* the first sections[0] by axis 0, the next sections[1] by axis 1, ... */
#define PKV_SECTIONS_CYCLE 1  /* frequency i by axis a = i % num_axes while i < num_axes * sections[a],
                                 else by axis 0 */

#define PKV_MAX_AXES 4

typedef struct pkv_rotation {
  int32_t head_dim;      /* D: 64, 128, 192 or 256 */
  int32_t rot_dims;      /* dims that turn: a multiple of 8, 8 .. head_dim */
  int32_t pairing;       /* PKV_PAIRS_* */
  int32_t num_axes;      /* 1 .. PKV_MAX_AXES */
  int32_t section_order; /* PKV_SECTIONS_* (num_axes > 1) */
  int32_t sections[PKV_MAX_AXES]; /* frequencies of each axis, >= 0, rot_dims/2 in all (num_axes > 1); with
                                     PKV_SECTIONS_CYCLE each axis must find its count below rot_dims/2 */
  int32_t weight_f32;    /* norm weights are f32, else bf16 */
  float eps;             /* >= 0 */
  float weight_offset;   /* 1 for weights stored less one, else 0 */
  float amplitude;       /* factor on cos and sin, usually 1 */
} pkv_rotation;

/* Head h of token j of sequence b begins at element b*seq + j*token + h*head; a row's values are
 * contiguous. Multiples of 8, >= 0; an output's rows must not overlap. Packed tokens
 * (tokens_per_seq = 0) are counted through by `token` alone. */
typedef struct pkv_row_strides {
  int64_t seq, token, head;
} pkv_row_strides;

/* Norm and rotation alone.
 *   q, k              bf16 rows of num_q_heads and num_kv_heads heads of num_seqs * tokens_per_seq
 *                     tokens, 16-byte aligned (num_kv_heads = 0: no keys, k and k_out NULL)
 *   q_weight, k_weight [head_dim], NULL: no norm of the queries or the keys
 *   positions         int32 [num_axes][num_seqs * tokens_per_seq]
 *   inv_freq          f32 [rot_dims/2]
 *   q_out, k_out      bf16; may be q and k with the same strides
 * Asynchronous on `stream`. No tokens: nothing is launched. */
int pkv_norm_rotate(const pkv_rotation* rotation, int32_t num_seqs, int32_t tokens_per_seq, int32_t num_q_heads,
                    int32_t num_kv_heads, const void* q, const pkv_row_strides* q_strides, const void* k,
                    const pkv_row_strides* k_strides, const void* q_weight, const void* k_weight,
                    const int32_t* positions, const float* inv_freq, void* q_out,
                    const pkv_row_strides* q_out_strides, void* k_out, const pkv_row_strides* k_out_strides,
                    void* stream);

/* The same with the write: queries go to q_out, keys and values into their pages. What the
 * pages then hold is bit for bit what pkv_norm_rotate followed by pkv_paged_append writes.
 *   num_tokens        new tokens of all sequences
 *   tokens_per_seq    tokens of each (num_tokens = num_seqs * tokens_per_seq), or 0: packed, and
 *                     sequence b's are query_starts[b] .. query_starts[b+1] - 1
 *   query_starts      int32 [num_seqs + 1], not falling, within 0 .. num_tokens (packed; else unused).
 *                     Tokens outside [query_starts[0], query_starts[num_seqs]) are left alone, their
 *                     q_out rows too. A sequence may have none.
 *   v                 bf16 rows of v_head_dim values
 *   positions         as above ([num_axes][num_tokens]), or NULL with one axis: the rows'
 *                     places in the cache, seq_lens[b] + 0, 1, ...
 *   seq_lens          rows held BEFORE the write
 * Layouts, pools, planes, bad block ids and bad lengths (no row of that sequence is
 * written) as pkv_paged_append; starts that fall or leave 0 .. num_tokens set
 * PKV_DEVERR_BAD_SEQ_LEN. Queries are normed and rotated whatever becomes of their sequence's
 * rows, except where their starts are bad. A block that receives rows must belong to one sequence only. */
int pkv_norm_rotate_append(const pkv_pool_layout* layout, const pkv_rotation* rotation, int32_t num_seqs,
                           int32_t num_tokens, int32_t tokens_per_seq, int32_t num_q_heads,
                           int32_t max_blocks_per_seq, const void* q, const pkv_row_strides* q_strides, const void* k,
                           const pkv_row_strides* k_strides, const void* v, const pkv_row_strides* v_strides,
                           const void* q_weight, const void* k_weight, const int32_t* positions,
                           const float* inv_freq, const int32_t* query_starts, const int32_t* block_tables,
                           const int32_t* seq_lens, void* k_pool, void* v_pool, void* k_scales, void* k_biases,
                           void* v_scales, void* v_biases, void* q_out, const pkv_row_strides* q_out_strides,
                           int32_t* error_flag, void* stream);

/* Prompt attention: many new tokens of each sequence over the pages that hold them and the
 * rows before them, as many query rows as there are (the decode calls stop at 64 per KV head).
 * The queries of all sequences are packed: sequence b's n = query_starts[b+1] - query_starts[b]
 * tokens are its newest, and its token i sees
 *     keys t <= seq_lens[b] - n + i   and, with a window W, t > seq_lens[b] - n + i - W.
 * Everything else is as for pkv_paged_decode_attention. The reference leaves prompts to its
 * framework's own attention over gathered rows; it has no counterpart of this call. */
typedef struct pkv_prefill_params {
  int32_t num_seqs;           /* B, 1 .. 65535 */
  int32_t num_tokens;         /* tokens in q, >= 0 */
  int32_t num_q_heads;        /* HQ, a multiple of num_kv_heads, at most 64 per KV head */
  int32_t max_blocks_per_seq; /* row stride of block_tables, > 0 */
  int32_t window;             /* sliding window in rows, 0 = none */
  int32_t splits;             /* CTAs that share the keys of one tile of queries: 0 = chosen from the
                                 tokens, the table's width and the SM count, 1 .. 64 */
  int32_t reading;            /* how pages of codes are read (bf16 pages: ignored):
                                 PKV_READING_VALUES (2): a pass before the attention writes 16-bit
                                 values of all rows that any query sees to the workspace, bf16 of
                                 e4m3 pages, fp16 of affine ones (with a power of two for each
                                 (sequence, KV head) and plane; values below 2^-39 of the
                                 largest are lost, as are parts of a query row, and weights
                                 below 2^-32 of a row's largest);
                                 PKV_READING_DIRECT (1): e4m3 pages alone: every CTA turns the codes it
                                 needs into bf16;
                                 PKV_READING_AUTO (0): direct for e4m3 pages where sequences have
                                 fewer tokens than one CTA on average or the values would take more
                                 than 8 GB, else values */
} pkv_prefill_params;

#define PKV_READING_AUTO 0
#define PKV_READING_DIRECT 1
#define PKV_READING_VALUES 2

typedef struct pkv_prefill_plan {
  int32_t unit_tokens;    /* tokens of one CTA */
  int32_t key_tile;       /* key rows per step */
  int32_t units;          /* CTAs per KV head and split, those of short last tiles included (of a group of
                             sequences, see workspace_bytes) */
  int32_t splits;
  int32_t smem_bytes;     /* dynamic shared memory of a CTA */
  int32_t value_blocks;   /* blocks of 128 rows of values in the workspace (0: pages are read directly) */
  size_t workspace_bytes; /* f32 states of split key ranges (none with splits = 1), and the values: as many as
                             the tables have rows, or the tokens and the window need; tables cut to the
                             longest sequence keep it, and the pass over it, small. Affine pages, which have no
                             other reading: where all values would take more than 8 GB, those of a group of
                             sequences, as many as 8 GB hold (at least one), and the groups go through the
                             workspace one after the other. 2^31 rows of values at once (KV heads counted) are
                             refused: PKV_ERR_UNSUPPORTED_SHAPE */
} pkv_prefill_plan;

int pkv_make_prefill_plan(const pkv_pool_layout* layout, const pkv_prefill_params* params, int32_t sm_count,
                          pkv_prefill_plan* plan);
int pkv_prefill_plan_for_current_device(const pkv_pool_layout* layout, const pkv_prefill_params* params,
                                        pkv_prefill_plan* plan);

/*   q             bf16 rows of num_q_heads heads, 16-byte aligned; q_strides as for
 *                 pkv_norm_rotate, packed; not zero for a dim of more than one
 *   query_starts  int32 [num_seqs + 1], not falling, within 0 .. num_tokens. Rows of tokens outside
 *                 [query_starts[0], query_starts[num_seqs]) are neither read nor written.
 *   seq_lens      rows held, the new ones included
 *   out           bf16 [num_tokens, num_q_heads, v_head_dim]
 *   workspace     plan.workspace_bytes; calls that overlap on the GPU need one each
 * A seq_len below the sequence's tokens or above the table's rows writes zeros for the sequence and sets
 * PKV_DEVERR_BAD_SEQ_LEN, as do starts that fall or leave 0 .. num_tokens (their sequences' outputs are
 * then unspecified). Rows of bad blocks are skipped and flagged; a query that sees no row gets zeros.
 * Cached rows below seq_len must be finite; blocks wholly outside the window are not read. */
int pkv_paged_prefill_attention(const pkv_pool_layout* layout, const pkv_prefill_params* params, const void* q,
                                const pkv_row_strides* q_strides, const void* k_pool, const void* v_pool,
                                const void* k_scales, const void* k_biases, const void* v_scales,
                                const void* v_biases, const int32_t* block_tables, const int32_t* seq_lens,
                                const int32_t* query_starts, float scale, void* out, void* workspace,
                                size_t workspace_bytes, int32_t* error_flag, void* stream);

/* Bit-exact gather of one pool plane into contiguous per-sequence rows, the
 * fetch copy of the pages' BlockPool.gather / pickBlocks (state/paged/cache.ts):
 *   out[b][h][t][:] = pool[block_tables[b][t / block_size]][h][t % block_size][:]
 * for t < seq_lens[b] (<= max_len); rows t >= seq_lens[b] of out are left as they
 * were. pool: [num_blocks, num_kv_heads, block_size, row_bytes] bytes;
 * out: [num_seqs, num_kv_heads, max_len, row_bytes] bytes. row_bytes must be a
 * positive multiple of 4; pool and out 16-byte aligned. Bad block ids skip the
 * row and set PKV_DEVERR_BAD_BLOCK; a seq_len outside [0, max_len] or above
 * max_blocks_per_seq*block_size sets PKV_DEVERR_BAD_SEQ_LEN and copies nothing
 * for that sequence. */
int pkv_paged_gather(const void* pool, int32_t num_blocks, int32_t num_kv_heads, int32_t block_size,
                     int32_t row_bytes, const int32_t* block_tables, const int32_t* seq_lens,
                     int32_t num_seqs, int32_t max_blocks_per_seq, int32_t max_len, void* out,
                     int32_t* error_flag, void* stream);

/* Message for a PKV_ERR_* code (static storage). */
const char* pkv_strerror(int code);

/* Text of the last PKV_ERR_CUDA failure on this thread (static per-thread storage). */
const char* pkv_last_cuda_error(void);

/* Sets the bound, in nanoseconds, of one wait of the partial kernel's main loop for
 * the data of a pipeline stage, for every decode call prepared after it in this
 * process (a pkv_step keeps the bound it was created with), and returns the previous
 * bound; 0 restores the default of one second. The pages have no counterpart of it.
 * A wait that runs out gives up without a fault: the kernel sets PKV_DEVERR_TIMEOUT
 * in *error_flag, stops reading, lets every copy it has issued land (that drain waits
 * up to the default bound), finishes its epilogue and returns, so the stream and the
 * context stay usable and the output of that call is unspecified. It exists to check
 * this give-up path on a working GPU: a bound shorter than the time a stage takes
 * to arrive from HBM (a few microseconds) makes it run out on any input. Not
 * thread-safe against calls being prepared on other threads. */
uint64_t pkv_set_wait_limit_ns(uint64_t ns);

/* Library version, major*10000 + minor*100 + patch. */
int pkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_DECODE_H */
