/*
 * pkv.h -- C ABI of the paged KV cache library (libpkv.so).
 *
 * The library implements the data-parallel hot path of PagedAttention for one
 * GPU (sm_103a):
 *
 *   pkv_paged_attention_decode  single-query decode attention that reads the
 *                               KV cache through per-sequence block tables;
 *   pkv_paged_attention_decode_append
 *                               the same, writing each sequence's new token
 *                               in the same launch;
 *   pkv_decode_plan_*           a decode call validated once and launched (or
 *                               run as a whole serving step) many times;
 *   pkv_paged_attention_chunk   attention of any number of new tokens per
 *                               sequence over the cache (prompts, chunks of
 *                               prompts, drafted tokens, an encoder's states);
 *   pkv_qk_norm_rope[_and_cache] the norm of each query and key head and the
 *                               position rotation, with the slot-mapped write;
 *   pkv_reshape_and_cache       the slot-mapped write of new tokens' K/V;
 *   pkv_reshape_and_cache_q8, pkv_paged_attention_decode_q8
 *                               the write and the decode of a cache held in 8
 *                               bits with a scale per block and KV head;
 *   pkv_block_key_bounds, pkv_select_blocks, pkv_paged_attention_decode_selected
 *                               decode over the blocks whose keys can score
 *                               highest;
 *   pkv_copy_blocks             the whole-block copy behind copy-on-write;
 *   pkv_swap_blocks             block copies between device and page-locked
 *                               host pools (swap out / in);
 *   *_layers                    the cache ops over every layer's pool in one
 *                               launch;
 *   pkv_alloc_* / pkv_seq_* ... the host block manager that hands out blocks,
 *                               counts references, forks and copies on write,
 *                               swaps sequences out and in, exports the block
 *                               tables, and checkpoints its state.
 *
 * Sources (cited by page title and section):
 *   [P1] "Paged Attention: OS-Inspired Memory Management for KV Caches",
 *        modernaiengineering.com, lesson 13.6;
 *   [P2] "What is PagedAttention and how does it manage KV cache?", n4n.ai;
 *   [P3] worksonmygpu.com, deep-dive post "PagedAttention (vLLM)".
 *
 * Conventions for every call:
 *   - Every entry point returns an int status (pkv_status below).  A call that
 *     fails leaves every host-side object exactly as it was.
 *   - Device pointers are BORROWED: the caller owns and allocates all device
 *     memory (KV pools, tables, outputs, workspace).  The library never
 *     allocates device memory itself.
 *   - Kernels are launched asynchronously on the caller's stream (NULL = the
 *     legacy default stream).  Argument errors are detected on the host before
 *     any launch.  Errors that depend on device data (a slot or table entry
 *     outside the pool, a device wait that gave up) are written to the
 *     caller's int32 device status word: the first error wins (0 -> code), the
 *     word is never cleared by the library, and a NULL status pointer means
 *     "do not report".  Kernels never trap: after a device error the affected
 *     outputs are unspecified but the CUDA context stays usable.
 *   - Cache layout (chosen here; [P2] "How PagedAttention works" only fixes
 *     that tokens are contiguous inside a block): key_cache and value_cache
 *     are separate fp16 tensors [num_blocks][num_kv_heads][block_size][head_dim],
 *     row-major.  Token `off` of physical block `b`, KV head `h`, element `i`
 *     sits at element ((b*num_kv_heads + h)*block_size + off)*head_dim + i.
 *   - A slot names one token position of the pool: slot = b*block_size + off
 *     ([P1] paged_vs_contiguous.py example: token 37 -> logical block 2,
 *     offset 5).
 *   - Base pointers of the caches, query, key, value and out must be 16-byte
 *     aligned (torch allocations are 256-byte aligned).
 *   - Calls launch on the calling thread's current CUDA device, which must be
 *     the one that holds their device pointers.  Several devices in one process
 *     are fine (each decode kernel's dynamic shared-memory limit is raised per
 *     device); a plan, like any call, runs on the device it was created on.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; declared here so that this header
 * needs no CUDA header. */
typedef struct CUstream_st *pkv_stream_t;

typedef enum pkv_status {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,     /* bad pointer, size, shape or id (host check) */
    PKV_ERR_OUT_OF_BLOCKS = 2,   /* block manager: free list cannot satisfy the call */
    PKV_ERR_CUDA = 3,            /* a CUDA runtime call failed (launch, attribute) */
    PKV_ERR_DEVICE_TIMEOUT = 4,  /* device: a bounded wait gave up (status word only) */
    PKV_ERR_OUT_OF_RANGE = 5,    /* device: slot / table entry / context outside the pool or table */
    PKV_ERR_NOT_FOUND = 6,       /* block manager: unknown or released sequence id */
    PKV_ERR_UNSUPPORTED = 7,     /* shape not compiled into this build (head_dim, block_size, group) */
    PKV_ERR_SWAPPED = 8          /* block manager: the sequence is swapped out (or, for a swap in, resident) */
} pkv_status;

/* Human-readable name of a status code (static string, never NULL). */
const char *pkv_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int pkv_version(void);

/* ------------------------------------------------------------------------ */
/* Decode attention                                                          */
/* ------------------------------------------------------------------------ */

/*
 * pkv_paged_attention_decode
 *
 * [P1] "How PagedAttention works", step 4: each decode step walks the block
 * table, loads each block's keys and values and computes attention exactly as
 * if they were contiguous.  For every sequence s and query head h, with
 * L = context_lens[s], kvh = h / (num_heads / num_kv_heads) (consecutive
 * query-head groups share a KV head), and token t stored in physical block
 * block_tables[s][t / block_size] at offset t % block_size:
 *
 *     out[s][h] = sum_t softmax_t(scale * q[s][h] . K[t][kvh]) * V[t][kvh]
 *
 * computed in fp32 (online softmax, fp32 accumulation) and rounded to fp16 to
 * nearest even.  L == 0 gives an all-zero row.  Entries of a table row past
 * ceil(L / block_size) are never read (they may hold -1).
 *
 * Arguments (all device pointers unless noted):
 *   out          fp16 [num_seqs][num_heads][head_dim]           (written)
 *   query        fp16 [num_seqs][num_heads][head_dim]
 *   key_cache    fp16 [num_blocks][num_kv_heads][block_size][head_dim]
 *   value_cache  same shape as key_cache
 *   block_tables int32 [num_seqs][max_blocks_per_seq], row-major
 *   context_lens int32 [num_seqs]
 *   scale        softmax scale (host value), usually 1/sqrt(head_dim)
 *   num_ctas     persistent grid size; 0 = one full wave (SM count x CTAs
 *                per SM).  A small batch leaves some of them idle (every
 *                worker warp gets at least 4 chunks of 16 rows; while the
 *                (sequence, KV head) segments are short, no more CTAs work
 *                than there are segments).  Any value >= 1 gives the same
 *                result within rounding; 1 makes every sequence a single
 *                pass.
 *   workspace    device scratch of at least pkv_decode_workspace_size(...)
 *                bytes for the same (num_seqs, num_heads, num_kv_heads,
 *                head_dim, block_size, num_ctas); 256-byte aligned.  It
 *                carries state from call to call (an epoch word that every
 *                call advances, and completion counters that each call
 *                prepares for the next), so keep one workspace per stream of
 *                calls; what it holds on first use does not matter (zeroed
 *                or not), nor does a call that gave up, and a launch recorded
 *                once and replayed (a CUDA graph) works.  It must not be used
 *                by another call that runs at the same time.
 *   dev_status   int32 device status word (nullable), see conventions.
 *   stream       CUDA stream.
 *
 * Supported: head_dim in {64, 128}; block_size in {8, 16, 32, 64, 128};
 * num_heads / num_kv_heads in {1, 2, 4, 8}; 1 <= num_seqs <= 4096;
 * num_blocks * num_kv_heads * block_size < 2^31 (the cache rows the tensor
 * copies address: up to 512 GB per cache at head_dim 128, 256 GB at 64) and
 * max_blocks_per_seq * block_size <= 2^30, else PKV_ERR_INVALID_ARG.
 * A context longer than max_blocks_per_seq*block_size, or a table entry
 * outside [0, num_blocks), sets PKV_ERR_OUT_OF_RANGE in dev_status; such a
 * context is clamped to its table and such an entry reads block 0.
 * Launches one kernel on `stream`, with programmatic dependent launch: it may
 * start while the preceding kernel in the stream finishes, and reads
 * context_lens and block_tables before it waits for that kernel (everything
 * else — the caches, query, workspace, out — only after).  So context_lens
 * and block_tables must not be written by a kernel that signals its
 * dependents early (griddepcontrol.launch_dependents /
 * cudaTriggerProgrammaticLaunchCompletion) before it writes them; memory
 * copies, ordinary kernels and this library's kernels never do.
 */
int pkv_paged_attention_decode(void *out, const void *query,
                               const void *key_cache, const void *value_cache,
                               const int32_t *block_tables, int max_blocks_per_seq,
                               const int32_t *context_lens,
                               int num_seqs, int num_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               float scale, int num_ctas,
                               void *workspace, size_t workspace_bytes,
                               int32_t *dev_status, pkv_stream_t stream);

/*
 * pkv_paged_attention_decode_append
 *
 * One decode step in one launch: what pkv_reshape_and_cache of each
 * sequence's new token followed by pkv_paged_attention_decode computes ([P1]
 * "How PagedAttention works", steps 2-4: write the token into the next slot
 * of the last block, then attend over the whole table).  For every sequence s
 * with L = context_lens[s] > 0, the new token is position L-1: key[s] and
 * value[s] ([num_kv_heads][head_dim] each) are written to that position's
 * slot (block block_tables[s][(L-1)/block_size], offset (L-1)%block_size) of
 * key_cache / value_cache, and attention covers positions 0..L-1 with them.
 * No slot mapping is needed: the slot follows from the table.  Outputs and
 * cache contents are identical to the two-call sequence.  Copy-on-write
 * copies (pkv_copy_blocks) must still run before it.
 *
 *   key, value   fp16 [num_seqs][num_kv_heads][head_dim] (device)
 *   key_cache, value_cache  written at the new tokens' slots (device)
 * Other arguments, workspace, errors and launch ordering (which inputs are
 * read before the wait for the preceding kernel) as pkv_paged_attention_decode.
 */
int pkv_paged_attention_decode_append(void *out, const void *query,
                                      const void *key, const void *value,
                                      void *key_cache, void *value_cache,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *context_lens,
                                      int num_seqs, int num_heads, int num_kv_heads,
                                      int head_dim, int block_size, int num_blocks,
                                      float scale, int num_ctas,
                                      void *workspace, size_t workspace_bytes,
                                      int32_t *dev_status, pkv_stream_t stream);

/*
 * Decode plans: validate once, launch many times.
 *
 * A serving loop calls the decode with the same buffers every step; only
 * their contents (queries, new tokens, tables, lengths) change.
 * pkv_decode_plan_create checks the arguments, picks the kernel and grid and
 * encodes the caches' TMA descriptors once; pkv_decode_plan_launch then
 * launches exactly what pkv_paged_attention_decode_append (key/value
 * non-NULL) or pkv_paged_attention_decode (both NULL) would, with no host
 * work but the launch.  Same results, errors and device status as those
 * calls.  The plan borrows every pointer: the buffers must outlive it, and
 * must not be moved or freed while it is in use.  A plan is read-only after
 * creation (launches from several host threads are fine; on one workspace
 * they must be stream-ordered, as for the direct calls).
 *
 * A plan's out may also be page-locked host memory mapped into the device's
 * address space (cudaHostAlloc / cudaMallocHost memory on a system with
 * unified addressing, or memory registered with cudaHostRegisterMapped).
 * The kernel then writes each output row over the CPU-GPU link as soon as it
 * is final, so a serving step needs no copy of the output back
 * (pkv_decode_plan_step with host_out == NULL); the host reads out once the
 * stream has passed the launch.  pkv_decode_plan_create checks where out
 * lives (cudaPointerGetAttributes): device memory of the current device,
 * managed memory or mapped host memory; anything else (pageable host memory,
 * another device's memory) is PKV_ERR_INVALID_ARG, a failed query
 * PKV_ERR_CUDA.  The direct calls take device or managed memory only.
 */
typedef struct pkv_decode_plan pkv_decode_plan_t;
int pkv_decode_plan_create(void *out, const void *query, const void *key, const void *value,
                           void *key_cache, void *value_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens,
                           int num_seqs, int num_heads, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks,
                           float scale, int num_ctas,
                           void *workspace, size_t workspace_bytes,
                           int32_t *dev_status, pkv_decode_plan_t **plan);
int pkv_decode_plan_launch(const pkv_decode_plan_t *plan, pkv_stream_t stream);

/*
 * pkv_decode_plan_step: one serving step in one call, all on `stream`:
 * in_bytes from host_in to dev_in (the step's inputs -- queries, new K/V,
 * tables, lengths -- staged in one region that the plan's device pointers
 * lie in), then the plan's launch, then the plan's output (fp16
 * [num_seqs][num_heads][head_dim]) to host_out.  in_bytes == 0 skips the
 * first copy and host_out == NULL the last.  host_in / host_out should be
 * page-locked for the copies to be asynchronous.  The caller synchronises the
 * stream before reading host_out or reusing host_in.  PKV_ERR_INVALID_ARG for
 * a NULL plan or a missing pointer; PKV_ERR_CUDA when a copy or the launch
 * fails to enqueue (nothing after it is enqueued).
 */
int pkv_decode_plan_step(const pkv_decode_plan_t *plan, void *dev_in, const void *host_in, size_t in_bytes,
                         void *host_out, pkv_stream_t stream);

/*
 * pkv_decode_plan_step_mapped: one serving step whose inputs the kernel reads
 * straight from page-locked host memory, with no copy in: every input pointer
 * of the plan (query, key, value, block_tables, context_lens, shared_blocks)
 * that lies in [dev_base, dev_base + in_bytes) is read at the same offset of
 * host_in, over the CPU-GPU link; the others as created.  dev_base is only an
 * address here (the region the plan was created on): it is neither read nor
 * written.  The queries and new K/V rows are copied by the kernel's lanes 16
 * bytes at a time, a few chunks ahead of their use, and the lengths and
 * tables are read in its prologue.  Then the output goes to host_out as in
 * pkv_decode_plan_step (NULL: none; a plan whose out is mapped host memory
 * needs none).  Same results, bit for bit, as staging host_in into dev_base
 * and launching.
 *
 *   host_in  page-locked host memory mapped for the current device
 *            (cudaHostAlloc / cudaMallocHost with unified addressing, or
 *            cudaHostRegisterMapped), in_bytes long, holding the inputs at
 *            their offsets in the plan's region; query, key and value
 *            16-byte aligned.  The caller must not write it until the
 *            stream has passed the launch.
 * PKV_ERR_INVALID_ARG for a NULL plan, in_bytes == 0, host_in that is not
 * such memory (cudaPointerGetAttributes), a misaligned input, or an input
 * that starts inside the region but runs past its end (nothing is
 * enqueued); PKV_ERR_UNSUPPORTED if the library was built without the
 * kernels that read host inputs; PKV_ERR_CUDA when the launch or the copy
 * out fails to enqueue.
 */
int pkv_decode_plan_step_mapped(const pkv_decode_plan_t *plan, const void *dev_base, const void *host_in,
                                size_t in_bytes, void *host_out, pkv_stream_t stream);
void pkv_decode_plan_destroy(pkv_decode_plan_t *plan);

/*
 * Decode attention with prefix sharing.
 *
 * [P1] "Memory sharing across requests" and [P2] "How PagedAttention works"
 * (prefix sharing): sequences forked from one prompt read the same physical
 * blocks for it.  These calls compute exactly what
 * pkv_paged_attention_decode_append (key/value non-NULL) or
 * pkv_paged_attention_decode (both NULL) compute, and take one more input:
 *
 *   shared_blocks  int32 [num_seqs] (device): for s >= 1, how many leading
 *                  logical blocks sequence s has in common with sequence
 *                  s - 1 (same physical block at the same logical index);
 *                  entry 0 is ignored.  pkv_export_shared_prefix computes it.
 *                  It must not claim more than the tables hold in common
 *                  (the shared blocks are read through the first sequence's
 *                  table); smaller values are always correct, and all zeros
 *                  is the plain decode.
 *
 * Up to 8 consecutive sequences that share blocks form a group; the group's
 * shared full blocks (never the block of a member's last token) are read
 * once for all of them, with the members' queries as the rows of one
 * tensor-core tile, then each member's own blocks with only its row live.
 * Results are run-to-run deterministic for a fixed grid and agree with the
 * plain decode within rounding (not bit for bit).  On a batch without
 * sharing the plain calls are faster (the grouped kernel keeps 8 rows per
 * segment): pass the hints where forks share blocks.  The grouped kernel serves group 1
 * (num_heads == num_kv_heads), block sizes 16 to 128 and up to 1024
 * sequences; other calls run the plain kernel (shared_blocks is then not
 * read).  The workspace is pkv_decode_workspace_size_shared(...) bytes, and
 * otherwise follows the rules of pkv_paged_attention_decode.  A NULL
 * shared_blocks with num_seqs > 0 is PKV_ERR_INVALID_ARG.
 */
int pkv_paged_attention_decode_shared(void *out, const void *query, const void *key,
                                      const void *value, void *key_cache, void *value_cache,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *context_lens, const int32_t *shared_blocks,
                                      int num_seqs, int num_heads, int num_kv_heads,
                                      int head_dim, int block_size, int num_blocks,
                                      float scale, int num_ctas,
                                      void *workspace, size_t workspace_bytes,
                                      int32_t *dev_status, pkv_stream_t stream);
int pkv_decode_plan_create_shared(void *out, const void *query, const void *key, const void *value,
                                  void *key_cache, void *value_cache,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *context_lens, const int32_t *shared_blocks,
                                  int num_seqs, int num_heads, int num_kv_heads,
                                  int head_dim, int block_size, int num_blocks,
                                  float scale, int num_ctas,
                                  void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, pkv_decode_plan_t **plan);
size_t pkv_decode_workspace_size_shared(int num_seqs, int num_heads, int num_kv_heads,
                                        int head_dim, int block_size, int num_ctas);

/* Bytes of workspace pkv_paged_attention_decode needs (host call; queries the
 * current device's SM count when num_ctas == 0).  Returns 0 for unsupported
 * shapes. */
size_t pkv_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                 int head_dim, int block_size, int num_ctas);

/* The grid size num_ctas == 0 resolves to on the current device for this
 * shape (host call), or 0 for unsupported shapes. */
int pkv_decode_default_ctas(int num_heads, int num_kv_heads, int head_dim,
                            int block_size);

/*
 * pkv_paged_attention_decode_noalloc
 *
 * The pages have no counterpart to this entry point: it exists for callers
 * that cannot allocate device memory themselves.  Typical ones are a serving
 * engine or framework that has already handed nearly all of the GPU's memory
 * to its own KV pool and caching allocator (a separate cudaMalloc would fail,
 * or fragment memory the engine budgets to the byte), a plug-in that the host
 * application gives no allocation rights, and hot loops that cannot afford
 * cudaMalloc/cudaFree, which may synchronise the whole device.
 *
 * It computes exactly what pkv_paged_attention_decode computes, with the same
 * arguments minus workspace / workspace_bytes.  Its scratch is a fixed array
 * of PKV_DECODE_NOALLOC_SCRATCH_BYTES (16 MiB) that lives inside the library
 * as a static device variable: every GPU that loads the library holds those
 * 16 MiB until the process exits.  The call itself allocates nothing: no
 * cudaMalloc, no cudaFree, no allocating library routine.
 *
 * Limit: the scratch a call needs is pkv_decode_workspace_size(num_seqs,
 * num_heads, num_kv_heads, head_dim, block_size, num_ctas); a call that needs
 * more than PKV_DECODE_NOALLOC_SCRATCH_BYTES returns PKV_ERR_INVALID_ARG and
 * launches nothing.  The need grows with num_seqs * num_kv_heads (16 bytes
 * each) and with the grid.  At the default grid of one CTA per SM on a
 * 152-SM GB300 the call fits while num_seqs * num_kv_heads is at most:
 *
 *                 group 1    group 2    group 4    group 8
 *   head_dim 64   1,003,408    958,272    867,984    687,408
 *   head_dim 128    959,632    870,720    692,880    337,200
 *
 * (so at num_seqs = 4096, group 8, head_dim 128, num_kv_heads may be at most
 * 82).  A larger num_ctas leaves less room.
 *
 * Set-up: the first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it; make that
 * first call before any stream capture.  A failed look-up returns
 * PKV_ERR_CUDA.  Devices with ordinals 0 to 63 are served; a call with a
 * higher ordinal current returns PKV_ERR_UNSUPPORTED.
 *
 * Sharing: all calls in the process share the one array, and it keeps what
 * the last call left in it.  Nothing needs clearing between calls: partial
 * results are rewritten before they are read, and the completion counters
 * are tagged with an epoch that every call advances, so leftovers of an
 * earlier call (even one that failed) are never taken for the current one.
 * Two calls whose kernels
 * overlap on the GPU (different streams, or different host threads) race on
 * the array and give wrong results: serialise them, for example on one
 * stream.  Other errors and the device status word behave as for
 * pkv_paged_attention_decode.
 */
#define PKV_DECODE_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)
int pkv_paged_attention_decode_noalloc(void *out, const void *query,
                                       const void *key_cache, const void *value_cache,
                                       const int32_t *block_tables, int max_blocks_per_seq,
                                       const int32_t *context_lens,
                                       int num_seqs, int num_heads, int num_kv_heads,
                                       int head_dim, int block_size, int num_blocks,
                                       float scale, int num_ctas,
                                       int32_t *dev_status, pkv_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Chunk attention                                                           */
/* ------------------------------------------------------------------------ */

/*
 * pkv_paged_attention_chunk
 *
 * Attention of several new tokens per sequence over the paged cache: a whole
 * prompt, a chunk of a long prompt, drafted tokens to verify, single tokens,
 * or any mixture of them in one call.  The new tokens' keys and values must
 * be in the cache already (pkv_reshape_and_cache or
 * pkv_qk_norm_rope_and_cache with the slots of pkv_append_tokens).
 *
 * Sequence s owns the query rows query_starts[s] .. query_starts[s+1]-1; let
 * n be their number and L = context_lens[s].  Row i of them is position
 * p = L - n + i of its sequence.  For every query head h, with
 * kvh = h / (num_heads / num_kv_heads) and K[t], V[t] found through the block
 * table as in pkv_paged_attention_decode:
 *
 *     out[row][h] = sum_t softmax_t(scale * q[row][h] . K[t][kvh]) * V[t][kvh]
 *
 * over the visible t: with causal != 0, t <= p, and with window > 0 also
 * t > p - window; with causal == 0 every t < L, whatever n is (the cache then
 * holds another sequence's states, for instance an encoder's, and window must
 * be 0).  A row that sees no position (L == 0, or p < 0 where n > L), or none
 * whose score is above minus infinity, gives zeros.  Scores, softmax
 * statistics and the weighted sum are held in fp32; the softmax weights are
 * rounded to fp16 for the second product (11 significant bits down to 2^-23 of
 * the row's largest weight, steps of 2^-33 of it below), and the result is
 * rounded to fp16, to nearest even.
 *
 * What no row of a sequence sees is not read for the result: table entries
 * past ceil(L / block_size), or of blocks that lie wholly before every
 * row's window, may hold -1, and cache positions outside may hold anything.
 * A position that some rows see and others do not does not reach the others,
 * also where its value is infinite or NaN.
 *
 * Arguments (device pointers unless noted):
 *   out          fp16 [num_tokens][num_heads][head_dim]         (written; must
 *                not overlap any input)
 *   query        fp16 [num_tokens][num_heads][head_dim]
 *   key_cache, value_cache, block_tables, max_blocks_per_seq, scale,
 *   dev_status, stream: as for pkv_paged_attention_decode
 *   context_lens int32 [num_seqs]
 *   query_starts int32 [num_seqs + 1], not decreasing, from 0 up to at most
 *                num_tokens.  Rows before the first sequence's and behind the
 *                last one's are left as they were; a sequence may have no rows.
 *   num_tokens   rows of query and out (host value)
 *   causal, window  the mask (host values), above
 *   num_ctas     persistent grid size; 0 = one CTA per SM.  Any value >= 1
 *                gives the same result within rounding.
 *   workspace    device scratch of at least pkv_chunk_workspace_size(...)
 *                bytes for the same (num_tokens, num_heads, num_kv_heads,
 *                head_dim, num_ctas); 256-byte aligned.  It carries nothing
 *                from call to call and needs no clearing, but must not be
 *                used by another call that runs at the same time (two
 *                captured graphs that share one must not overlap).
 *
 * Results are deterministic for a fixed grid.  Supported: head_dim in
 * {64, 128}; block_size in {8, 16, 32, 64, 128}; num_heads / num_kv_heads
 * from 1 to 16; 1 <= num_seqs <= 4096; num_blocks * num_kv_heads * block_size
 * < 2^31; max_blocks_per_seq * block_size <= 2^30; num_ctas <= 4096.
 * num_tokens == 0 or num_seqs == 0 launches nothing.
 * A context longer than its table (clamped to it) or negative (taken as 0), a
 * table entry outside [0, num_blocks) among those read (block 0 is read), and
 * query_starts that decrease or leave [0, num_tokens] (clamped to the rows
 * there are) set PKV_ERR_OUT_OF_RANGE.
 */
int pkv_paged_attention_chunk(void *out, const void *query,
                              const void *key_cache, const void *value_cache,
                              const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *context_lens, const int32_t *query_starts,
                              int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                              int head_dim, int block_size, int num_blocks,
                              float scale, int causal, int window, int num_ctas,
                              void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, pkv_stream_t stream);

/* Bytes of workspace pkv_paged_attention_chunk needs (host call; queries the
 * current device's SM count when num_ctas == 0).  Returns 0 for unsupported
 * shapes. */
size_t pkv_chunk_workspace_size(int num_tokens, int num_heads, int num_kv_heads,
                                int head_dim, int num_ctas);

/* ------------------------------------------------------------------------ */
/* Cache writes                                                              */
/* ------------------------------------------------------------------------ */

/*
 * pkv_reshape_and_cache
 *
 * [P1] "How PagedAttention works", steps 2-3: a new token goes into the next
 * slot of its sequence's last block.  For t in [0, num_tokens): if
 * slot_mapping[t] >= 0, copy key[t][h][:] and value[t][h][:] (every KV head h)
 * to slot slot_mapping[t] of key_cache / value_cache.  A negative slot is
 * skipped.  Bit-exact copies.
 *
 *   key, value    fp16 [num_tokens][num_kv_heads][head_dim] (device)
 *   key_cache, value_cache   pool, layout above (device, written)
 *   slot_mapping  int64 [num_tokens] (device)
 *   dev_status    a slot >= num_blocks*block_size sets PKV_ERR_OUT_OF_RANGE
 *                 and that token is not written.
 * head_dim must be a multiple of 8.  num_tokens == 0 launches nothing.
 * Two tokens with the same slot race (the caller's block manager never
 * produces that).
 */
int pkv_reshape_and_cache(const void *key, const void *value,
                          void *key_cache, void *value_cache,
                          const int64_t *slot_mapping, int num_tokens,
                          int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, int32_t *dev_status,
                          pkv_stream_t stream);

/*
 * pkv_qk_norm_rope, pkv_qk_norm_rope_and_cache
 *
 * The step between a model's projections and its attention: an RMS norm of
 * every query and key head and the position rotation, in one pass over the
 * data.  For each token t and each head x of its queries (and keys):
 *
 *     y = x * weight / sqrt(mean(x^2) + eps)     where the weight is not NULL
 *     y = x                                      where it is NULL
 *
 * then the first rot_dim elements of y are rotated by the position's angles
 * in pairs (a, b) -> (a cos - b sin, b cos + a sin): pair i is elements i and
 * i + rot_dim/2 (interleaved == 0) or 2i and 2i + 1 (interleaved != 0); the
 * other elements stay.  Computed in fp32, rounded once to fp16.
 *
 * pkv_qk_norm_rope writes the queries and keys to query_out and key_out (for
 * pkv_paged_attention_decode_append, which writes the cache itself).
 * pkv_qk_norm_rope_and_cache writes the queries to query_out, and the keys
 * and the (unchanged) values to their cache slots, as pkv_reshape_and_cache
 * does: for pkv_paged_attention_chunk or pkv_paged_attention_decode.
 *
 *   query        fp16 [num_tokens][num_heads][head_dim], a token's heads
 *                contiguous, tokens query_stride elements apart; key, value:
 *                the same with num_kv_heads.  The strides are multiples of 8
 *                and at least one token's elements, so the three may be views
 *                of one projection's output.
 *   query_out, key_out  written, with strides of their own; each may be the
 *                tensor it is made from (same pointer and stride), but must
 *                not overlap an input in any other way
 *   positions    int64 [num_tokens] (device): rows of cos_sin
 *   cos_sin      fp32 [max_positions][rot_dim] (device): rot_dim/2 cosines,
 *                then rot_dim/2 sines; 16-byte aligned
 *   rot_dim      multiple of 16, 0 <= rot_dim <= head_dim; 0: no rotation
 *                (positions and cos_sin may then be NULL)
 *   query_weight, key_weight  fp16 [head_dim] (device, nullable; 16-byte aligned)
 *   eps          >= 0 (host value)
 *   key_cache, value_cache, slot_mapping  as for pkv_reshape_and_cache: a
 *                negative slot writes no key or value (the query is computed)
 *   dev_status   a position outside [0, max_positions) sets
 *                PKV_ERR_OUT_OF_RANGE and nothing of that token is written; a
 *                slot >= num_blocks * block_size sets it and the token's key
 *                and value are not written.
 * head_dim is a multiple of 8 up to 256.  num_tokens == 0 launches nothing.
 */
int pkv_qk_norm_rope(void *query_out, int64_t query_out_stride,
                     void *key_out, int64_t key_out_stride,
                     const void *query, int64_t query_stride,
                     const void *key, int64_t key_stride,
                     const int64_t *positions, const float *cos_sin, int max_positions,
                     int rot_dim, int interleaved,
                     const void *query_weight, const void *key_weight, float eps,
                     int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                     int32_t *dev_status, pkv_stream_t stream);
int pkv_qk_norm_rope_and_cache(void *query_out, int64_t query_out_stride,
                               const void *query, int64_t query_stride,
                               const void *key, int64_t key_stride,
                               const void *value, int64_t value_stride,
                               void *key_cache, void *value_cache,
                               const int64_t *slot_mapping,
                               const int64_t *positions, const float *cos_sin, int max_positions,
                               int rot_dim, int interleaved,
                               const void *query_weight, const void *key_weight, float eps,
                               int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks,
                               int32_t *dev_status, pkv_stream_t stream);

/*
 * pkv_copy_blocks
 *
 * [P1] "Memory sharing across requests": copy-on-write copies a shared block
 * to a fresh block before the writer's token goes in.  For each pair
 * (src, dst) = block_pairs[2*i], block_pairs[2*i+1], copy the block_bytes
 * bytes of physical block src over block dst, in key_cache and in
 * value_cache.  Bit-exact.  Must run before the pkv_reshape_and_cache that
 * writes the copying sequence's token.
 *
 *   block_pairs  int64 [num_pairs][2] (device)
 *   block_bytes  bytes of one physical block in one cache
 *                (num_kv_heads*block_size*head_dim*2 for fp16); multiple of 16
 *   dev_status   a pair outside [0, num_blocks) sets PKV_ERR_OUT_OF_RANGE and
 *                is skipped.
 * The destinations must be pairwise distinct and no destination may also be
 * a source in the same call (pkv_validate_block_pairs checks this on a host
 * copy).  num_pairs == 0 launches nothing.
 */
int pkv_copy_blocks(void *key_cache, void *value_cache,
                    const int64_t *block_pairs, int num_pairs,
                    size_t block_bytes, int num_blocks,
                    int32_t *dev_status, pkv_stream_t stream);

/*
 * Multi-layer cache ops.  [P2] "How PagedAttention works": a block holds its
 * tokens for all layers and heads, so one slot mapping (and one list of
 * copy-on-write pairs) serves every layer.  These do, in ONE launch, what
 * num_layers calls of pkv_reshape_and_cache / pkv_copy_blocks would do, one
 * per layer, with every layer's pool shaped alike.
 *
 *   keys, values            HOST arrays [num_layers] of device pointers, each
 *                           fp16 [num_tokens][num_kv_heads][head_dim]
 *   key_caches, value_caches HOST arrays [num_layers] of device pointers to
 *                           each layer's pool (layout above)
 *   slot_mapping, block_pairs, dev_status: device, as for the one-layer calls
 * 1 <= num_layers <= PKV_MAX_LAYERS.  The pointer arrays are copied into the
 * kernel's parameters; nothing is allocated.  Same errors as the one-layer
 * calls; a NULL or misaligned pointer in an array is PKV_ERR_INVALID_ARG.
 */
#define PKV_MAX_LAYERS 128
int pkv_reshape_and_cache_layers(const void *const *keys, const void *const *values,
                                 void *const *key_caches, void *const *value_caches,
                                 int num_layers, const int64_t *slot_mapping,
                                 int num_tokens, int num_kv_heads, int head_dim,
                                 int block_size, int num_blocks, int32_t *dev_status,
                                 pkv_stream_t stream);
int pkv_copy_blocks_layers(void *const *key_caches, void *const *value_caches,
                           int num_layers, const int64_t *block_pairs, int num_pairs,
                           size_t block_bytes, int num_blocks, int32_t *dev_status,
                           pkv_stream_t stream);

/*
 * pkv_swap_blocks
 *
 * [P2] "Why it matters for KV cache", "Swapping and preemption": blocks are
 * evicted to CPU memory when GPU memory runs short and fetched back when the
 * request resumes ([P1] "Common misconceptions": a technique separate from
 * paging itself).  For each pair (src, dst) = block_pairs[2*i],
 * block_pairs[2*i+1], copy the block_bytes bytes of block src of the SOURCE
 * pool over block dst of the DESTINATION pool, in the key and the value
 * pools.  Bit-exact.  Both pools have the cache layout above (block-major,
 * block_bytes per block); one of them is normally page-locked host memory,
 * which the kernel reads or writes directly over the CPU-GPU link (no copy
 * engine, one launch for any number of scattered blocks).
 *
 *   src_key, src_value    source pools: device memory of the current device
 *                         or page-locked host memory (cudaHostAlloc,
 *                         cudaHostRegister); src_num_blocks blocks each
 *   dst_key, dst_value    destination pools, same rules; dst_num_blocks
 *   block_pairs           int64 [num_pairs][2] (device-accessible): (source
 *                         block, destination block), e.g. the pairs of
 *                         pkv_swap_out (device -> host) or pkv_swap_in
 *                         (host -> device)
 *   block_bytes           bytes of one block in one cache; multiple of 16
 *   dev_status            a pair outside either pool sets
 *                         PKV_ERR_OUT_OF_RANGE and is skipped
 * Pageable (unregistered) host memory, or another device's memory, is
 * PKV_ERR_INVALID_ARG before anything is launched (the pointer attributes are
 * queried on the host; on a machine without a GPU that query fails with
 * PKV_ERR_CUDA).  Destination blocks must be pairwise distinct and must not
 * overlap the source blocks of the same call.  num_pairs == 0 launches
 * nothing.
 */
int pkv_swap_blocks(const void *src_key, const void *src_value,
                    void *dst_key, void *dst_value,
                    const int64_t *block_pairs, int num_pairs, size_t block_bytes,
                    int src_num_blocks, int dst_num_blocks,
                    int32_t *dev_status, pkv_stream_t stream);

/* pkv_swap_blocks for every layer in one launch: HOST arrays [num_layers] of
 * pool pointers (each under the rules above), one pair list for all layers
 * (a block id spans all layers).  1 <= num_layers <= PKV_MAX_LAYERS. */
int pkv_swap_blocks_layers(const void *const *src_keys, const void *const *src_values,
                           void *const *dst_keys, void *const *dst_values, int num_layers,
                           const int64_t *block_pairs, int num_pairs, size_t block_bytes,
                           int src_num_blocks, int dst_num_blocks,
                           int32_t *dev_status, pkv_stream_t stream);

/* Host check of a pair list for pkv_copy_blocks: ids in range, destinations
 * distinct, no destination also a source.  PKV_OK or PKV_ERR_INVALID_ARG. */
int pkv_validate_block_pairs(const int64_t *host_pairs, int num_pairs,
                             int num_blocks);

/* ------------------------------------------------------------------------ */
/* The 8-bit cache                                                           */
/* ------------------------------------------------------------------------ */

/*
 * Writes of any number of tokens and decode of single ones.  Attention of several
 * new tokens (a prompt, a chunk of one, drafts) and decode plans take fp16 caches
 * only.
 *
 * Element type of a cache.  An 8-bit cache has the layout of the fp16 one with
 * one byte per element, and for each of key_cache and value_cache an fp32 scale
 * per (block, KV head): num_blocks rows of num_kv_heads, scale_stride floats
 * apart.  An element is its code times the scale of its block and head.  Codes
 * are int8, -127 .. 127, or e4m3 (four significant bits, up to 448; the format
 * without infinities).
 * A pool's blocks and their scales are copied and swapped like any other:
 * pkv_copy_blocks and pkv_swap_blocks with block_bytes = num_kv_heads *
 * block_size * head_dim for the codes and 4 * scale_stride for the scales (a
 * multiple of 16 for that: scale_stride a multiple of 4).
 */
typedef enum pkv_cache_type {
    PKV_CACHE_F16 = 0,
    PKV_CACHE_INT8 = 1,
    PKV_CACHE_E4M3 = 2
} pkv_cache_type;

/*
 * pkv_reshape_and_cache_q8
 *
 * The write of new tokens into an 8-bit cache: each sequence's newest tokens go
 * to their positions through its block table (the slots of pkv_append_tokens).
 * Sequence s owns the rows query_starts[s] .. query_starts[s+1]-1 of key and
 * value; with n of them and L = context_lens[s] (new tokens counted), row i is
 * position L - n + i.  query_starts NULL: one row per sequence (num_tokens ==
 * num_seqs), sequences with L == 0 have none.
 *
 * A block and head's scale is a / M, rounded to fp32: a the largest magnitude
 * of what the block holds for that head, an fp16 value, and M = 127 (int8) or
 * 448 (e4m3).  For each block that gets new tokens, a0 = 0 if its first position
 * is among them, else a0 = the scale times M, rounded to fp16 (which gives back
 * the a that the scale was made from), and a = max(a0, largest finite |x| of its
 * new rows).  The new rows become the codes nearest to M x / a (ties to even);
 * where a > a0, the block's earlier rows are rounded again, to the codes nearest
 * to code * a0 / a.  Every code is that of the exact quotient.  Infinite elements
 * become the largest code; NaN becomes 0 in int8 and stays NaN in e4m3.  Rows of
 * the block behind the new ones are not written.
 *
 *   key, value    fp16 [num_tokens][num_kv_heads][head_dim] (device), a token's
 *                 heads contiguous, tokens key_stride / value_stride elements
 *                 apart (multiples of 8, at least one token's elements)
 *   key_cache, value_cache   codes [num_blocks][num_kv_heads][block_size]
 *                 [head_dim] (device, written)
 *   key_scale, value_scale   fp32 [num_blocks] rows of num_kv_heads (device,
 *                 written), scale_stride >= num_kv_heads floats apart
 *   block_tables, max_blocks_per_seq   as for pkv_paged_attention_decode
 *   context_lens  int32 [num_seqs]
 *   query_starts  int32 [num_seqs + 1] (nullable), not decreasing, from 0 up to
 *                 at most num_tokens; rows outside are not looked at
 *   cache_type    PKV_CACHE_INT8 or PKV_CACHE_E4M3
 * head_dim in {64, 128}, block_size in {8, 16, 32, 64, 128}, num_seqs <= 4096,
 * num_blocks * num_kv_heads * block_size <= 2^31, max_blocks_per_seq *
 * block_size <= 2^30.  num_tokens == 0 or num_seqs == 0 launches nothing.
 * A context that is negative or longer than its table, more new tokens than
 * context (the tokens before position 0 and past the table are not written), a
 * table entry of a block to write outside [0, num_blocks) (not written), and
 * query_starts that decrease or leave [0, num_tokens] (what is written is then
 * unspecified) set PKV_ERR_OUT_OF_RANGE.  Two sequences that write one block
 * race (the block manager's copy-on-write never lets them).
 */
int pkv_reshape_and_cache_q8(const void *key, int64_t key_stride,
                             const void *value, int64_t value_stride,
                             void *key_cache, void *value_cache,
                             float *key_scale, float *value_scale, int scale_stride,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, const int32_t *query_starts,
                             int num_tokens, int num_seqs, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks, int cache_type,
                             int32_t *dev_status, pkv_stream_t stream);

/*
 * pkv_paged_attention_decode_q8
 *
 * pkv_paged_attention_decode over an 8-bit cache: out[s][h] = sum_t
 * softmax_t(scale * q[s][h] . K[t][kvh]) * V[t][kvh] with K and V the codes
 * times their scales.  The products take the codes as they are (exact in fp16)
 * and accumulate in fp32; softmax statistics and outputs are held in fp32; a
 * weight, with the value's scale in it, goes into the second product as two fp16
 * terms (22 significant bits down to 2^-18 of the weight of the row's largest
 * score with its largest scale, steps of 2^-39 of that below); one rounding to
 * fp16 at the end.  A context of 0 gives zeros.  A row with a score that is not
 * finite is unspecified.
 *
 * With block lists (selected not NULL) the sum runs over the listed blocks'
 * positions below context_lens[s] only, a list for each sequence and KV head:
 *   selected      int32 [num_seqs][num_kv_heads][max_selected]: logical blocks of
 *                 the sequence, in any order.  A block listed twice counts twice.
 *   num_selected  int32 [num_seqs][num_kv_heads]: entries that count, at most
 *                 max_selected and the context's blocks.  No entry: zeros.
 *                 (The work is shared out as if max_selected of them did, or all
 *                 the context's blocks: entries that do not cost steps of zeros.)
 * selected and num_selected go together (both NULL: every block).
 *
 *   key_scale, value_scale, scale_stride  as for pkv_reshape_and_cache_q8; any
 *                 scales from 0 to 2^100
 *   cache_type    PKV_CACHE_INT8 or PKV_CACHE_E4M3
 *   num_ctas      grid size; 0 = as many as run at once.  Any value gives the
 *                 same result within rounding; deterministic for a fixed grid.
 *   workspace     at least pkv_decode_team_workspace_size(...) bytes for the same
 *                 (num_heads, num_kv_heads, head_dim, num_ctas); 256-byte
 *                 aligned.  It carries nothing from call to call and needs no
 *                 clearing, but must not be used by another call that runs at
 *                 the same time.
 * Other arguments as for pkv_paged_attention_decode.  Supported: head_dim in
 * {64, 128}; block_size in {8, 16, 32, 64, 128}; num_heads / num_kv_heads from 1
 * to 16; num_kv_heads <= 2^16; num_seqs <= 4096; num_ctas <= 4096; num_blocks *
 * num_kv_heads * block_size <= 2^31; max_blocks_per_seq * block_size <= 2^30.
 * A context that is negative (taken as 0) or longer than its table (clamped), a
 * table entry outside [0, num_blocks) among those read (block 0 is read), a
 * listed block outside the context (left out) and num_selected out of its range
 * (clamped) set PKV_ERR_OUT_OF_RANGE.
 */
int pkv_paged_attention_decode_q8(void *out, const void *query,
                                  const void *key_cache, const void *value_cache,
                                  const float *key_scale, const float *value_scale, int scale_stride,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *context_lens,
                                  const int32_t *selected, const int32_t *num_selected, int max_selected,
                                  int num_seqs, int num_heads, int num_kv_heads,
                                  int head_dim, int block_size, int num_blocks, int cache_type,
                                  float scale, int num_ctas,
                                  void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, pkv_stream_t stream);

/* Bytes of workspace pkv_paged_attention_decode_q8 and
 * pkv_paged_attention_decode_selected need (host call; queries the current
 * device's SM count when num_ctas == 0).  Returns 0 for unsupported shapes. */
size_t pkv_decode_team_workspace_size(int num_heads, int num_kv_heads, int head_dim, int num_ctas);

/* ------------------------------------------------------------------------ */
/* Decode over selected blocks                                               */
/* ------------------------------------------------------------------------ */

/*
 * pkv_paged_attention_decode_selected: the decode over block lists (as for
 * pkv_paged_attention_decode_q8, selected and num_selected required) of an fp16
 * cache.
 */
int pkv_paged_attention_decode_selected(void *out, const void *query,
                                        const void *key_cache, const void *value_cache,
                                        const int32_t *block_tables, int max_blocks_per_seq,
                                        const int32_t *context_lens,
                                        const int32_t *selected, const int32_t *num_selected,
                                        int max_selected,
                                        int num_seqs, int num_heads, int num_kv_heads,
                                        int head_dim, int block_size, int num_blocks,
                                        float scale, int num_ctas,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_status, pkv_stream_t stream);

/*
 * pkv_block_key_bounds
 *
 * The largest and the smallest key, channel by channel, of each block that
 * holds new tokens, over the block's positions below the context length (all of
 * them are read from the cache again, so nothing depends on what the bounds held
 * before).  To be called after the write of the new tokens, with the same
 * tables, lengths and query_starts.  Blocks that are swapped in again need theirs
 * at the new places: swapped along (pkv_swap_blocks, two layers' bounds as the two
 * pools, block_bytes = 4 * num_kv_heads * head_dim), or made anew with query_starts
 * over whole contexts.  A copy on write needs nothing, since the write that it is
 * for is followed by this call.  A channel with a NaN has NaN for both.
 *
 *   key_bounds  fp16 [num_blocks][num_kv_heads][2][head_dim] (device, written):
 *               the largest, then the smallest; of an 8-bit cache the codes'
 *               times the scale, rounded to fp16
 *   key_scale, scale_stride  8-bit caches only (else NULL, any)
 *   cache_type  PKV_CACHE_F16, PKV_CACHE_INT8 or PKV_CACHE_E4M3
 * Other arguments, shapes and errors as for pkv_reshape_and_cache_q8.  A block
 * that two sequences share may be given by both (they write the same bounds if
 * both see all of it).
 */
int pkv_block_key_bounds(void *key_bounds, const void *key_cache, const float *key_scale, int scale_stride,
                         const int32_t *block_tables, int max_blocks_per_seq,
                         const int32_t *context_lens, const int32_t *query_starts,
                         int num_tokens, int num_seqs, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, int cache_type,
                         int32_t *dev_status, pkv_stream_t stream);

/*
 * pkv_select_blocks
 *
 * For each sequence s and KV head, the blocks whose keys can score highest for
 * the single-token query.  Block b's score is the largest, over the KV head's
 * query heads h, of
 *
 *     sum_i max(q[s][h][i], 0) * hi[b][i] + min(q[s][h][i], 0) * lo[b][i]
 *
 * with hi and lo the block's key bounds: no key of an fp16 cache's block has a
 * larger product with the query (of an 8-bit cache's, whose bounds are rounded to
 * the nearest fp16, none by more than that rounding of its terms).  Of the
 * context's B = ceil(L / block_size) blocks, min(B, max_selected) are kept: the
 * first first_blocks and the last last_blocks, and of the others those with the
 * largest scores, of equal ones the lowest index.  A score that is not finite
 * counts as the largest.  Scores
 * that fp32 sums may not tell apart are summed again as whole numbers of 2^-48,
 * which all these scores are: what is kept is what the exact scores say.
 *
 *   selected      int32 [num_seqs][num_kv_heads][max_selected] (device, written):
 *                 the kept blocks' logical indices in ascending order, then -1
 *   num_selected  int32 [num_seqs][num_kv_heads] (device, written)
 *   query         fp16 [num_seqs][num_heads][head_dim]
 *   key_bounds    as pkv_block_key_bounds writes it
 *   max_selected >= 1, first_blocks >= 0, last_blocks >= 0 (host values),
 *                 first_blocks + last_blocks <= max_selected
 *   workspace     at least pkv_select_workspace_size(num_seqs, num_kv_heads,
 *                 max_blocks_per_seq) bytes, 12 per table entry and KV head;
 *                 256-byte aligned; as for pkv_paged_attention_decode_q8
 * The kernel goes by the table's width, since contexts are known on the device
 * only: tables of more than 4096 columns take two kernels with the scores in the
 * workspace, several times as slow, whatever the contexts are; up to there a table
 * four times as wide as the contexts costs up to 7 us.
 * Supported: head_dim in {64, 128}; block_size in {8, 16, 32, 64, 128};
 * num_heads / num_kv_heads from 1 to 16; num_kv_heads <= 65535; num_seqs <= 4096;
 * sizes as for pkv_paged_attention_decode_q8.  A context that is negative (taken
 * as 0) or longer than its table (clamped) and a table entry outside
 * [0, num_blocks) among those read (block 0's bounds are taken) set
 * PKV_ERR_OUT_OF_RANGE.
 */
int pkv_select_blocks(int32_t *selected, int32_t *num_selected,
                      const void *query, const void *key_bounds,
                      const int32_t *block_tables, int max_blocks_per_seq,
                      const int32_t *context_lens,
                      int num_seqs, int num_heads, int num_kv_heads,
                      int head_dim, int block_size, int num_blocks,
                      int max_selected, int first_blocks, int last_blocks,
                      void *workspace, size_t workspace_bytes,
                      int32_t *dev_status, pkv_stream_t stream);

/* Bytes of workspace pkv_select_blocks needs.  Returns 0 for sizes out of
 * range. */
size_t pkv_select_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq);

/* ------------------------------------------------------------------------ */
/* Block manager (host)                                                      */
/* ------------------------------------------------------------------------ */

/*
 * A pool of num_blocks physical blocks of block_size token slots each
 * ([P1] "What PagedAttention is"; [P2] "How PagedAttention works": a global
 * pool handed out block by block).
 *
 * Rules ([P1] "How PagedAttention works", "Memory sharing across requests",
 * practice block manager and its exercises):
 *   - The free list is FIFO: blocks are taken from the front and released
 *     blocks are put at the back, in table order.  initial_free_order (host,
 *     nullable) gives the starting order (a permutation of 0..num_blocks-1);
 *     NULL means 0, 1, 2, ...
 *   - Every block has a reference count (sequences using it) and a fill
 *     (token slots written).
 *   - Appending a token: if the sequence has no block or its last block is
 *     full, a fresh block is taken; else if the last block is shared
 *     (count > 1) it is copied on write: a fresh block takes the old block's
 *     fill, the table points at it, the old block's count drops by one, and
 *     the pair (old, new) is returned for pkv_copy_blocks.  Then the token
 *     takes the next slot of the last block.
 *   - Fork: the child's table is a copy of the parent's (partial last block
 *     included); every block's count rises by one.  No device work.
 *   - Release: every block's count drops by one; blocks reaching zero go back
 *     to the free list.  No device work.
 *   - Sequence ids are handed out 0, 1, 2, ... and never reused.
 * An operation that needs more free blocks than there are returns
 * PKV_ERR_OUT_OF_BLOCKS and changes nothing.  The object is not thread-safe.
 *
 * Swapping ([P2] "Why it matters for KV cache", "Swapping and preemption";
 * [P1] "Common misconceptions").  An optional second pool of host blocks
 * (pkv_alloc_host_pool) with its own FIFO free list, counts and fills:
 *   - Swap out of a group of distinct resident sequences: every distinct
 *     device block the group holds gets one host block, in order of first
 *     appearance (sequences in the given order, each table in logical order),
 *     with count = the group members holding it and the block's fill.  The
 *     device block's count drops by that many; at zero it returns to the
 *     device free list (same order).  The tables then name host blocks.
 *   - Swap in: the mirror image, host blocks -> fresh device blocks.
 *   - Sharing inside a group survives the round trip; sharing with sequences
 *     outside it does not (each keeps its own copy).
 *   - A swapped-out sequence can be released (its host blocks go back to the
 *     host free list) or swapped in; append, fork, export and swap out return
 *     PKV_ERR_SWAPPED.
 *   - Each call returns the (source, destination) pairs whose data
 *     pkv_swap_blocks must move, in allocation order, before the blocks are
 *     used.  Out of blocks in the destination pool: PKV_ERR_OUT_OF_BLOCKS,
 *     nothing changed.
 */
typedef struct pkv_alloc pkv_alloc_t;

int pkv_alloc_create(int num_blocks, int block_size,
                     const int32_t *initial_free_order, pkv_alloc_t **out);
void pkv_alloc_destroy(pkv_alloc_t *a);

int pkv_seq_new(pkv_alloc_t *a, int *seq_id);

/* Append one token.  *slot_out = its slot; cow_pair_out = {src, dst} of a
 * copy-on-write, or {-1, -1}.  cow_pair_out may be NULL only if the caller
 * knows no copy can happen. */
int pkv_append_token(pkv_alloc_t *a, int seq, int64_t *slot_out,
                     int32_t cow_pair_out[2]);

/* Append n tokens to one sequence, all or nothing.  slots_out [n] (nullable)
 * receives their slots.  At most one copy-on-write can happen (the first
 * token's); cow_pair_out [2] (nullable) receives it, *n_cow (nullable) is 0
 * or 1. */
int pkv_append_tokens(pkv_alloc_t *a, int seq, int n, int64_t *slots_out,
                      int32_t *cow_pair_out, int *n_cow);

/* One decode step's appends: one token to each of the n DISTINCT sequences
 * seqs[0..n), in that order, all or nothing.  slots_out [n]; cow_pairs_out
 * [n][2] receives the copy-on-write pairs in order, *n_cow their count. */
int pkv_append_batch(pkv_alloc_t *a, const int32_t *seqs, int n,
                     int64_t *slots_out, int32_t *cow_pairs_out, int *n_cow);

int pkv_fork(pkv_alloc_t *a, int parent, int *child);

/* Release a sequence; *n_freed (nullable) = blocks returned to the free list. */
int pkv_release(pkv_alloc_t *a, int seq, int *n_freed);

/* Block tables and context lengths of n sequences, for the decode call.
 * tables [n][max_blocks_per_seq] row-major, padded with -1; ctx_lens [n]
 * (nullable).  A table longer than max_blocks_per_seq is an
 * PKV_ERR_INVALID_ARG (nothing written). */
int pkv_export_tables(const pkv_alloc_t *a, const int32_t *seqs, int n,
                      int32_t *tables, int max_blocks_per_seq,
                      int32_t *ctx_lens);

/* Prefix sharing of a batch, for pkv_paged_attention_decode_shared: for i in
 * [1, n), shared_out[i] = the number of leading logical blocks of sequence
 * seqs[i] whose physical block is the one of seqs[i-1] at the same logical
 * index (the blocks a fork shares with its parent until copy-on-write);
 * shared_out[0] = 0.  Same errors as pkv_export_tables (nothing written). */
int pkv_export_shared_prefix(const pkv_alloc_t *a, const int32_t *seqs, int n,
                             int32_t *shared_out);

int pkv_seq_length(const pkv_alloc_t *a, int seq, int *num_tokens);
int pkv_seq_num_blocks(const pkv_alloc_t *a, int seq, int *num_blocks);
int pkv_seq_table(const pkv_alloc_t *a, int seq, int32_t *table, int cap,
                  int *num_blocks);
int pkv_block_refcount(const pkv_alloc_t *a, int block, int *refs);
int pkv_block_fill(const pkv_alloc_t *a, int block, int *fill);
int pkv_num_free(const pkv_alloc_t *a, int *num_free);
/* The free list, front first: out [cap]; *n = its length. */
int pkv_free_list(const pkv_alloc_t *a, int32_t *out, int cap, int *n);

/* Give the manager a host pool of num_host_blocks blocks; host_free_order
 * (nullable) as for pkv_alloc_create.  Allowed while no host block is in use
 * (replaces the previous host pool). */
int pkv_alloc_host_pool(pkv_alloc_t *a, int num_host_blocks,
                        const int32_t *host_free_order);
/* Swap out / in n distinct sequences seqs[0..n).  pairs_out [cap][2] receives
 * the (source, destination) pairs, *n_pairs their count; cap must be at least
 * the total table length of the group (else PKV_ERR_INVALID_ARG, nothing
 * changed). */
int pkv_swap_out(pkv_alloc_t *a, const int32_t *seqs, int n, int32_t *pairs_out,
                 int cap, int *n_pairs);
int pkv_swap_in(pkv_alloc_t *a, const int32_t *seqs, int n, int32_t *pairs_out,
                int cap, int *n_pairs);
int pkv_seq_swapped(const pkv_alloc_t *a, int seq, int *swapped);
int pkv_host_block_refcount(const pkv_alloc_t *a, int block, int *refs);
int pkv_host_block_fill(const pkv_alloc_t *a, int block, int *fill);
int pkv_num_free_host(const pkv_alloc_t *a, int *num_free);
int pkv_host_free_list(const pkv_alloc_t *a, int32_t *out, int cap, int *n);

/*
 * Checkpoint of the block manager: its whole state as a byte blob, and an
 * object rebuilt from one.  The KV contents are the caller's device (or
 * pinned host) memory and are not part of it; a blob restores the tables
 * that index them.
 *
 * pkv_alloc_save: *bytes (required) receives the blob's size.  buf == NULL
 *   asks for the size only (PKV_OK).  Otherwise cap must be >= that size
 *   (else PKV_ERR_INVALID_ARG, nothing written) and the blob is written to
 *   buf (host memory, caller-owned).
 * pkv_alloc_load: builds a new object from `bytes` bytes at buf and stores
 *   it in *out (destroy it with pkv_alloc_destroy).  The restored object is
 *   indistinguishable from the saved one: same free-list orders, counts,
 *   fills, sequence ids (the next new id included), swap states and tables,
 *   so every later call gives the same results on both.
 *
 * Blob format (version 1), every field a little-endian int32 unless noted:
 *   magic 0x41564B50 ("PKVA" in memory), version, num_blocks, block_size,
 *   num_host_blocks, number of sequence ids handed out (M);
 *   device free list: its length F, then F block ids in FIFO order;
 *   device fills: num_blocks entries;
 *   host free list: length, then ids in FIFO order; host fills:
 *   num_host_blocks entries;
 *   M sequence records: flags (bit 0 alive, bit 1 swapped out), table
 *   length L, then L block ids (host block ids when swapped out).
 * Reference counts are not stored: they are the number of table entries
 * naming each block.  A blob is accepted only if it is a state the rules
 * above can reach: fields in range, every block either free (count 0, fill
 * 0, listed once) or held, every block but a table's last one full, a last
 * block holding 1..block_size tokens, no table or swap flag on a released
 * id, and no bytes left over.  Anything else returns PKV_ERR_INVALID_ARG
 * and leaves *out untouched.
 */
int pkv_alloc_save(const pkv_alloc_t *a, void *buf, size_t cap, size_t *bytes);
int pkv_alloc_load(const void *buf, size_t bytes, pkv_alloc_t **out);

/* ------------------------------------------------------------------------ */
/* Self-test                                                                 */
/* ------------------------------------------------------------------------ */

/*
 * Launches one CTA that waits, with the same bounded mbarrier wait the decode
 * kernel uses, on a barrier that nothing ever completes, giving up after
 * limit_ns nanoseconds.  The kernel then writes PKV_ERR_DEVICE_TIMEOUT to
 * dev_status and returns normally.  Lets a test check the give-up path
 * without a hang.  limit_ns must be in [1e3, 1e9].
 */
int pkv_selftest_wait_timeout(int32_t *dev_status, uint64_t limit_ns,
                              pkv_stream_t stream);

/*
 * The chunk attention's bounded waits.
 *
 * pkv_selftest_chunk_waits launches one CTA that waits, with the kernel's own
 * limits, for a barrier that nothing completes (one warp) and for a counter
 * that nothing advances (another).  It writes how long each took to give up,
 * in nanoseconds, to elapsed_ns[0] and [1] (device) and
 * PKV_ERR_DEVICE_TIMEOUT to dev_status, and returns normally after two
 * seconds or so.
 *
 * pkv_selftest_chunk_give_up is pkv_paged_attention_chunk with waits that give
 * up after wait_tries failed tries (0 to 2^19, a try takes one to
 * four microseconds): with a few of them the kernel gives up in mid-work, leaves
 * out unspecified, writes PKV_ERR_DEVICE_TIMEOUT to dev_status and returns
 * normally.
 */
int pkv_selftest_chunk_waits(int32_t *dev_status, uint64_t *elapsed_ns,
                             pkv_stream_t stream);
int pkv_selftest_chunk_give_up(void *out, const void *query,
                               const void *key_cache, const void *value_cache,
                               const int32_t *block_tables, int max_blocks_per_seq,
                               const int32_t *context_lens, const int32_t *query_starts,
                               int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               float scale, int causal, int window, int num_ctas,
                               void *workspace, size_t workspace_bytes,
                               int32_t *dev_status, pkv_stream_t stream, int wait_tries);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
