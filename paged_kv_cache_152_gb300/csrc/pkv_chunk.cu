// pkv_chunk.cu -- host entry points of the chunk attention (the kernels are in
// pkv_chunk_impl.cuh): argument checks, grid, workspace and tensor maps.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <atomic>

#include "../../include/pkv.h"
#include "pkv_chunk_impl.cuh"
#include "pkv_host.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxCtas = 4096;
constexpr int kMaxGroup = 16;

bool shape_ok(int num_heads, int num_kv_heads, int head_dim) {
    return num_heads > 0 && num_kv_heads > 0 && num_heads % num_kv_heads == 0 &&
           num_heads / num_kv_heads <= kMaxGroup && (head_dim == 64 || head_dim == 128);
}

// Tries of a bounded device wait.  One that fails takes 1.3 to 3.8 us (a suspended
// mbarrier try; kSpinsPerTry looks at a counter, 69 ns each, 3.3 us), so about two
// seconds.
constexpr uint32_t kWaitTries = 1u << 19;
// Units of an item besides its positions: what a piece costs before its first
// step (queries in, output out), in positions.  With 128, 192, 256, 320, 384 of
// them: 64 x 5 tokens over 50 to 900 take 129, 110, 113, 114, 118 us, 28 single
// tokens and 4 prompt chunks 93, 96, 87, 90, 91, a prompt of 4096 tokens 134, 138,
// 137, 139, 139.
constexpr int kOverhead = 256;

// The workspace: records of the items cut between CTAs, the parts' (maximum,
// sum) and outputs.
struct ChunkWorkspace {
    size_t ml, o, total;
    int part_rows;
    static ChunkWorkspace plan(int num_tokens, int group, int head_dim, int ctas) {
        auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        ChunkWorkspace w;
        // one tile's rows, or two tiles'
        w.part_rows = num_tokens <= kChunkRows / group ? num_tokens * group : 2 * kChunkRows;
        w.ml = up(sizeof(ChunkPart) * (size_t)ctas);
        w.o = w.ml + up(sizeof(float2) * 2 * (size_t)ctas * 2 * kChunkRows);
        w.total = w.o + up(sizeof(float) * 2 * (size_t)ctas * w.part_rows * head_dim);
        return w;
    }
};

int default_ctas(int *ctas) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(ctas, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

// The queries as a 3-D tensor [T][H][D], in boxes of 64 dims of one KV head's
// query heads of one tile's tokens.
int encode_query_map(CUtensorMap *map, const void *query, int num_tokens, int num_heads, int head_dim, int group) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return PKV_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)num_heads, (cuuint64_t)num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)num_heads * head_dim * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kChunkRows / group)};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(query), dims, strides, box,
                              elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

// The kernel hands registers from its four helper warps to its softmax warps;
// that must add up to what it is launched with, or it would wait for good.
bool registers_add_up(const void *fn) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, fn) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.numRegs == kChunkLaunchRegs;
}

// A call whose waits give up after wait_tries tries.
int call(void *out, const void *query, const void *key_cache, const void *value_cache, const int32_t *block_tables,
         int max_blocks_per_seq, const int32_t *context_lens, const int32_t *query_starts, int num_tokens,
         int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
         int causal, int window, int num_ctas, void *workspace, size_t workspace_bytes, int32_t *dev_status,
         pkv_stream_t stream, uint32_t wait_tries) {
    if (num_tokens == 0 || num_seqs == 0) return PKV_OK;
    if (num_tokens < 0 || num_seqs < 0 || num_seqs > kMaxSeqs || max_blocks_per_seq < 1 || num_blocks < 1 ||
        num_ctas < 0 || num_ctas > kMaxCtas || block_size < 1)
        return PKV_ERR_INVALID_ARG;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens || !query_starts || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (window < 0 || (window > 0 && !causal)) return PKV_ERR_INVALID_ARG;
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > (1 << 30)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (INT64_C(1) << 31)) return PKV_ERR_INVALID_ARG;
    if (!shape_ok(num_heads, num_kv_heads, head_dim)) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return PKV_ERR_UNSUPPORTED;
    if (num_ctas == 0 && default_ctas(&num_ctas) != PKV_OK) return PKV_ERR_CUDA;
    const int group = num_heads / num_kv_heads;
    const ChunkWorkspace ws = ChunkWorkspace::plan(num_tokens, group, head_dim, num_ctas);
    if (workspace_bytes < ws.total) return PKV_ERR_INVALID_ARG;

    ChunkParams p = {};
    int rc = encode_query_map(&p.tmap_q, query, num_tokens, num_heads, head_dim, group);
    if (rc == PKV_OK)
        rc = encode_cache_map(&p.tmap_k, key_cache, num_blocks, num_kv_heads, block_size, head_dim, block_size, 1);
    if (rc == PKV_OK)
        rc = encode_cache_map(&p.tmap_v, value_cache, num_blocks, num_kv_heads, block_size, head_dim, block_size, 1);
    if (rc != PKV_OK) return rc;
    unsigned char *wsb = static_cast<unsigned char *>(workspace);
    p.out = static_cast<__half *>(out);
    p.value_cache = static_cast<const __half *>(value_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_starts = query_starts;
    p.parts = reinterpret_cast<ChunkPart *>(wsb);
    p.part_ml = reinterpret_cast<float2 *>(wsb + ws.ml);
    p.part_o = reinterpret_cast<float *>(wsb + ws.o);
    p.status = dev_status;
    p.shape.tile_tokens = kChunkRows / group;
    p.shape.num_kv_heads = num_kv_heads;
    p.shape.causal = causal != 0;
    p.shape.window = std::min(window, 1 << 30);  // no context is longer
    p.shape.overhead = kOverhead;
    p.shape.quantum_shift = 0;  // the kernel goes by the share
    p.fits_32 = chunk_fits_32(p.shape, num_tokens, num_seqs, (int64_t)max_blocks_per_seq * block_size);
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.group = group;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
    p.part_rows = ws.part_rows;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    p.wait_tries = wait_tries;

    const bool d64 = head_dim == 64;
    const void *fn = d64 ? reinterpret_cast<const void *>(&chunk_kernel<64>)
                         : reinterpret_cast<const void *>(&chunk_kernel<128>);
    const size_t smem = d64 ? ChunkConfig<64>::kSmem : ChunkConfig<128>::kSmem;
    static std::atomic<bool> good_regs{false};  // only a good answer is kept: a query may fail once
    if (!good_regs) {
        if (!registers_add_up(reinterpret_cast<const void *>(&chunk_kernel<64>)) ||
            !registers_add_up(reinterpret_cast<const void *>(&chunk_kernel<128>)))
            return PKV_ERR_CUDA;
        good_regs = true;
    }
    rc = ensure_smem_attr(fn, smem);
    if (rc != PKV_OK) return rc;
    void *args[] = {&p};
    if (launch_pdl(fn, dim3((unsigned)num_ctas), dim3(kChunkThreads), smem, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    // No table is long enough for an item to be cut: nothing to join.
    if ((int64_t)max_blocks_per_seq * block_size <= kChunkTile || num_ctas == 1) return PKV_OK;
    fn = d64 ? reinterpret_cast<const void *>(&chunk_join_kernel<64>)
             : reinterpret_cast<const void *>(&chunk_join_kernel<128>);
    if (launch_pdl(fn, dim3((unsigned)num_ctas, (unsigned)(ws.part_rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0,
                   stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_chunk_workspace_size(int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                           int num_ctas) {
    if (num_tokens < 0 || num_ctas < 0 || num_ctas > kMaxCtas || !shape_ok(num_heads, num_kv_heads, head_dim))
        return 0;
    if (num_ctas == 0 && default_ctas(&num_ctas) != PKV_OK) return 0;
    return ChunkWorkspace::plan(num_tokens, num_heads / num_kv_heads, head_dim, num_ctas).total;
}

extern "C" int pkv_paged_attention_chunk(void *out, const void *query, const void *key_cache,
                                         const void *value_cache, const int32_t *block_tables,
                                         int max_blocks_per_seq, const int32_t *context_lens,
                                         const int32_t *query_starts, int num_tokens, int num_seqs, int num_heads,
                                         int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                         float scale, int causal, int window, int num_ctas, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, pkv_stream_t stream) {
    return call(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens, query_starts,
                num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, causal, window,
                num_ctas, workspace, workspace_bytes, dev_status, stream, kWaitTries);
}

extern "C" int pkv_selftest_chunk_give_up(void *out, const void *query, const void *key_cache,
                                          const void *value_cache, const int32_t *block_tables,
                                          int max_blocks_per_seq, const int32_t *context_lens,
                                          const int32_t *query_starts, int num_tokens, int num_seqs, int num_heads,
                                          int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                          float scale, int causal, int window, int num_ctas, void *workspace,
                                          size_t workspace_bytes, int32_t *dev_status, pkv_stream_t stream,
                                          int wait_tries) {
    if (wait_tries < 0 || (uint32_t)wait_tries > kWaitTries) return PKV_ERR_INVALID_ARG;
    return call(out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens, query_starts,
                num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, causal, window,
                num_ctas, workspace, workspace_bytes, dev_status, stream, (uint32_t)wait_tries);
}

extern "C" int pkv_selftest_chunk_waits(int32_t *dev_status, uint64_t *elapsed_ns, pkv_stream_t stream) {
    if (!dev_status || !elapsed_ns) return PKV_ERR_INVALID_ARG;
    chunk_waits_selftest_kernel<<<1, 64, 0, reinterpret_cast<cudaStream_t>(stream)>>>(dev_status, elapsed_ns, kWaitTries);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
