// pkv_chunk.cu -- attention of each sequence's newest tokens over its paged
// cache: host entry points and kernel.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxCtas = 4096;
constexpr int kMaxGroup = 16;

struct ChunkParams {
    __half *out;
    const __half *query;
    const __half *key_cache;
    const __half *value_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_starts;
    int32_t *status;
    int num_tokens;
    int num_seqs;
    int num_heads;
    int num_kv_heads;
    int max_blocks_per_seq;
    int num_blocks;
    int block_size;
    int causal;
    int window;
    float scale_log2;
};

// One warp per (row, head): the softmax's running maximum and sum over the
// visible positions, one key at a time.
template <int D>
__global__ void __launch_bounds__(128) chunk_rows_kernel(const __grid_constant__ ChunkParams p) {
    grid_dependency_wait();
    launch_dependents();
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32;
    const int64_t total = (int64_t)p.num_tokens * p.num_heads;
    for (int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 32; w < total; w += (int64_t)gridDim.x * 4) {
        const int row = (int)(w / p.num_heads), head = (int)(w - (int64_t)row * p.num_heads);
        const int kvh = head / (p.num_heads / p.num_kv_heads);
        int seq = -1, lo = 0, hi = 0;
        for (int s = 0; s < p.num_seqs; ++s) {
            int a = p.query_starts[s], b = p.query_starts[s + 1];
            if (a < 0 || b < a || b > p.num_tokens) {
                if (w == 0 && lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
                a = min(max(a, 0), p.num_tokens);
                b = min(max(b, a), p.num_tokens);
            }
            if (row >= a && row < b) {
                seq = s;
                lo = a;
                hi = b;
            }
        }
        if (seq < 0) continue;
        int len = p.context_lens[seq];
        if (len < 0 || len > p.max_blocks_per_seq * p.block_size) {
            if (lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
            len = min(max(len, 0), p.max_blocks_per_seq * p.block_size);
        }
        int t0 = 0, t1 = len;
        if (p.causal) {
            const int pos = len - (hi - lo) + (row - lo);
            t1 = max(pos + 1, 0);
            if (p.window) t0 = max(0, pos - p.window + 1);
        }
        float q[E], acc[E] = {};
        const int64_t at = ((int64_t)row * p.num_heads + head) * D + lane * E;
#pragma unroll
        for (int k = 0; k < E; ++k) q[k] = __half2float(p.query[at + k]) * p.scale_log2;
        float top = -INFINITY, sum = 0.f;
        for (int t = t0; t < t1; ++t) {
            int blk = p.block_tables[(int64_t)seq * p.max_blocks_per_seq + t / p.block_size];
            if (blk < 0 || blk >= p.num_blocks) {
                if (lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
                blk = 0;
            }
            const int64_t kv = (((int64_t)blk * p.num_kv_heads + kvh) * p.block_size + t % p.block_size) * D + lane * E;
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < E; ++k) dot = fmaf(q[k], __half2float(p.key_cache[kv + k]), dot);
#pragma unroll
            for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFullMask, dot, d);
            const float next = fmaxf(top, dot);
            const float base = next == -INFINITY ? 0.f : next;  // nothing but -inf (or NaN) yet
            const float fade = exp2f(top - base);
            const float weight = exp2f(dot - base);
            sum = sum * fade + weight;
#pragma unroll
            for (int k = 0; k < E; ++k) acc[k] = acc[k] * fade + weight * __half2float(p.value_cache[kv + k]);
            top = next;
        }
#pragma unroll
        for (int k = 0; k < E; ++k) p.out[at + k] = __float2half_rn(t1 > t0 ? acc[k] / sum : 0.f);
    }
}

bool shape_ok(int num_heads, int num_kv_heads, int head_dim) {
    return num_heads > 0 && num_kv_heads > 0 && num_heads % num_kv_heads == 0 &&
           num_heads / num_kv_heads <= kMaxGroup && (head_dim == 64 || head_dim == 128);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_chunk_workspace_size(int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                           int num_ctas) {
    if (num_tokens < 0 || num_ctas < 0 || num_ctas > kMaxCtas || !shape_ok(num_heads, num_kv_heads, head_dim))
        return 0;
    return 256;
}

extern "C" int pkv_paged_attention_chunk(void *out, const void *query, const void *key_cache,
                                         const void *value_cache, const int32_t *block_tables,
                                         int max_blocks_per_seq, const int32_t *context_lens,
                                         const int32_t *query_starts, int num_tokens, int num_seqs, int num_heads,
                                         int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                                         int causal, int window, int num_ctas, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, pkv_stream_t stream) {
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
    const size_t need = pkv_chunk_workspace_size(num_tokens, num_heads, num_kv_heads, head_dim, num_ctas);
    if (need == 0) return PKV_ERR_CUDA;
    if (workspace_bytes < need) return PKV_ERR_INVALID_ARG;

    ChunkParams p = {};
    p.out = static_cast<__half *>(out);
    p.query = static_cast<const __half *>(query);
    p.key_cache = static_cast<const __half *>(key_cache);
    p.value_cache = static_cast<const __half *>(value_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_starts = query_starts;
    p.status = dev_status;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.causal = causal;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    void *args[] = {&p};
    const void *fn = head_dim == 64 ? reinterpret_cast<const void *>(&chunk_rows_kernel<64>)
                                    : reinterpret_cast<const void *>(&chunk_rows_kernel<128>);
    const int64_t blocks = std::min<int64_t>(((int64_t)num_tokens * num_heads + 3) / 4, 65536);
    if (launch_pdl(fn, dim3((unsigned)blocks), dim3(128), 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
