// pkv_team.cu -- host entry points of the team decode (the kernels are in
// pkv_team_impl.cuh): the 8-bit cache's decode and the decode over listed blocks.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "../../include/pkv.h"
#include "pkv_host.h"
#include "pkv_launch.h"
#include "pkv_team_impl.cuh"

namespace pkv {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxCtas = 4096;
constexpr int kMaxKvHeads = 1 << 16;

bool shape_ok(int num_heads, int num_kv_heads, int head_dim) {
    return num_heads > 0 && num_kv_heads > 0 && num_kv_heads <= kMaxKvHeads && num_heads % num_kv_heads == 0 &&
           num_heads / num_kv_heads <= kTeamMaxGroup && (head_dim == 64 || head_dim == 128);
}

// Shared memory of an SM, and what a CTA takes of it besides its dynamic part.
constexpr size_t kSmemOfSm = 228 * 1024, kSmemOfCta = 1024 + 256;

int multiprocessors(int *n) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

int decode(void *out, const void *query, const void *key_cache, const void *value_cache, const float *key_scale,
           const float *value_scale, int scale_stride, const int32_t *block_tables, int max_blocks_per_seq,
           const int32_t *context_lens, const int32_t *selected, const int32_t *num_selected, int max_selected,
           int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
           int cache_type, float scale, int num_ctas, void *workspace, size_t workspace_bytes, int32_t *dev_status,
           pkv_stream_t stream) {
    if (num_seqs == 0) return PKV_OK;
    if (num_seqs < 0 || num_seqs > kMaxSeqs || max_blocks_per_seq < 1 || num_blocks < 1 || num_ctas < 0 ||
        num_ctas > kMaxCtas || block_size < 1 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads)
        return PKV_ERR_INVALID_ARG;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (cache_type != PKV_CACHE_F16 && (!key_scale || !value_scale || scale_stride < num_kv_heads))
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_ERR_INVALID_ARG;
    if (!selected != !num_selected || (selected && max_selected < 1)) return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > (1 << 30)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads > (INT64_C(1) << 31) / block_size) return PKV_ERR_INVALID_ARG;
    if (!shape_ok(num_heads, num_kv_heads, head_dim)) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return PKV_ERR_UNSUPPORTED;
    const int group = num_heads / num_kv_heads;
    const TeamKernel k = cache_type == PKV_CACHE_F16    ? team_kernel_f16(head_dim, group)
                         : cache_type == PKV_CACHE_INT8 ? team_kernel_int8(head_dim, group)
                                                        : team_kernel_e4m3(head_dim, group);
    const size_t smem = k.smem_fixed + 8 * (size_t)num_seqs;
    if (num_ctas == 0) {
        if (multiprocessors(&num_ctas) != PKV_OK) return PKV_ERR_CUDA;
        num_ctas *= std::max(1, std::min(k.ctas_per_sm, (int)(kSmemOfSm / (smem + kSmemOfCta))));
    }
    const TeamWorkspace ws = TeamWorkspace::plan(num_ctas, group, head_dim);
    if (workspace_bytes < ws.total) return PKV_ERR_INVALID_ARG;

    unsigned char *wsb = static_cast<unsigned char *>(workspace);
    TeamParams p = {};
    p.out = static_cast<__half *>(out);
    p.query = static_cast<const __half *>(query);
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.key_scale = key_scale;
    p.value_scale = value_scale;
    p.scale_stride = scale_stride;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.selected = selected;
    p.num_selected = num_selected;
    p.cut = reinterpret_cast<int2 *>(wsb);
    p.part_ml = reinterpret_cast<float2 *>(wsb + ws.ml);
    p.part_o = reinterpret_cast<float *>(wsb + ws.o);
    p.status = dev_status;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_selected = selected ? max_selected : 0;
    p.num_blocks = num_blocks;
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)

    const int rc = ensure_smem_attr(k.fn, smem);
    if (rc != PKV_OK) return rc;
    void *args[] = {&p};
    if (launch_pdl(k.fn, dim3((unsigned)num_ctas), dim3((unsigned)k.threads), smem, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    // No segment is long enough to be cut: nothing to join.
    const int64_t most = team_rows((int64_t)max_blocks_per_seq * block_size, p.block_shift, selected ? max_selected : -1);
    if (num_ctas == 1 || team_steps(most, k.step_rows) <= 2 * kTeamSnap) return PKV_OK;
    const void *join = head_dim == 64 ? reinterpret_cast<const void *>(&team_join_kernel<64>)
                                      : reinterpret_cast<const void *>(&team_join_kernel<128>);
    if (launch_pdl(join, dim3((unsigned)num_ctas, (unsigned)group), dim3(kTeamJoinThreads), 0, stream, args) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_decode_team_workspace_size(int num_heads, int num_kv_heads, int head_dim, int num_ctas) {
    if (num_ctas < 0 || num_ctas > kMaxCtas || !shape_ok(num_heads, num_kv_heads, head_dim)) return 0;
    if (num_ctas == 0) {
        if (multiprocessors(&num_ctas) != PKV_OK) return 0;
        num_ctas *= 2;  // the most that the default is
    }
    return TeamWorkspace::plan(num_ctas, num_heads / num_kv_heads, head_dim).total;
}

extern "C" int pkv_paged_attention_decode_q8(void *out, const void *query, const void *key_cache,
                                             const void *value_cache, const float *key_scale,
                                             const float *value_scale, int scale_stride,
                                             const int32_t *block_tables, int max_blocks_per_seq,
                                             const int32_t *context_lens,
                                             const int32_t *selected, const int32_t *num_selected, int max_selected,
                                             int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                             int block_size, int num_blocks, int cache_type, float scale,
                                             int num_ctas, void *workspace, size_t workspace_bytes,
                                             int32_t *dev_status, pkv_stream_t stream) {
    if (cache_type != PKV_CACHE_INT8 && cache_type != PKV_CACHE_E4M3) return PKV_ERR_INVALID_ARG;
    return decode(out, query, key_cache, value_cache, key_scale, value_scale, scale_stride, block_tables,
                  max_blocks_per_seq, context_lens, selected, num_selected, max_selected, num_seqs, num_heads, num_kv_heads, head_dim,
                  block_size, num_blocks, cache_type, scale, num_ctas, workspace, workspace_bytes, dev_status, stream);
}

extern "C" int pkv_paged_attention_decode_selected(void *out, const void *query, const void *key_cache,
                                                   const void *value_cache, const int32_t *block_tables,
                                                   int max_blocks_per_seq, const int32_t *context_lens,
                                                   const int32_t *selected, const int32_t *num_selected,
                                                   int max_selected, int num_seqs, int num_heads, int num_kv_heads,
                                                   int head_dim, int block_size, int num_blocks, float scale,
                                                   int num_ctas, void *workspace, size_t workspace_bytes,
                                                   int32_t *dev_status, pkv_stream_t stream) {
    if (num_seqs > 0 && !selected) return PKV_ERR_INVALID_ARG;
    return decode(out, query, key_cache, value_cache, nullptr, nullptr, 0, block_tables, max_blocks_per_seq,
                  context_lens, selected, num_selected, max_selected, num_seqs, num_heads, num_kv_heads, head_dim,
                  block_size, num_blocks, PKV_CACHE_F16, scale, num_ctas, workspace, workspace_bytes, dev_status,
                  stream);
}
