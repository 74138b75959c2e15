// pkv_rope.cu -- the norm of each query and key head and the position
// rotation, with the keys and values written to their cache slots.
//
// One pass over the data.  With inv = 1 / sqrt(mean(x^2) + eps) a head becomes
// y = x * inv * w, and pair (a, b) of y becomes (a cos - b sin, b cos + a sin).
// Bound by HBM: each element is read once and written once, and the tables
// (cos_sin, slots, positions) are small and shared by a token's heads.
//
// A head is held by LANES = 8, 16 or 32 lanes, 8 elements (16 bytes) each, so
// the sum of squares is a shuffle reduction inside the group and a pair's
// other half is one shuffle away: rot_dim is a multiple of 16, so the halves
// of a rotation start on whole 8-element vectors.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_launch.h"

namespace pkv {
namespace {

struct RopeParams {
    const __half *query;
    const __half *key;
    const __half *value;      // with a cache only
    __half *query_out;
    __half *key_out;          // without a cache only
    __half *key_cache;        // NULL: no cache
    __half *value_cache;
    const int64_t *slots;
    const int64_t *positions;  // NULL: no rotation
    const float *cos_sin;
    const __half *query_weight;  // nullable
    const __half *key_weight;    // nullable
    int32_t *status;
    int64_t query_stride, key_stride, value_stride, query_out_stride, key_out_stride;
    int64_t num_slots;
    int64_t tasks;  // tokens x rows, where rows = query heads + KV heads (+ KV heads of values with a cache)
    int rows;
    int num_heads;
    int num_kv_heads;
    int head_dim;
    int rot_dim;
    int interleaved;
    int max_positions;
    int block_size;
    float eps;
};

template <int LANES>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    grid_dependency_wait();
    launch_dependents();
    constexpr int kGroups = 256 / LANES;
    const int lane = threadIdx.x % LANES;
    const unsigned mask = LANES == 32 ? kFullMask : ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
    const int e0 = lane * 8;
    const bool live = e0 < p.head_dim;
    for (int64_t task = (int64_t)blockIdx.x * kGroups + threadIdx.x / LANES; task < p.tasks;
         task += (int64_t)gridDim.x * kGroups) {
        const int64_t t = task / p.rows;
        const int row = (int)(task - t * p.rows);
        const bool is_q = row < p.num_heads;
        const bool is_k = !is_q && row < p.num_heads + p.num_kv_heads;
        const int64_t pos = p.positions ? __ldg(p.positions + t) : 0;
        if (p.positions && (pos < 0 || pos >= p.max_positions)) {
            if (row == 0 && lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
            continue;
        }
        const __half *src;
        __half *dst;
        if (is_q) {
            src = p.query + t * p.query_stride + (int64_t)row * p.head_dim;
            dst = p.query_out + t * p.query_out_stride + (int64_t)row * p.head_dim;
        } else {
            const int h = is_k ? row - p.num_heads : row - p.num_heads - p.num_kv_heads;
            src = is_k ? p.key + t * p.key_stride : p.value + t * p.value_stride;
            src += (int64_t)h * p.head_dim;
            if (p.key_cache) {
                const int64_t slot = __ldg(p.slots + t);
                if (slot < 0) continue;
                if (slot >= p.num_slots) {
                    if (row == p.num_heads && lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
                    continue;
                }
                const int64_t blk = slot / p.block_size;
                const int64_t off = slot - blk * p.block_size;
                dst = (is_k ? p.key_cache : p.value_cache) +
                      ((blk * p.num_kv_heads + h) * p.block_size + off) * p.head_dim;
            } else {
                dst = p.key_out + t * p.key_out_stride + (int64_t)h * p.head_dim;
            }
        }
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = *reinterpret_cast<const uint4 *>(src + e0);
        if (is_q || is_k) {
            float x[8];
            unpack8(raw, x);
            const __half *w = is_q ? p.query_weight : p.key_weight;
            if (w) {
                float sq = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) sq = fmaf(x[k], x[k], sq);
#pragma unroll
                for (int d = LANES / 2; d; d >>= 1) sq += __shfl_xor_sync(mask, sq, d, LANES);
                const float inv = 1.f / sqrtf(sq / (float)p.head_dim + p.eps);
                float wf[8] = {};
                if (live) unpack8(__ldg(reinterpret_cast<const uint4 *>(w + e0)), wf);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = x[k] * inv * wf[k];
            }
            if (p.positions) {
                const float *cs = p.cos_sin + pos * p.rot_dim;
                const int half = p.rot_dim / 2;
                if (p.interleaved) {
                    if (e0 < p.rot_dim) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float c = __ldg(cs + e0 / 2 + k), s = __ldg(cs + half + e0 / 2 + k);
                            const float a = x[2 * k], b = x[2 * k + 1];
                            x[2 * k] = a * c - b * s;
                            x[2 * k + 1] = b * c + a * s;
                        }
                    }
                } else {
                    const int step = half / 8;  // lanes between a pair's halves
                    const bool first = e0 < half;
                    const int peer = first ? lane + step : lane - step;
                    const int i0 = first ? e0 : e0 - half;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float other = __shfl_sync(mask, x[k], peer, LANES);
                        if (e0 < p.rot_dim) {
                            const float c = __ldg(cs + i0 + k), s = __ldg(cs + half + i0 + k);
                            x[k] = first ? x[k] * c - other * s : x[k] * c + other * s;
                        }
                    }
                }
            }
            raw = pack8(x);
        }
        if (live) *reinterpret_cast<uint4 *>(dst + e0) = raw;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good_stride(int64_t stride, int64_t least) { return stride >= least && stride % 8 == 0; }

// The checks that both calls share, and the launch.
int launch(RopeParams &p, int num_tokens, pkv_stream_t stream) {
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens < 0 || p.num_heads <= 0 || p.num_kv_heads <= 0 || p.head_dim <= 0 || p.head_dim % 8)
        return PKV_ERR_INVALID_ARG;
    if (p.head_dim > 256) return PKV_ERR_UNSUPPORTED;
    if (p.num_heads > (1 << 20) || p.num_kv_heads > (1 << 20)) return PKV_ERR_INVALID_ARG;
    if (p.rot_dim < 0 || p.rot_dim > p.head_dim || p.rot_dim % 16) return PKV_ERR_INVALID_ARG;
    if (!(p.eps >= 0.f) || !isfinite(p.eps)) return PKV_ERR_INVALID_ARG;
    if (!p.query || !p.key || !p.query_out || !aligned16(p.query) || !aligned16(p.key) || !aligned16(p.query_out))
        return PKV_ERR_INVALID_ARG;
    const int64_t q_row = (int64_t)p.num_heads * p.head_dim, k_row = (int64_t)p.num_kv_heads * p.head_dim;
    if (!good_stride(p.query_stride, q_row) || !good_stride(p.query_out_stride, q_row) ||
        !good_stride(p.key_stride, k_row))
        return PKV_ERR_INVALID_ARG;
    if (p.rot_dim) {
        if (!p.positions || !p.cos_sin || !aligned16(p.cos_sin) || p.max_positions < 1) return PKV_ERR_INVALID_ARG;
    } else {
        p.positions = nullptr;
    }
    if (!aligned16(p.query_weight) || !aligned16(p.key_weight)) return PKV_ERR_INVALID_ARG;
    p.rows = p.num_heads + p.num_kv_heads * (p.key_cache ? 2 : 1);
    p.tasks = (int64_t)num_tokens * p.rows;
    const int lanes = p.head_dim <= 64 ? 8 : p.head_dim <= 128 ? 16 : 32;
    const void *fn = lanes == 8    ? reinterpret_cast<const void *>(&qk_norm_rope_kernel<8>)
                     : lanes == 16 ? reinterpret_cast<const void *>(&qk_norm_rope_kernel<16>)
                                   : reinterpret_cast<const void *>(&qk_norm_rope_kernel<32>);
    const int64_t per_block = 256 / lanes;
    const int64_t blocks = std::min<int64_t>((p.tasks + per_block - 1) / per_block, 65536);
    void *args[] = {&p};
    if (launch_pdl(fn, dim3((unsigned)blocks), dim3(256), 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

RopeParams common(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                  const void *key, int64_t key_stride, const int64_t *positions, const float *cos_sin,
                  int max_positions, int rot_dim, int interleaved, const void *query_weight, const void *key_weight,
                  float eps, int num_heads, int num_kv_heads, int head_dim, int32_t *dev_status) {
    RopeParams p = {};
    p.query = static_cast<const __half *>(query);
    p.key = static_cast<const __half *>(key);
    p.query_out = static_cast<__half *>(query_out);
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.query_weight = static_cast<const __half *>(query_weight);
    p.key_weight = static_cast<const __half *>(key_weight);
    p.status = dev_status;
    p.query_stride = query_stride;
    p.key_stride = key_stride;
    p.query_out_stride = query_out_stride;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved;
    p.max_positions = max_positions;
    p.eps = eps;
    return p;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_qk_norm_rope(void *query_out, int64_t query_out_stride, void *key_out, int64_t key_out_stride,
                                const void *query, int64_t query_stride, const void *key, int64_t key_stride,
                                const int64_t *positions, const float *cos_sin, int max_positions, int rot_dim,
                                int interleaved, const void *query_weight, const void *key_weight, float eps,
                                int num_tokens, int num_heads, int num_kv_heads, int head_dim, int32_t *dev_status,
                                pkv_stream_t stream) {
    RopeParams p = common(query_out, query_out_stride, query, query_stride, key, key_stride, positions, cos_sin,
                          max_positions, rot_dim, interleaved, query_weight, key_weight, eps, num_heads, num_kv_heads,
                          head_dim, dev_status);
    p.key_out = static_cast<__half *>(key_out);
    p.key_out_stride = key_out_stride;
    if (num_tokens > 0 && (!key_out || !aligned16(key_out) ||
                           !good_stride(key_out_stride, (int64_t)num_kv_heads * head_dim)))
        return PKV_ERR_INVALID_ARG;
    return launch(p, num_tokens, stream);
}

extern "C" int pkv_qk_norm_rope_and_cache(void *query_out, int64_t query_out_stride, const void *query,
                                          int64_t query_stride, const void *key, int64_t key_stride,
                                          const void *value, int64_t value_stride, void *key_cache,
                                          void *value_cache, const int64_t *slot_mapping, const int64_t *positions,
                                          const float *cos_sin, int max_positions, int rot_dim, int interleaved,
                                          const void *query_weight, const void *key_weight, float eps,
                                          int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                          int block_size, int num_blocks, int32_t *dev_status,
                                          pkv_stream_t stream) {
    RopeParams p = common(query_out, query_out_stride, query, query_stride, key, key_stride, positions, cos_sin,
                          max_positions, rot_dim, interleaved, query_weight, key_weight, eps, num_heads, num_kv_heads,
                          head_dim, dev_status);
    p.value = static_cast<const __half *>(value);
    p.value_stride = value_stride;
    p.key_cache = static_cast<__half *>(key_cache);
    p.value_cache = static_cast<__half *>(value_cache);
    p.slots = slot_mapping;
    p.num_slots = (int64_t)num_blocks * block_size;
    p.block_size = block_size;
    if (num_tokens > 0) {
        if (!value || !key_cache || !value_cache || !slot_mapping || block_size <= 0 || num_blocks <= 0)
            return PKV_ERR_INVALID_ARG;
        if (!aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
            !good_stride(value_stride, (int64_t)num_kv_heads * head_dim))
            return PKV_ERR_INVALID_ARG;
    }
    return launch(p, num_tokens, stream);
}
