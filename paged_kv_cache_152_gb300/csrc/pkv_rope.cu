// pkv_rope.cu -- the norm of each query and key head and the position
// rotation, with the keys and values written to their cache slots.
//
// One pass over the data.  With inv = 1 / sqrt(mean(x^2) + eps) a head becomes
// y = x * inv * w, and pair (a, b) of y becomes (a cos - b sin, b cos + a sin).
// Bound by HBM: each element is read once and written once, and the tables
// (cos_sin, slots, positions) are small and shared by a token's heads.
//
// A head is held by LANES = 8, 16 or 32 lanes, 8 elements each, chosen so that a
// lane holds both elements of its four pairs: in the rotated part, where pairs
// are half of it apart, four consecutive elements of each half (8-byte
// accesses, whole sectors across the lanes), elsewhere 8 consecutive ones.
// The sum of squares is a shuffle reduction inside the group.
//
// Measured (8192 tokens, 32 query and 8 KV heads of 128, into the cache): 37.7
// us, 5460 GB/s, 0.80 of the copy bandwidth; what is left is latency (64
// registers, 1024 threads per SM) and 520 instructions per warp and four heads.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_launch.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

// From this many lanes (heads x lanes per head) a lane group takes four heads:
// 64 tokens of 48 heads of 128 (49 thousand lanes) take 2.03 us with one head
// per group and 2.26 with four, 128 tokens 2.65 and 2.33, 8192 tokens 68.7 and
// 37.7; with heads of 64, 128 tokens of 48 heads 2.04 and 2.26, 256 tokens 2.63
// and 2.23.
constexpr int64_t kManyLanes = 65536;

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
    int num_tokens;
    int chunks;  // lane groups a token's heads take: queries, keys, and with a cache values
    int q_chunks, k_chunks;
    int num_heads;
    int num_kv_heads;
    int head_dim;
    int rot_dim;
    int interleaved;
    int max_positions;
    int block_size;
    float eps;
    float inv_dim;  // 1 / head_dim
};

// A lane's 8 elements: four at a, four at b.
template <bool CONSTANT>
__device__ __forceinline__ uint4 load8(const __half *row, int a, int b) {
    const uint2 *pa = reinterpret_cast<const uint2 *>(row + a), *pb = reinterpret_cast<const uint2 *>(row + b);
    const uint2 x = CONSTANT ? __ldg(pa) : *pa, y = CONSTANT ? __ldg(pb) : *pb;
    return make_uint4(x.x, x.y, y.x, y.y);
}

__device__ __forceinline__ void store8(__half *row, int a, int b, const uint4 &v) {
    *reinterpret_cast<uint2 *>(row + a) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2 *>(row + b) = make_uint2(v.z, v.w);
}

// Two packed fp16 values -> a packed pair of fp32, and back (rounded to nearest even).
__device__ __forceinline__ uint64_t widen(uint32_t v) {
    const float2 f = unpack_half2(v);
    return pack2(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
    float x, y;
    unpack2(v, x, y);
    return pack_half2(x, y);
}

// Up to ROWS consecutive heads of one token and one kind (queries, keys or
// values) per lane group: their loads are in flight together, the token's
// angles and the weight are loaded once for all of them, and no branch stands
// between the rows, so that their latencies overlap.
template <int LANES, int ROWS, bool INTERLEAVED>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    const int64_t unit = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const unsigned mask = LANES == 32 ? kFullMask : ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
    const bool live = lane * 8 < p.head_dim;
    const bool halves = !INTERLEAVED && lane < p.rot_dim / 8;
    const int ea = halves ? lane * 4 : lane * 8, eb = halves ? lane * 4 + p.rot_dim / 2 : lane * 8 + 4;
    const int64_t t = unit / p.chunks;
    const int chunk = (int)(unit - t * p.chunks);
    const bool is_q = chunk < p.q_chunks, is_v = chunk >= p.q_chunks + p.k_chunks;
    const int head = (chunk - (is_q ? 0 : is_v ? p.q_chunks + p.k_chunks : p.q_chunks)) * ROWS;
    const int rows = min(ROWS, (is_q ? p.num_heads : p.num_kv_heads) - head);
    grid_dependency_wait();
    launch_dependents();
    if (t >= p.num_tokens) return;
    int64_t pos = 0, slot = 0;
    if (p.positions) pos = __ldg(p.positions + t);
    if (p.key_cache) slot = __ldg(p.slots + t);

    const __half *src = (is_q ? p.query + t * p.query_stride : is_v ? p.value + t * p.value_stride
                                                                    : p.key + t * p.key_stride) +
                        (int64_t)head * p.head_dim;
    uint4 raw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        raw[r] = make_uint4(0, 0, 0, 0);
        if (live && r < rows) raw[r] = load8<false>(src + r * p.head_dim, ea, eb);
    }
    const __half *weight = is_q ? p.query_weight : is_v ? nullptr : p.key_weight;
    uint4 w = make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);  // ones
    if (weight && live) w = load8<true>(weight, ea, eb);

    if (p.positions && (pos < 0 || pos >= p.max_positions)) {
        if (chunk == 0 && lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
        return;
    }
    __half *dst;
    int64_t step = p.head_dim;  // between heads of dst
    if (is_q) {
        dst = p.query_out + t * p.query_out_stride + (int64_t)head * p.head_dim;
    } else if (p.key_cache) {
        if (slot >= p.num_slots && chunk == p.q_chunks && lane == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
        if (slot < 0 || slot >= p.num_slots) return;
        const int64_t blk = slot / p.block_size;
        step = (int64_t)p.block_size * p.head_dim;
        dst = (is_v ? p.value_cache : p.key_cache) + (blk * p.num_kv_heads + head) * step +
              (slot - blk * p.block_size) * p.head_dim;
    } else {
        dst = p.key_out + t * p.key_out_stride + (int64_t)head * p.head_dim;
    }

    if (is_v) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (live && r < rows) store8(dst + r * step, ea, eb, raw[r]);
        return;
    }
    // This lane's four pairs turn by c + i s.
    const bool turns = p.positions && lane < p.rot_dim / 8;
    uint64_t c[2] = {}, s[2] = {}, s_neg[2] = {};
    if (turns) {
        const float *cs = p.cos_sin + pos * p.rot_dim + 4 * lane;
        const float4 x = __ldg(reinterpret_cast<const float4 *>(cs));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(cs + p.rot_dim / 2));
        c[0] = pack2(x.x, x.y), c[1] = pack2(x.z, x.w);
        s[0] = pack2(y.x, y.y), s[1] = pack2(y.z, y.w);
        s_neg[0] = pack2(-y.x, -y.y), s_neg[1] = pack2(-y.z, -y.w);
    }
    float scale[ROWS];
    if (weight) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const uint64_t a = widen(raw[r].x), b = widen(raw[r].y), d = widen(raw[r].z), e = widen(raw[r].w);
            const uint64_t sum = fma2(e, e, fma2(d, d, fma2(b, b, mul2(a, a))));
            float x, y;
            unpack2(sum, x, y);
            scale[r] = x + y;
        }
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) scale[r] += __shfl_xor_sync(mask, scale[r], d, LANES);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) scale[r] = rsqrtf(fmaf(scale[r], p.inv_dim, p.eps));
    }
    const uint64_t wf[4] = {widen(w.x), widen(w.y), widen(w.z), widen(w.w)};
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        uint64_t x[4] = {widen(raw[r].x), widen(raw[r].y), widen(raw[r].z), widen(raw[r].w)};
        if (weight) {
            const uint64_t f = pack2(scale[r], scale[r]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = mul2(mul2(x[k], f), wf[k]);
        }
        if (turns) {
            if (INTERLEAVED) {
                float cf[4], sf[4];
                unpack2(c[0], cf[0], cf[1]), unpack2(c[1], cf[2], cf[3]);
                unpack2(s[0], sf[0], sf[1]), unpack2(s[1], sf[2], sf[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float a, b;
                    unpack2(x[k], a, b);
                    x[k] = fma2(pack2(b, a), pack2(-sf[k], sf[k]), mul2(x[k], pack2(cf[k], cf[k])));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint64_t a = x[k], b = x[2 + k];
                    x[k] = fma2(b, s_neg[k], mul2(a, c[k]));
                    x[2 + k] = fma2(a, s[k], mul2(b, c[k]));
                }
            }
        }
        const uint4 y = make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
        if (live && r < rows) store8(dst + r * step, ea, eb, y);
    }
}

template <int LANES>
const void *rope_kernel(bool many, bool interleaved) {
    if (interleaved)
        return many ? reinterpret_cast<const void *>(&qk_norm_rope_kernel<LANES, 4, true>)
                    : reinterpret_cast<const void *>(&qk_norm_rope_kernel<LANES, 1, true>);
    return many ? reinterpret_cast<const void *>(&qk_norm_rope_kernel<LANES, 4, false>)
                : reinterpret_cast<const void *>(&qk_norm_rope_kernel<LANES, 1, false>);
}

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
    p.num_tokens = num_tokens;
    p.inv_dim = 1.f / (float)p.head_dim;
    const int lanes = p.head_dim <= 64 ? 8 : p.head_dim <= 128 ? 16 : 32;
    const int kinds = p.key_cache ? 2 : 1;
    const bool many = (int64_t)num_tokens * (p.num_heads + kinds * p.num_kv_heads) * lanes >= kManyLanes;
    const bool inter = p.interleaved != 0;
    const int per_group = many ? 4 : 1;
    p.q_chunks = (p.num_heads + per_group - 1) / per_group;
    p.k_chunks = (p.num_kv_heads + per_group - 1) / per_group;
    p.chunks = p.q_chunks + kinds * p.k_chunks;
    const void *fn = lanes == 8    ? rope_kernel<8>(many, inter)
                     : lanes == 16 ? rope_kernel<16>(many, inter)
                                   : rope_kernel<32>(many, inter);
    const int64_t per_block = 256 / lanes;
    const int64_t blocks = ((int64_t)num_tokens * p.chunks + per_block - 1) / per_block;
    if (blocks > INT32_MAX) return PKV_ERR_INVALID_ARG;
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
