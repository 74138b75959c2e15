// pkv_select.cu -- the blocks of a context whose keys can score highest.
//
// With hi, lo a block's largest and smallest key channel by channel, no key k of
// the block has q . k above
//
//     sum_i max(q_i hi_i, q_i lo_i) = sum_i max(q_i, 0) hi_i + min(q_i, 0) lo_i,
//
// a product of vectors of 2 D fp16 values: the blocks' bounds (contiguous, hi then
// lo) with (max(q, 0), min(q, 0)), on the tensor cores.  A block's score is the
// largest over its KV head's query heads.
//
// First kernel: the scores in fp32, bound by HBM (4 D bytes per block and head are
// read once, straight into the fragments: the products' inner index is taken in
// the order that 16-byte loads bring it).  Second kernel, a CTA per (sequence, KV
// head): the blocks kept.  fp32 scores are off by E or less (below), so blocks
// more than 2 E above the last kept score are kept and those more than 2 E below
// it are not; the few between are scored again in 64 bits and ranked, ties to the
// lowest index, so that the choice does not hang on the order of a sum.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <float.h>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxGroup = 16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTileBlocks = 16;                 // of a warp's product
constexpr int kCtaBlocks = kWarps * kTileBlocks;
// A product of 2 D terms in the tensor cores: an instruction adds 16 products to
// the sum, each cut at 2^-23 of the largest or finer, so 17 x 2^-23 of the terms'
// magnitudes, and at most 16 instructions follow one another: 2^-14.9.
constexpr float kScoreError = 6.103515625e-5f;  // 2^-14
constexpr float kNoNumber = FLT_MAX;            // the score of a block whose product is not finite

struct SelectParams {
    int32_t *selected;
    int32_t *num_selected;
    const __half *query;
    const __half *bounds;         // [NB][Hkv][2][D]
    const int32_t *block_tables;
    const int32_t *context_lens;
    float *score;                 // [N][Hkv][row]
    double *score64;              // [N][Hkv][row]
    float *reach;                 // [N][Hkv][row / 16]: the largest finite |bound| of 16 blocks
    int32_t *status;
    int64_t row;                  // max_blocks_per_seq rounded up to 16
    int num_heads;
    int num_kv_heads;
    int group;
    int max_blocks_per_seq;
    int max_selected;
    int num_blocks;
    int block_shift;
    int first_blocks, last_blocks;
};

__device__ __forceinline__ int select_blocks_of(const SelectParams &p, int s, bool *bad) {
    const int64_t reach = (int64_t)p.max_blocks_per_seq << p.block_shift;
    int len = __ldg(p.context_lens + s);
    *bad = len < 0 || len > reach;
    len = len < 0 ? 0 : len > reach ? (int)reach : len;
    return (len + (1 << p.block_shift) - 1) >> p.block_shift;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) select_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int kLoads = 4 * D / 64;  // 64 bytes of a row per load of four lanes
    grid_dependency_wait();
    launch_dependents();
    const int s = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    bool bad;
    const int count = select_blocks_of(p, s, &bad);
    if (bad && blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
    const int64_t b0 = (int64_t)blockIdx.x * kCtaBlocks + warp * kTileBlocks;
    if (b0 >= count || count <= p.max_selected) return;

    uint4 x[2][kLoads];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t block = min(b0 + g + 8 * r, (int64_t)count - 1);  // a row past the end repeats the last
        int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + block);
        if (phys < 0 || phys >= p.num_blocks) {
            if (t == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
            phys = 0;
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + ((int64_t)phys * p.num_kv_heads + kvh) * 2 * D);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) x[r][i] = __ldg(src + i * 4 + t);
    }
    float acc[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[n][c][0] = acc[n][c][1] = acc[n][c][2] = acc[n][c][3] = 0.f;
    const __half *q = p.query + ((int64_t)s * p.num_heads + (int64_t)kvh * p.group) * D;
    const __half2 zero = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        // the first half of the loads are hi, for max(q, 0), the others lo, for min(q, 0)
        const int dim = (i * 4 + t) * 8 - (i < kLoads / 2 ? 0 : D);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (n * 8 + g < p.group) raw = __ldg(reinterpret_cast<const uint4 *>(q + (n * 8 + g) * D + dim));
            __half2 *h = reinterpret_cast<__half2 *>(&raw);
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = i < kLoads / 2 ? __hmax2_nan(h[k], zero) : __hmin2_nan(h[k], zero);
            mma_16816(acc[n][0], x[0][i].x, x[1][i].x, x[0][i].y, x[1][i].y, raw.x, raw.y);
            mma_16816(acc[n][1], x[0][i].z, x[1][i].z, x[0][i].w, x[1][i].w, raw.z, raw.w);
        }
    }
    // rows g and g + 8: the largest over the heads 2t, 2t + 1 (+ 8), then over t
    float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = acc[n][0][e] + acc[n][1][e];
            v = fabsf(v) < CUDART_INF_F ? v : kNoNumber;  // not finite
            if (n * 8 + 2 * t + (e & 1) < p.group) best[e >> 1] = fmaxf(best[e >> 1], v);
        }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1)
#pragma unroll
        for (int r = 0; r < 2; ++r) best[r] = fmaxf(best[r], __shfl_xor_sync(kFullMask, best[r], d));
    __half2 top = zero;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const __half2 *h = reinterpret_cast<const __half2 *>(&x[r][i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __hmax2(top, __habs2(h[k]));  // a NaN gives way
        }
    float reach = fminf(fmaxf(__low2float(top), __high2float(top)), 65504.f);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) reach = fmaxf(reach, __shfl_xor_sync(kFullMask, reach, d));
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    if (t == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (b0 + g + 8 * r < count) p.score[seg * p.row + b0 + g + 8 * r] = best[r];
    if (lane == 0) p.reach[(seg * p.row + b0) / kTileBlocks] = reach;
}

// ---- a CTA's sums, maxima and places ----

__device__ __forceinline__ int cta_sum(int v, int *scratch) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += scratch[w];
    return sum;
}

__device__ __forceinline__ float cta_max(float v, float *scratch) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float top = scratch[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, scratch[w]);
    return top;
}

// Threads with a true flag before this one, and how many there are.
__device__ __forceinline__ int cta_place(bool flag, int *scratch, int *total) {
    const unsigned mask = __ballot_sync(kFullMask, flag);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) scratch[warp] = __popc(mask);
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scratch[w];
        sum += scratch[w];
    }
    *total = sum;
    return before + __popc(mask & ((1u << lane) - 1));
}

// Keys in the order of the values.
__device__ __forceinline__ uint32_t order32(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unorder32(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t order64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}

constexpr int kBins = 1024;
constexpr int kList = 256;     // candidates ranked in one step
constexpr int kCached = 8192;  // scores kept in shared memory

// The block's score in 64 bits, by a warp (the same on all lanes).
template <int D>
__device__ double exact_score(const SelectParams &p, int s, int kvh, int64_t block, int lane) {
    int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + block);
    if (phys < 0 || phys >= p.num_blocks) phys = 0;
    const __half *hi = p.bounds + ((int64_t)phys * p.num_kv_heads + kvh) * 2 * D;
    double best = -CUDART_INF;
    for (int h = 0; h < p.group; ++h) {
        const __half *q = p.query + ((int64_t)s * p.num_heads + (int64_t)kvh * p.group + h) * D;
        double sum = 0;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const int i = k * 32 + lane;
            const double v = __half2float(q[i]);
            sum += fmax(v, 0.0) * (double)__half2float(hi[i]) + fmin(v, 0.0) * (double)__half2float(hi[D + i]);
            if (v != v) sum = CUDART_NAN;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        best = fmax(best, fabs(sum) < CUDART_INF ? sum : CUDART_INF);
    }
    return best;
}

// A CTA per (sequence, KV head).
template <int D>
__global__ void __launch_bounds__(kThreads) select_keep_kernel(const __grid_constant__ SelectParams p) {
    __shared__ float cached[kCached];
    __shared__ int bins[kBins];
    __shared__ int scratch[kWarps];
    __shared__ float scratch_f[kWarps];
    __shared__ int list[kList];
    __shared__ double list64[kList];
    __shared__ int list_n, edge[2];
    grid_dependency_wait();
    launch_dependents();
    const int s = blockIdx.y, kvh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    int32_t *out = p.selected + seg * p.max_selected;
    bool bad;
    const int count = select_blocks_of(p, s, &bad);
    const int kept = min(count, p.max_selected);
    if (tid == 0) p.num_selected[seg] = kept;
    if (count <= p.max_selected) {
        for (int i = tid; i < p.max_selected; i += kThreads) out[i] = i < count ? i : -1;
        return;
    }
    // Always kept: the first and the last; `need` of the m blocks between.
    const int m0 = p.first_blocks, m = count - p.first_blocks - p.last_blocks;
    const int need = kept - p.first_blocks - p.last_blocks;
    float *score = p.score + seg * p.row + m0;
    if (m <= kCached) {
        for (int i = tid; i < m; i += kThreads) cached[i] = score[i];
        score = cached;
    }
    // ---- E: the error bound of this row's scores ----
    float size = 0.f, norm = 0.f;
    for (int i = tid; i < (count + kTileBlocks - 1) / kTileBlocks; i += kThreads)
        size = fmaxf(size, p.reach[seg * p.row / kTileBlocks + i]);
    for (int h = warp; h < p.group; h += kWarps) {
        const __half *q = p.query + ((int64_t)s * p.num_heads + (int64_t)kvh * p.group + h) * D;
        float sum = 0.f;
        for (int i = lane; i < D; i += 32) sum += fminf(fabsf(__half2float(q[i])), 65504.f);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        norm = fmaxf(norm, sum);
    }
    size = cta_max(size, scratch_f);
    norm = cta_max(norm, scratch_f);
    const float twice = 2.f * kScoreError * size * norm;

    // ---- the need-th largest fp32 score ----
    float last = CUDART_INF_F;
    bool all_near = false;
    if (need > 0) {
        // A histogram over the finite scores' range finds its bin.
        float top = -CUDART_INF_F, low = -CUDART_INF_F;  // low: of the negated scores
        for (int i = tid; i < m; i += kThreads) {
            const float v = score[i];
            low = fmaxf(low, -v);
            if (v < kNoNumber) top = fmaxf(top, v);
        }
        top = cta_max(top, scratch_f);
        low = -cta_max(low, scratch_f);
        const float per = top > low ? (float)(kBins - 2) / (top - low) : 0.f;
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
        if (tid == 0) list_n = 0;
        __syncthreads();
        auto bin_of = [&](float v) { return v < kNoNumber ? min((int)((v - low) * per), kBins - 2) : kBins - 1; };
        for (int i = tid; i < m; i += kThreads) atomicAdd(bins + bin_of(score[i]), 1);
        __syncthreads();
        if (warp == 0) {  // from the top: the bin in which the count passes `need`
            int above = 0;
            for (int base = kBins - 32; base >= 0; base -= 32) {
                const int n = bins[base + 31 - lane];
                int sum = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int v = __shfl_up_sync(kFullMask, sum, d);
                    if (lane >= d) sum += v;
                }
                const unsigned hit = __ballot_sync(kFullMask, above + sum >= need);
                if (hit) {
                    const int l = __ffs(hit) - 1;
                    if (lane == l) edge[0] = base + 31 - l, edge[1] = above + sum - n;
                    break;
                }
                above += __shfl_sync(kFullMask, sum, 31);
            }
        }
        __syncthreads();
        const int bin = edge[0], rank = need - edge[1], inside = bins[bin];  // the rank-th of the bin, from 1
        if (inside <= kList) {
            for (int i = tid; i < m; i += kThreads)
                if (bin_of(score[i]) == bin) list[atomicAdd(&list_n, 1)] = i;
            __syncthreads();
            if (tid < inside) {
                const float v = score[list[tid]];
                int above = 0, same = 0;
                for (int j = 0; j < inside; ++j) {
                    const float u = score[list[j]];
                    above += u > v;
                    same += u == v;
                }
                if (above < rank && rank <= above + same) scratch_f[0] = v;  // equal values write the same
            }
            __syncthreads();
            last = scratch_f[0];
            __syncthreads();
        } else {  // many alike: its bits one by one
            uint32_t key = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t trial = key | 1u << bit;
                int n = 0;
                for (int i = tid; i < m; i += kThreads) n += order32(score[i]) >= trial;
                if (cta_sum(n, scratch) >= need) key = trial;
            }
            last = unorder32(key);
        }

        // ---- the blocks about the border ----
        int above = 0, near = 0;
        if (tid == 0) list_n = 0;
        for (int i = tid; i < m; i += kThreads) {
            const float v = score[i];
            above += v > last + twice;
            near += v <= last + twice && v >= last - twice;
        }
        above = cta_sum(above, scratch);
        near = cta_sum(near, scratch);
        const int want = need - above;  // of the `near` ones
        if (want < near) {
            if (near <= kList) {
                for (int i = tid; i < m; i += kThreads) {
                    const float v = score[i];
                    if (v <= last + twice && v >= last - twice) list[atomicAdd(&list_n, 1)] = i;
                }
                __syncthreads();
                for (int i = warp; i < near; i += kWarps) {
                    const double v = exact_score<D>(p, s, kvh, m0 + list[i], lane);
                    if (lane == 0) list64[i] = v;
                }
                __syncthreads();
                int mine = -1, before = 0;
                if (tid < near) {
                    mine = list[tid];
                    const double v = list64[tid];
                    for (int j = 0; j < near; ++j)
                        before += list64[j] > v || (list64[j] == v && list[j] < mine);
                }
                __syncthreads();
                if (mine >= 0) score[mine] = before < want ? CUDART_INF_F : -CUDART_INF_F;
            } else {
                double *exact = p.score64 + seg * p.row;
                for (int64_t i = warp; i < m; i += kWarps) {
                    const float v = score[i];
                    if (v <= last + twice && v >= last - twice) {
                        const double e = exact_score<D>(p, s, kvh, m0 + i, lane);
                        if (lane == 0) exact[i] = e;
                    }
                }
                __syncthreads();
                uint64_t key = 0;
                for (int bit = 63; bit >= 0; --bit) {
                    const uint64_t trial = key | 1ull << bit;
                    int n = 0;
                    for (int i = tid; i < m; i += kThreads) {
                        const float v = score[i];
                        if (v <= last + twice && v >= last - twice) n += order64(exact[i]) >= trial;
                    }
                    if (cta_sum(n, scratch) >= want) key = trial;
                }
                int more = 0;  // above the border's value; the first of its equals fill up
                for (int i = tid; i < m; i += kThreads) {
                    const float v = score[i];
                    if (v <= last + twice && v >= last - twice) more += order64(exact[i]) > key;
                }
                int ties = want - cta_sum(more, scratch);
                for (int base = 0; base < m; base += kThreads) {
                    const int i = base + tid;
                    const float v = i < m ? score[i] : 0.f;
                    const bool close = i < m && v <= last + twice && v >= last - twice;
                    const uint64_t e = close ? order64(exact[i]) : 0;
                    int total;
                    const int place = cta_place(close && e == key, scratch, &total);
                    if (close) score[i] = e > key || (e == key && place < ties) ? CUDART_INF_F : -CUDART_INF_F;
                    ties -= min(ties, total);
                }
            }
            __syncthreads();
        }
        all_near = want == near;
    }
    // ---- the list, in ascending order ----
    // (where not all of the border's blocks are kept, infinities mark which are)
    const float bar = all_near ? last - twice : last + twice;
    int at = m0;
    for (int i = tid; i < m0; i += kThreads) out[i] = i;
    for (int base = 0; base < m; base += kThreads) {
        const int i = base + tid;
        const bool keep = i < m && (all_near ? score[i] >= bar : score[i] > bar);
        int total;
        const int place = cta_place(keep, scratch, &total);
        if (keep) out[at + place] = m0 + i;
        at += total;
    }
    for (int i = tid; i < p.last_blocks; i += kThreads) out[kept - p.last_blocks + i] = count - p.last_blocks + i;
}

// Workspace carve-up (byte offsets).  It carries nothing from call to call.
struct SelectWorkspace {
    size_t score, score64, reach, total;
    int64_t row;
    static SelectWorkspace plan(int num_seqs, int num_kv_heads, int max_blocks_per_seq) {
        auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        SelectWorkspace w;
        w.row = ((int64_t)max_blocks_per_seq + kTileBlocks - 1) / kTileBlocks * kTileBlocks;
        const size_t n = (size_t)num_seqs * num_kv_heads * (size_t)w.row;
        w.score = 0;
        w.score64 = up(4 * n);
        w.reach = w.score64 + up(8 * n);
        w.total = w.reach + up(4 * (n / kTileBlocks));
        return w;
    }
};

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_select_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq) {
    if (num_seqs < 0 || num_seqs > kMaxSeqs || num_kv_heads < 1 || num_kv_heads > 65535 || max_blocks_per_seq < 1 ||
        max_blocks_per_seq > (1 << 27))
        return 0;
    return SelectWorkspace::plan(num_seqs, num_kv_heads, max_blocks_per_seq).total;
}

extern "C" int pkv_select_blocks(int32_t *selected, int32_t *num_selected, const void *query, const void *key_bounds,
                                 const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                 int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                 int num_blocks, int max_selected, int first_blocks, int last_blocks,
                                 void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                 pkv_stream_t stream) {
    if (num_seqs == 0) return PKV_OK;
    if (num_seqs < 0 || num_seqs > kMaxSeqs || max_blocks_per_seq < 1 || num_blocks < 1 || num_heads <= 0 ||
        num_kv_heads <= 0 || num_heads % num_kv_heads || block_size < 1)
        return PKV_ERR_INVALID_ARG;
    if (!selected || !num_selected || !query || !key_bounds || !block_tables || !context_lens || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(query) || !aligned16(key_bounds) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_ERR_INVALID_ARG;
    if (max_selected < 1 || first_blocks < 0 || last_blocks < 0 || first_blocks > max_selected ||
        last_blocks > max_selected - first_blocks)
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > (1 << 30)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads > (INT64_C(1) << 31) / block_size) return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || num_heads / num_kv_heads > kMaxGroup || num_kv_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return PKV_ERR_UNSUPPORTED;
    const SelectWorkspace ws = SelectWorkspace::plan(num_seqs, num_kv_heads, max_blocks_per_seq);
    if (workspace_bytes < ws.total) return PKV_ERR_INVALID_ARG;

    unsigned char *wsb = static_cast<unsigned char *>(workspace);
    SelectParams p = {};
    p.selected = selected;
    p.num_selected = num_selected;
    p.query = static_cast<const __half *>(query);
    p.bounds = static_cast<const __half *>(key_bounds);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.score = reinterpret_cast<float *>(wsb + ws.score);
    p.score64 = reinterpret_cast<double *>(wsb + ws.score64);
    p.reach = reinterpret_cast<float *>(wsb + ws.reach);
    p.status = dev_status;
    p.row = ws.row;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_selected = max_selected;
    p.num_blocks = num_blocks;
    p.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
    p.first_blocks = first_blocks;
    p.last_blocks = last_blocks;

    void *args[] = {&p};
    const bool d64 = head_dim == 64, wide = p.group > 8;
    const void *fn = d64 ? (wide ? reinterpret_cast<const void *>(&select_score_kernel<64, 2>)
                                 : reinterpret_cast<const void *>(&select_score_kernel<64, 1>))
                         : (wide ? reinterpret_cast<const void *>(&select_score_kernel<128, 2>)
                                 : reinterpret_cast<const void *>(&select_score_kernel<128, 1>));
    const unsigned tiles = (unsigned)((max_blocks_per_seq + kCtaBlocks - 1) / kCtaBlocks);
    if (launch_pdl(fn, dim3(tiles, (unsigned)num_kv_heads, (unsigned)num_seqs), dim3(kThreads), 0, stream, args) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    fn = d64 ? reinterpret_cast<const void *>(&select_keep_kernel<64>)
             : reinterpret_cast<const void *>(&select_keep_kernel<128>);
    if (launch_pdl(fn, dim3((unsigned)num_kv_heads, (unsigned)num_seqs), dim3(kThreads), 0, stream, args) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
