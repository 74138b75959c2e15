// pkv_select.cu -- the blocks of a context whose keys can score highest.
//
// With hi, lo a block's largest and smallest key channel by channel, no key k of
// the block has q . k above (but for the rounding to fp16 of an 8-bit cache's bounds)
//
//     sum_i max(q_i hi_i, q_i lo_i) = sum_i max(q_i, 0) hi_i + min(q_i, 0) lo_i,
//
// a product of vectors of 2 D fp16 values: the blocks' bounds (contiguous, hi then
// lo) with (max(q, 0), min(q, 0)), on the tensor cores.  A block's score is the
// largest over its KV head's query heads.
//
// The scores are fp32 sums, bound by HBM (4 D bytes per block and head are read
// once, straight into the fragments: the products' inner index is taken in the
// order that 16-byte loads bring it) where there is much of them, and by latency
// where there is little: so one kernel does both parts, a cluster of CTAs per
// (sequence, KV head), and the scores never leave shared memory.  (Tables of more
// than 4096 columns take two kernels, with the scores in global memory.)
//
// The choice: fp32 scores are off by E or less (below), so blocks more than 2 E
// above the last kept score are kept and those more than 2 E below it are not; the
// few between are scored again as whole numbers, without any rounding, and ranked,
// ties to the lowest index, so that the choice is that of the exact scores.
//
// Measured: 8 contexts of 8000 to 32768 tokens, blocks of 32, 8 KV heads 11.7 us (the
// 23 MB of bounds need 3.4 of them; all that comes before the choice, three look-ups
// and two rounds of loads, takes 6.3; the choice is some ten steps of a CTA, each a
// few hundred cycles of latency); 64 contexts of 4000 to 16384, blocks of 16, 40.2 us,
// 4100 GB/s, 0.60 of the copy bandwidth (all CTAs run at once, so the longest contexts'
// end the call; without the choice 34.2).  With the border's scores as pairs of fp32
// values 11.9 and 40.4, but the second one is rounded, so that large terms that cancel
// took the last digits with them and equal scores of other terms differed; as 96-bit
// integers from shifts 12.1 and 40.7; in fp64 and at most 128 keys ranked instead of 32
// 13.2 and 42.2; with as many rounds as the keys have pairs of bits 13.9.  Where one
// channel is 30000 in every block, E is so wide that all are scored again: 317 and 375 us
// (pairs of fp32 values 400 and 493, integers from shifts 575 and 665).  With tables of 4096 columns for the same contexts
// 18.7 and 46.3 us (more scores a thread, larger clusters); of 8192, with the two kernels,
// 36 and 106; 131072 tokens in blocks of 16 of one sequence 82 us, of eight 191.
// Scoring by persistent warps over all segments and choosing in a second kernel took 48
// for the 64; queries in shared memory instead of registers, for six CTAs an SM instead
// of four, 57.
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
constexpr int kTileBlocks = 16;                 // of a warp's product
// A product of 2 D terms in the tensor cores: an instruction adds 16 products to
// the sum, each cut at 2^-23 of the largest or finer, so 17 x 2^-23 of the terms'
// magnitudes, and at most 8 instructions follow one another in each of two sums,
// which are added at the end: 2^-15.9 of the magnitudes of both, and 2^-24.
constexpr float kScoreError = 2.2e-5f;  // 2^-15.5
constexpr float kNoNumber = FLT_MAX;            // the score of a block whose product is not finite

struct SelectParams {
    int32_t *selected;
    int32_t *num_selected;
    const __half *query;
    const __half *bounds;         // [NB][Hkv][2][D]
    const int32_t *block_tables;
    const int32_t *context_lens;
    float *score;                 // [N][Hkv][row]
    int64_t *score_hi;            // [N][Hkv][row]: exact_score's hi (its lo takes score's place)
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

// The fragments of a KV head's queries: 16 bytes of head n * 8 + g at each of the
// places that a lane's loads of a block's bounds cover, with max(q, 0) for the
// first half of the loads, which are hi, and min(q, 0) for the others.
template <int D, int NT>
struct SelectQueries {
    static constexpr int kLoads = 4 * D / 64;  // 64 bytes of a row per load of four lanes
    uint4 q[NT][kLoads];

    __device__ __forceinline__ void load(const SelectParams &p, int64_t seg, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const __half *rows = p.query + seg * p.group * D;
        const __half2 zero = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < kLoads / 2; ++i) {
                uint4 raw = make_uint4(0, 0, 0, 0);
                if (n * 8 + g < p.group)
                    raw = __ldg(reinterpret_cast<const uint4 *>(rows + (n * 8 + g) * D + (i * 4 + t) * 8));
                q[n][i] = q[n][i + kLoads / 2] = raw;
                __half2 *up = reinterpret_cast<__half2 *>(&q[n][i]);
                __half2 *down = reinterpret_cast<__half2 *>(&q[n][i + kLoads / 2]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    up[k] = __hmax2_nan(up[k], zero);
                    down[k] = __hmin2_nan(down[k], zero);
                }
            }
    }
};

// Scores 16 blocks, by a warp: best[r] is that of row g + 8 r (on all four lanes of the row), reach the largest finite
// |bound| (on all lanes).  phys: this lane's rows' physical blocks.
template <int D, int NT>
__device__ __forceinline__ void score_tile(const SelectParams &p, const SelectQueries<D, NT> &queries, const int (&phys)[2],
                                           int kvh, int lane, float (&best)[2], float &reach) {
    constexpr int kLoads = SelectQueries<D, NT>::kLoads;
    const int t = lane & 3;
    uint4 x[2][kLoads];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + ((int64_t)phys[r] * p.num_kv_heads + kvh) * 2 * D);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) x[r][i] = __ldg(src + i * 4 + t);
    }
    float acc[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[n][c][0] = acc[n][c][1] = acc[n][c][2] = acc[n][c][3] = 0.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 q = queries.q[n][i];
            mma_16816(acc[n][0], x[0][i].x, x[1][i].x, x[0][i].y, x[1][i].y, q.x, q.y);
            mma_16816(acc[n][1], x[0][i].z, x[1][i].z, x[0][i].w, x[1][i].w, q.z, q.w);
        }
    // the largest over the heads 2t, 2t + 1 (+ 8), then over t
    best[0] = best[1] = -CUDART_INF_F;
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
    __half2 top = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const __half2 *h = reinterpret_cast<const __half2 *>(&x[r][i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __hmax2(top, __habs2(h[k]));  // a NaN gives way
        }
    const float most = fminf(fmaxf(__low2float(top), __high2float(top)), 65504.f);
    reach = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(most)));
}

// The physical block of block `block` (past the end: the last one's).
__device__ __forceinline__ int select_phys(const SelectParams &p, int s, int64_t block, int count, bool first) {
    int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + min(block, (int64_t)count - 1));
    if (phys < 0 || phys >= p.num_blocks) {
        if (first) report(p.status, PKV_ERR_OUT_OF_RANGE);
        phys = 0;
    }
    return phys;
}

// Tables of more columns than the fused kernel holds blocks: scores to global memory.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) select_score_kernel(const __grid_constant__ SelectParams p) {
    grid_dependency_wait();
    launch_dependents();
    const int s = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    bool bad;
    const int count = select_blocks_of(p, s, &bad);
    if (bad && blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
    const int64_t b0 = ((int64_t)blockIdx.x * (kThreads / 32) + warp) * kTileBlocks;
    if (b0 >= count || count <= p.max_selected) return;
    const int phys[2] = {select_phys(p, s, b0 + g, count, (lane & 3) == 0), select_phys(p, s, b0 + g + 8, count, (lane & 3) == 0)};
    SelectQueries<D, NT> queries;
    queries.load(p, seg, lane);
    float best[2], reach;
    score_tile<D, NT>(p, queries, phys, kvh, lane, best, reach);
    if ((lane & 3) == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (b0 + g + 8 * r < count) p.score[seg * p.row + b0 + g + 8 * r] = best[r];
    if (lane == 0) p.reach[(seg * p.row + b0) / kTileBlocks] = reach;
}

// ---- the blocks kept ----

// Keys in the order of the values.
__device__ __forceinline__ uint32_t order32(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unorder32(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr int kKeepThreads = 128;
constexpr int kKeepWarps = kKeepThreads / 32;
constexpr int kList = 128;  // candidates at the border ranked in one step

struct KeepScratch {
    int sums[2][kKeepWarps][4];  // two sets in turn, so that a sum takes one barrier
    int list[kList];
    int64_t list_hi[kList];
    uint32_t list_lo[kList];
    int keep[kList];
    int list_n;
    int few_n;
    uint32_t few[32], found;
};

// Sums over the CTA of four counts, the same on all threads; `turn` alternates.
__device__ __forceinline__ int4 cta_sums(int4 v, KeepScratch &sh, int &turn) {
    v.x = __reduce_add_sync(kFullMask, v.x);
    v.y = __reduce_add_sync(kFullMask, v.y);
    v.z = __reduce_add_sync(kFullMask, v.z);
    if ((threadIdx.x & 31) == 0) *reinterpret_cast<int4 *>(sh.sums[turn][threadIdx.x >> 5]) = v;
    __syncthreads();
    int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kKeepWarps; ++w) {
        const int4 x = *reinterpret_cast<const int4 *>(sh.sums[turn][w]);
        sum.x += x.x, sum.y += x.y, sum.z += x.z;
    }
    turn ^= 1;
    return sum;
}

// A score, exactly: a product of two fp16 values is a whole number of 2^-48 of 22 bits, and below 2^32 in size, so a sum
// of 128 of them is a whole number of 2^-48 below 2^87: (hi 2^32 + lo) 2^-48.  No order of the sum and no rounding enters,
// so equal scores are equal here.
struct ExactScore {
    int64_t hi;
    uint32_t lo;
};
constexpr int64_t kNoNumberHi = INT64_C(1) << 60;  // above every score: those that are not finite
__device__ __forceinline__ bool exact_above(int64_t hi, uint32_t lo, int64_t hi2, uint32_t lo2) {
    return hi > hi2 || (hi == hi2 && lo > lo2);
}

// An exact product in four parts, whole numbers of 2^10, 2^-13, 2^-36 and 2^-48 up to 2^22 in size, added to a sum: the
// product plus 1.5 2^23 of such a unit is rounded to a whole number of it, which the bits show; what is left of the
// product, at most half a unit, is exact too.
constexpr int kParts = 4;
__device__ __forceinline__ float part_place(int i) {  // 1.5 2^23 units
    return i == 0 ? 0x1.8p33f : i == 1 ? 0x1.8p10f : i == 2 ? 0x1.8p-13f : 0x1.8p-25f;
}
__device__ __forceinline__ void add_parts(uint32_t (&sum)[kParts], float x) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const float y = __fadd_rn(x, part_place(i));
        sum[i] += __float_as_uint(y);
        if (i + 1 < kParts) x = __fsub_rn(x, __fsub_rn(y, part_place(i)));
    }
}

// The physical block of a block that has been scored (a bad entry has been reported).
__device__ __forceinline__ int border_phys(const SelectParams &p, int s, int64_t block) {
    const int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + block);
    return phys < 0 || phys >= p.num_blocks ? 0 : phys;
}

// A lane's channels of a block's bounds, lane + 32 k: loaded a block ahead of their use.
template <int D>
struct BorderBounds {
    unsigned short hi[D / 32], lo[D / 32];
    __device__ __forceinline__ void load(const SelectParams &p, int kvh, int phys, int lane) {
        const unsigned short *at = reinterpret_cast<const unsigned short *>(p.bounds) +
                                   ((int64_t)phys * p.num_kv_heads + kvh) * 2 * D + lane;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) hi[k] = __ldg(at + k * 32), lo[k] = __ldg(at + D + k * 32);
    }
};

// The block's score, by a warp; the same on all lanes.
template <int D>
__device__ __forceinline__ ExactScore exact_score(const SelectParams &p, int s, int kvh, const BorderBounds<D> &bounds,
                                                  int lane) {
    bool finite = true;
    float up[D / 32], down[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        finite &= (bounds.hi[k] & 0x7c00) != 0x7c00 && (bounds.lo[k] & 0x7c00) != 0x7c00;
        up[k] = __half2float(__ushort_as_half(bounds.hi[k]));
        down[k] = __half2float(__ushort_as_half(bounds.lo[k]));
    }
    ExactScore best = {-kNoNumberHi, 0};
#pragma unroll 4
    for (int h = 0; h < p.group; ++h) {
        const __half *row = p.query + ((int64_t)s * p.num_heads + (int64_t)kvh * p.group + h) * D;
        uint32_t sum[kParts] = {};
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const float q = __half2float(row[k * 32 + lane]), x = q * (q < 0.f ? down[k] : up[k]);
            finite &= fabsf(x) < CUDART_INF_F;
            add_parts(sum, x);
        }
        int part[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            part[i] = (int)__reduce_add_sync(kFullMask, sum[i] - D / 32 * __float_as_uint(part_place(i)));
        // hi 2^32 + lo of the parts times 2^58, 2^35, 2^12 and 1
        const int64_t low = ((int64_t)part[2] << 12) + part[3];
        const int64_t hi = ((int64_t)part[0] << 26) + ((int64_t)part[1] << 3) + (low >> 32);
        const uint32_t lo = (uint32_t)low;
        if (exact_above(hi, lo, best.hi, best.lo)) best.hi = hi, best.lo = lo;
    }
    // an infinite or missing bound or query times any other makes a sum that is not finite
    if (!__all_sync(kFullMask, finite)) best.hi = kNoNumberHi, best.lo = 0;
    return best;
}

// Twice the error bound of a row's fp32 scores, partly: the largest |bound| of this thread's tiles and the largest
// sum of |q| of this warp's heads.
template <int D>
__device__ __forceinline__ float2 keep_bound(const SelectParams &p, int s, int kvh, const float *reach, int count) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float size = 0.f, norm = 0.f;
    for (int i = tid; i < (count + kTileBlocks - 1) / kTileBlocks; i += kKeepThreads)
        size = fmaxf(size, reach[i]);
    for (int h = warp; h < p.group; h += kKeepWarps) {
        const __half2 *q = reinterpret_cast<const __half2 *>(
            p.query + ((int64_t)s * p.num_heads + (int64_t)kvh * p.group + h) * D);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const float2 v = __half22float2(q[i * 32 + lane]);
            sum += fminf(fabsf(v.x), 65504.f) + fminf(fabsf(v.y), 65504.f);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        norm = fmaxf(norm, sum);
    }
    return make_float2(size, norm);
}

// Any number of blocks, and any number of them alike: the scores stay in global memory.  Marks what is kept of the
// border by infinities and returns the score above which (`all_near`: from which on) blocks are kept.
template <int D>
__device__ float keep_slowly(const SelectParams &p, KeepScratch &sh, int &turn, int s, int kvh, int64_t seg, int m0, int m,
                             int need, float twice, bool *all_near) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *score = p.score + seg * p.row + m0;
    uint32_t top = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = top | 1u << bit;
        int n = 0;
        for (int i = tid; i < m; i += kKeepThreads) n += order32(score[i]) >= trial;
        if (cta_sums(make_int4(n, 0, 0, 0), sh, turn).x >= need) top = trial;
    }
    const float last = unorder32(top);
    auto close = [&](float v) { return v <= last + twice && v >= last - twice; };
    int above = 0, near = 0;
    for (int i = tid; i < m; i += kKeepThreads) {
        above += score[i] > last + twice;
        near += close(score[i]);
    }
    const int4 sums = cta_sums(make_int4(above, near, 0, 0), sh, turn);
    const int want = need - sums.x;
    *all_near = want == sums.y;
    if (*all_near) return last - twice;
    // The border's exact scores; what is surely kept or not is marked.
    int64_t *hi = p.score_hi + seg * p.row;
    constexpr int64_t kMarked = INT64_MIN;
    int64_t highest = kMarked, lowest = INT64_MAX;
    for (int base = warp * 32; base < m; base += kKeepThreads) {
        const int i = base + lane;
        const float v = i < m ? score[i] : 0.f;
        const bool mine = i < m && close(v);
        if (i < m && !mine) {
            hi[i] = kMarked;
            score[i] = v > last ? CUDART_INF_F : -CUDART_INF_F;
        }
        const int phys = mine ? border_phys(p, s, m0 + i) : 0;
        unsigned mask = __ballot_sync(kFullMask, mine);
        BorderBounds<D> next;
        if (mask) next.load(p, kvh, __shfl_sync(kFullMask, phys, __ffs(mask) - 1), lane);
        while (mask) {
            const int b = __ffs(mask) - 1;
            const BorderBounds<D> now = next;
            mask &= mask - 1;
            if (mask) next.load(p, kvh, __shfl_sync(kFullMask, phys, __ffs(mask) - 1), lane);
            const ExactScore e = exact_score<D>(p, s, kvh, now, lane);
            highest = max(highest, e.hi);
            lowest = min(lowest, e.hi);
            if (lane == b) {
                hi[i] = e.hi;
                score[i] = __uint_as_float(e.lo);
            }
        }
    }
    if (lane == 0) sh.list_hi[warp] = highest, sh.list_hi[kKeepWarps + warp] = lowest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kKeepWarps; ++w) {
        highest = max(highest, sh.list_hi[w]);
        lowest = min(lowest, sh.list_hi[kKeepWarps + w]);
    }
    // the want-th largest: hi's bits in an unsigned order, past those that are all alike, then lo's among its equals
    constexpr uint64_t kSign = (uint64_t)1 << 63;
    auto key_hi = [&](int i) { return (uint64_t)hi[i] ^ kSign; };  // (marked: 0, below every score)
    const int alike = __clzll(highest ^ lowest);
    uint64_t key = ((uint64_t)highest ^ kSign) & ~(alike < 64 ? ~(uint64_t)0 >> alike : 0);
    for (int bit = 63 - alike; bit >= 0; --bit) {
        const uint64_t trial = key | 1ull << bit;
        int n = 0;
        for (int i = tid; i < m; i += kKeepThreads) n += key_hi(i) >= trial;
        if (cta_sums(make_int4(n, 0, 0, 0), sh, turn).x >= want) key = trial;
    }
    int past = 0, equal = 0;
    for (int i = tid; i < m; i += kKeepThreads) {
        past += key_hi(i) > key;
        equal += key_hi(i) == key;
    }
    const int4 about = cta_sums(make_int4(past, equal, 0, 0), sh, turn);
    past = about.x;
    uint32_t word = 0;  // (all its equals are kept: any lo)
    for (int bit = past + about.y == want ? -1 : 31; bit >= 0; --bit) {
        const uint32_t trial = word | 1u << bit;
        int n = 0;
        for (int i = tid; i < m; i += kKeepThreads) n += key_hi(i) == key && __float_as_uint(score[i]) >= trial;
        if (past + cta_sums(make_int4(n, 0, 0, 0), sh, turn).x >= want) word = trial;
    }
    int more = 0;  // above the border's value; the first of its equals fill up
    for (int i = tid; i < m; i += kKeepThreads) more += key_hi(i) == key && __float_as_uint(score[i]) > word;
    int ties = want - past - cta_sums(make_int4(more, 0, 0, 0), sh, turn).x;
    for (int base = 0; base < m; base += kKeepThreads) {
        const int i = base + tid;
        const uint64_t k = i < m ? key_hi(i) : 0;
        const uint32_t lo = k ? __float_as_uint(score[i]) : 0;
        const unsigned mask = __ballot_sync(kFullMask, k == key && lo == word);
        if (lane == 0) sh.sums[turn][warp][0] = __popc(mask);
        __syncthreads();
        int place = __popc(mask & ((1u << lane) - 1)), total = 0;
        for (int w = 0; w < kKeepWarps; ++w) {
            if (w < warp) place += sh.sums[turn][w][0];
            total += sh.sums[turn][w][0];
        }
        turn ^= 1;
        if (k) {
            const bool keep = k > key || (k == key && (lo > word || (lo == word && place < ties)));
            score[i] = keep ? CUDART_INF_F : -CUDART_INF_F;
        }
        ties -= min(ties, total);
    }
    __syncthreads();
    return 0.f;
}

// A CTA keeps the blocks of one (sequence, KV head) of more than max_selected.  score, reach: its blocks' scores and its
// tiles' reach; thread t holds the scores t, t + 128, ... of up to VALUES * 128 blocks (VALUES 0: any number, in global
// memory).  The need-th largest is found two bits of its key at a time, until at most 32 keys have those bits.
template <int D, int VALUES>
__device__ __forceinline__ void keep_blocks(const SelectParams &p, KeepScratch &sh, int4 *places, int s, int kvh, int count,
                                            const float *score, const float *reach) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    int32_t *out = p.selected + seg * p.max_selected;
    const int kept = p.max_selected;
    // Always kept: the first and the last; `need` of the m blocks between.
    const int m0 = p.first_blocks, m = count - p.first_blocks - p.last_blocks;
    const int need = kept - p.first_blocks - p.last_blocks;
    for (int i = tid; i < m0; i += kKeepThreads) out[i] = i;
    for (int i = tid; i < p.last_blocks; i += kKeepThreads) out[kept - p.last_blocks + i] = count - p.last_blocks + i;
    if (need == 0) return;
    int turn = 0;
    if (tid == 0) sh.list_n = sh.few_n = 0;

    float v[VALUES < 1 ? 1 : VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) {
        const int i = j * kKeepThreads + tid;
        v[j] = i < m ? score[m0 + i] : -CUDART_INF_F;
    }
    // the row's error bound, and the keys' leading bits that are all alike
    uint32_t high = 0, low = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < VALUES; ++j)
        if (j * kKeepThreads + tid < m) {
            high = max(high, order32(v[j]));
            low = min(low, order32(v[j]));
        }
    {
        const float2 part = keep_bound<D>(p, s, kvh, reach, count);
        const int4 mine = make_int4((int)__reduce_max_sync(kFullMask, __float_as_uint(part.x)), __float_as_int(part.y),
                                    (int)__reduce_max_sync(kFullMask, high), (int)__reduce_min_sync(kFullMask, low));
        if (lane == 0) *reinterpret_cast<int4 *>(sh.sums[turn][warp]) = mine;
    }
    __syncthreads();
    float size = 0.f, norm = 0.f;
#pragma unroll
    for (int w = 0; w < kKeepWarps; ++w) {
        const int4 x = *reinterpret_cast<const int4 *>(sh.sums[turn][w]);
        size = fmaxf(size, __int_as_float(x.x));
        norm = fmaxf(norm, __int_as_float(x.y));
        high = max(high, (uint32_t)x.z);
        low = min(low, (uint32_t)x.w);
    }
    turn ^= 1;
    const float twice = 2.f * kScoreError * size * norm;

    bool all_near = false;
    float bar;  // what is above it is kept (all_near: from it on)
    if constexpr (VALUES > 0) {
        // ---- the need-th largest key ----
        const int same = __clz(high ^ low) & ~1;  // leading bits, an even number (32: all)
        uint32_t key = same == 0 ? 0 : high & ~(uint32_t)((1ull << (32 - same)) - 1);
        int bit = 30 - same, above = 0, within = m;  // keys past key + 2^(bit + 2), and from key up to it
        for (; bit >= 0 && within > 32; bit -= 2) {
            const uint32_t one = key + (1u << bit), two = key + (2u << bit), three = key + (3u << bit);
            int4 n = make_int4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                const uint32_t k = order32(v[j]);
                n.x += k >= one;
                n.y += k >= two;
                n.z += k >= three;
            }
            n = cta_sums(n, sh, turn);
            const int all = above + within;
            key = n.z >= need ? three : n.y >= need ? two : n.x >= need ? one : key;
            within = n.z >= need ? n.z - above : n.y >= need ? n.y - n.z : n.x >= need ? n.x - n.y : all - n.x;
            above = n.z >= need ? above : n.y >= need ? n.z : n.x >= need ? n.y : n.x;
        }
        if (bit >= 0) {  // few are left: ranked
            const uint32_t span = (uint32_t)((4ull << bit) - 1);
            uint32_t mine = 0;
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (j * kKeepThreads + tid < m && order32(v[j]) - key <= span) mine |= 1u << j;
            if (mine) {
                int at = atomicAdd(&sh.few_n, __popc(mine));
#pragma unroll
                for (int j = 0; j < VALUES; ++j)
                    if (mine >> j & 1) sh.few[at++] = order32(v[j]);
            }
            __syncthreads();
            if (warp == 0 && lane < sh.few_n) {
                const uint32_t k = sh.few[lane];
                int more = above, alike = 0;
                for (int j = 0; j < sh.few_n; ++j) {
                    more += sh.few[j] > k;
                    alike += sh.few[j] == k;
                }
                if (more < need && more + alike >= need) sh.found = k;
            }
            __syncthreads();
            key = sh.found;
        }
        const float last = unorder32(key);
        // ---- the blocks about the border ----
        int4 n = make_int4(0, 0, 0, 0);
        uint32_t close = 0;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            n.x += v[j] > last + twice;
            if (v[j] <= last + twice && v[j] >= last - twice) close |= 1u << j;
        }
        const int closes = __popc(close);
        n.y = closes;
        n = cta_sums(n, sh, turn);
        const int want = need - n.x;
        all_near = want == n.y;
        bar = all_near ? last - twice : last + twice;
        if (!all_near && n.y <= kList) {
            const int at = closes ? atomicAdd(&sh.list_n, closes) : 0;
            int k = at;
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (close >> j & 1) sh.list[k++] = j * kKeepThreads + tid;
            __syncthreads();
            // a lane looks up one of the warp's (at most 32)
            const int ours = warp + lane * kKeepWarps;
            const int phys = ours < n.y ? border_phys(p, s, m0 + sh.list[ours]) : 0;
            BorderBounds<D> next;
            if (warp < n.y) next.load(p, kvh, __shfl_sync(kFullMask, phys, 0), lane);
            for (int i = warp, j = 1; i < n.y; i += kKeepWarps, ++j) {
                const BorderBounds<D> now = next;
                if (i + kKeepWarps < n.y) next.load(p, kvh, __shfl_sync(kFullMask, phys, j), lane);
                const ExactScore e = exact_score<D>(p, s, kvh, now, lane);
                if (lane == 0) sh.list_hi[i] = e.hi, sh.list_lo[i] = e.lo;
            }
            __syncthreads();
            if (tid < n.y) {
                const int mine = sh.list[tid];
                const int64_t hi = sh.list_hi[tid];
                const uint32_t lo = sh.list_lo[tid];
                int before = 0;
                for (int j = 0; j < n.y; ++j)
                    before += exact_above(sh.list_hi[j], sh.list_lo[j], hi, lo) ||
                              (sh.list_hi[j] == hi && sh.list_lo[j] == lo && sh.list[j] < mine);
                sh.keep[tid] = before < want;
            }
            __syncthreads();
            k = at;
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (close >> j & 1) v[j] = sh.keep[k++] ? CUDART_INF_F : -CUDART_INF_F;
        } else if (!all_near) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                const int i = j * kKeepThreads + tid;
                if (i < m) p.score[seg * p.row + m0 + i] = v[j];
            }
            __syncthreads();
            bar = keep_slowly<D>(p, sh, turn, s, kvh, seg, m0, m, need, twice, &all_near);
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                const int i = j * kKeepThreads + tid;
                if (i < m) v[j] = p.score[seg * p.row + m0 + i];
            }
        }
        // ---- the list, in ascending order ----
        uint32_t chosen = 0;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            const bool keep = all_near ? v[j] >= bar : v[j] > bar;
            const unsigned mask = __ballot_sync(kFullMask, keep);
            if (lane == 0) reinterpret_cast<int *>(places + j)[warp] = __popc(mask);
            if (keep) chosen |= 1u << j;
        }
        __syncthreads();
        int base = m0;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            const int4 x = places[j];
            const unsigned mask = __ballot_sync(kFullMask, chosen >> j & 1);
            const int at = base + (warp > 0 ? x.x : 0) + (warp > 1 ? x.y : 0) + (warp > 2 ? x.z : 0) +
                           __popc(mask & ((1u << lane) - 1));
            if (chosen >> j & 1) out[at] = m0 + j * kKeepThreads + tid;
            base += x.x + x.y + x.z + x.w;
        }
    } else {
        bar = keep_slowly<D>(p, sh, turn, s, kvh, seg, m0, m, need, twice, &all_near);
        int base = m0;
        for (int first = 0; first < m; first += kKeepThreads) {
            const int i = first + tid;
            const float x = i < m ? p.score[seg * p.row + m0 + i] : -CUDART_INF_F;
            const bool keep = all_near ? x >= bar : x > bar;
            const unsigned mask = __ballot_sync(kFullMask, keep);
            if (lane == 0) sh.sums[turn][warp][0] = __popc(mask);
            __syncthreads();
            int at = base + __popc(mask & ((1u << lane) - 1));
            for (int w = 0; w < kKeepWarps; ++w) {
                if (w < warp) at += sh.sums[turn][w][0];
                base += sh.sums[turn][w][0];
            }
            turn ^= 1;
            if (keep) out[at] = m0 + i;
        }
    }
}

// A sequence of at most max_selected blocks keeps all of them.
__device__ __forceinline__ void keep_all(const SelectParams &p, int64_t seg, int count) {
    for (uint32_t i = threadIdx.x; i < (uint32_t)p.max_selected; i += kKeepThreads)  // (up to 2^31 - 1)
        p.selected[seg * p.max_selected + i] = i < (uint32_t)count ? (int)i : -1;
    if (threadIdx.x == 0) p.num_selected[seg] = count;
}

template <int D>
__global__ void __launch_bounds__(kKeepThreads) select_keep_kernel(const __grid_constant__ SelectParams p) {
    __shared__ __align__(16) KeepScratch sh;
    grid_dependency_wait();
    launch_dependents();
    const int s = blockIdx.y, kvh = blockIdx.x;
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    bool bad;
    const int count = select_blocks_of(p, s, &bad);
    if (count <= p.max_selected) {
        keep_all(p, seg, count);
        return;
    }
    if (threadIdx.x == 0) p.num_selected[seg] = p.max_selected;
    keep_blocks<D, 0>(p, sh, nullptr, s, kvh, count, p.score + seg * p.row, p.reach + seg * p.row / kTileBlocks);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores to the shared memory of the cluster's CTA 0.
__device__ __forceinline__ void store_first(const float *at, float v) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_addr(at)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}

// A cluster of CTAs per (sequence, KV head) of up to VALUES * 128 blocks: its warps score 16 blocks in turn, the scores
// meet in the first CTA's shared memory, which keeps the blocks.
template <int D, int NT, int VALUES>
__global__ void __launch_bounds__(kKeepThreads) select_fused_kernel(const __grid_constant__ SelectParams p) {
    __shared__ __align__(16) KeepScratch sh;
    __shared__ int4 places[VALUES];
    __shared__ float scores[VALUES * kKeepThreads], reaches[VALUES * kKeepThreads / kTileBlocks];
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int s = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t seg = (int64_t)s * p.num_kv_heads + kvh;
    // asked into L2 while the kernel before still runs (nothing is read): the context, the table's row, the queries
    if (rank == 0) {
        if (threadIdx.x == 0) prefetch_l2(p.context_lens + s);
        const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
        if (kvh == 0)
            for (int i = threadIdx.x * 32; i < p.max_blocks_per_seq; i += kKeepThreads * 32) prefetch_l2(row + i);
        for (int i = threadIdx.x * 64; i < p.group * D; i += kKeepThreads * 64) prefetch_l2(p.query + seg * p.group * D + i);
    }
    grid_dependency_wait();
    launch_dependents();
    bool bad;
    const int count = select_blocks_of(p, s, &bad);
    if (bad && rank == 0 && kvh == 0 && threadIdx.x == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
    if (count <= p.max_selected) {  // for all CTAs of the cluster
        if (rank == 0) keep_all(p, seg, count);
        return;
    }
    cluster_arrive();  // this CTA runs: its shared memory may be written
    const int tiles = (count + kTileBlocks - 1) / kTileBlocks, step = (int)ctas * kKeepWarps;
    int tile = (int)rank * kKeepWarps + warp;
    int phys[2] = {0, 0};
    const bool first = (lane & 3) == 0;
    if (tile < tiles) {
        phys[0] = select_phys(p, s, tile * kTileBlocks + g, count, first);
        phys[1] = select_phys(p, s, tile * kTileBlocks + g + 8, count, first);
    }
    SelectQueries<D, NT> queries;
    queries.load(p, seg, lane);
    cluster_wait();
    for (; tile < tiles; tile += step) {
        float best[2], reach;
        score_tile<D, NT>(p, queries, phys, kvh, lane, best, reach);
        const int b0 = tile * kTileBlocks;
        if (tile + step < tiles) {
            phys[0] = select_phys(p, s, b0 + step * kTileBlocks + g, count, first);
            phys[1] = select_phys(p, s, b0 + step * kTileBlocks + g + 8, count, first);
        }
        if (first)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (b0 + g + 8 * r < count) store_first(scores + b0 + g + 8 * r, best[r]);
        if (lane == 0) store_first(reaches + tile, reach);
    }
    __syncwarp();
    cluster_arrive();
    if (rank != 0) {  // (a CTA waits for its barrier before it ends)
        cluster_wait();
        return;
    }
    cluster_wait();
    if (threadIdx.x == 0) p.num_selected[seg] = p.max_selected;
    keep_blocks<D, VALUES>(p, sh, places, s, kvh, count, scores, reaches);
}

// The fused kernel for up to max_blocks blocks a sequence, or NULL.
constexpr int kFusedBlocks = 32 * kKeepThreads;
template <int D, int NT>
const void *fused_kernel(int max_blocks) {
    return max_blocks <= 4 * kKeepThreads    ? reinterpret_cast<const void *>(&select_fused_kernel<D, NT, 4>)
           : max_blocks <= 8 * kKeepThreads  ? reinterpret_cast<const void *>(&select_fused_kernel<D, NT, 8>)
           : max_blocks <= 16 * kKeepThreads ? reinterpret_cast<const void *>(&select_fused_kernel<D, NT, 16>)
           : max_blocks <= kFusedBlocks      ? reinterpret_cast<const void *>(&select_fused_kernel<D, NT, 32>)
                                             : nullptr;
}

constexpr int kSelectFill = 608;
// CTAs of a cluster: at most 8, a tile per warp, and fewer with more segments than fill the GPU, which then take more
// tiles each.  Measured with up to 304, 608, 1216, 2500 and 5000 CTAs in all: 64 sequences x 8 heads of up to 1024 blocks
// 42, 42, 45, 46 and 56 us, 32 x 8 32, 26, 29, 32 and 32, 16 x 8 21, 19, 22, 22 and 22.
int cluster_ctas(int max_blocks, int64_t segments) {
    const int tiles = (max_blocks + kTileBlocks - 1) / kTileBlocks;
    int ctas = 8;
    while (ctas > 1 && (tiles <= ctas / 2 * kKeepWarps || segments * ctas > kSelectFill)) ctas /= 2;
    return ctas;
}

cudaError_t launch_cluster(const void *fn, dim3 grid, int ctas, pkv_stream_t stream, void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kKeepThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Workspace carve-up (byte offsets).  It carries nothing from call to call.
struct SelectWorkspace {
    size_t score, score_hi, reach, total;
    int64_t row;
    static SelectWorkspace plan(int num_seqs, int num_kv_heads, int max_blocks_per_seq) {
        auto up = [](size_t x) { return (x + 255) / 256 * 256; };
        SelectWorkspace w;
        w.row = ((int64_t)max_blocks_per_seq + kTileBlocks - 1) / kTileBlocks * kTileBlocks;
        const size_t n = (size_t)num_seqs * num_kv_heads * (size_t)w.row;
        w.score = 0;
        w.score_hi = up(4 * n);
        w.reach = w.score_hi + up(8 * n);
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
    p.score_hi = reinterpret_cast<int64_t *>(wsb + ws.score_hi);
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
    const void *fused = d64 ? (wide ? fused_kernel<64, 2>(max_blocks_per_seq) : fused_kernel<64, 1>(max_blocks_per_seq))
                            : (wide ? fused_kernel<128, 2>(max_blocks_per_seq) : fused_kernel<128, 1>(max_blocks_per_seq));
    if (fused) {
        const int ctas = cluster_ctas(max_blocks_per_seq, (int64_t)num_seqs * num_kv_heads);
        if (launch_cluster(fused, dim3((unsigned)ctas, (unsigned)num_kv_heads, (unsigned)num_seqs), ctas, stream, args) !=
            cudaSuccess) {
            cudaGetLastError();
            return PKV_ERR_CUDA;
        }
        return PKV_OK;
    }
    const void *fn = d64 ? (wide ? reinterpret_cast<const void *>(&select_score_kernel<64, 2>)
                                 : reinterpret_cast<const void *>(&select_score_kernel<64, 1>))
                         : (wide ? reinterpret_cast<const void *>(&select_score_kernel<128, 2>)
                                 : reinterpret_cast<const void *>(&select_score_kernel<128, 1>));
    constexpr int per = kThreads / 32 * kTileBlocks;
    if (launch_pdl(fn, dim3((unsigned)((max_blocks_per_seq + per - 1) / per), (unsigned)num_kv_heads, (unsigned)num_seqs),
                   dim3(kThreads), 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    fn = d64 ? reinterpret_cast<const void *>(&select_keep_kernel<64>) : reinterpret_cast<const void *>(&select_keep_kernel<128>);
    if (launch_pdl(fn, dim3((unsigned)num_kv_heads, (unsigned)num_seqs), dim3(kKeepThreads), 0, stream, args) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
