// pkv_q8.cu -- the write of new tokens into a cache of 8-bit codes.
//
// A (block, KV head) tile holds codes of one scale a / M: a the largest magnitude
// of the tile's rows so far (an fp16 value), M = 127 (int8) or 448 (e4m3).  A row
// x becomes rn(M x / a).  Where new rows raise a from a0, the rows before them are
// rounded again, rn(code a0 / a); a0 comes back exactly from the scale, as the
// fp16 value next to M times it.  Each code is the exact quotient's, ties to even:
// x (M / a) in fp32 is within 2^-22 of it, and is rounded to 20 bits first.  A tie t
// between two codes has 8 bits and a 11, so t a and M x (18 bits) differ, if they
// do, by 2^-19 of themselves or more, and what is no tie cannot round to one
// (2^-19 - 2^-22 > 2^-20), while what is one does.  code a0 / a goes the same way.
//
// A tile belongs to block_size * D / 64 threads, which hold its new rows in
// registers, 64 elements each, between the maximum and the codes, so that they are
// read once (2 bytes per element; 1 is written).  The codes are made two at a time
// (packed fp32 arithmetic), the blocks found from query_starts by a search in
// eighths.
//
// Measured: four prompts of 1000 to 4001 tokens, 8 heads of 128, 15.7 us, 3780 GB/s,
// 0.56 of the copy bandwidth (with fp32 divisions for the codes and a search in
// halves 25.1); in e4m3, with fewer steps to a code, 14.4.  No pipe is full (67% of the
// issue slots, integer pipe 48%, HBM 29%): a warp goes through search, look-ups, loads,
// maximum, conversion and stores of one tile, which only other warps overlap.  64 single
// tokens of 8 heads 4.4 us, three dependent look-ups behind a launch.
#include <cuda_runtime.h>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_launch.h"
#include "pkv_schedule.h"
#include "pkv_tcgen05.cuh"
#include "pkv_touched.cuh"

namespace pkv {
namespace {

struct WriteParams {
    TouchedParams t;
    const __half *rows[2];   // keys, values: a token's heads contiguous
    int64_t stride[2];       // elements between tokens
    unsigned char *cache[2];
    float *scale[2];
    int64_t tiles;
    int num_kv_heads;
    int scale_stride;
};

// Two values to 20 significant bits each, nearest (Veltkamp's splitting).
__device__ __forceinline__ uint64_t to_20_bits(uint64_t y) {
    const uint64_t minus = pack2(-1.f, -1.f), c = mul2(y, pack2(17.f, 17.f));
    return fma2(fma2(y, minus, c), minus, c);  // c - (c - y), each rounded once
}

template <bool E4M3>
struct Codes {
    static constexpr float kTop = E4M3 ? 448.f : 127.f;
    // Eight quotients in units of the scale, in pairs, each within 2^-22 of itself -> codes.
    __device__ static uint2 pack(const uint64_t (&y)[4]) {
        uint32_t r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float z[4];
            uint64_t a = to_20_bits(y[2 * k]), b = to_20_bits(y[2 * k + 1]);
            if (!E4M3) {  // 1.5 2^23 + z: the nearest integer to z is in the low bits
                const uint64_t place = pack2(12582912.f, 12582912.f);
                a = add2(a, place), b = add2(b, place);
            }
            unpack2(a, z[0], z[1]);
            unpack2(b, z[2], z[3]);
            if (E4M3)
                asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
                    : "=r"(r[k])
                    : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
            else
                r[k] = __byte_perm(__byte_perm(__float_as_uint(z[0]), __float_as_uint(z[1]), 0x0040),
                                   __byte_perm(__float_as_uint(z[2]), __float_as_uint(z[3]), 0x0040), 0x5410);
        }
        return make_uint2(r[0], r[1]);
    }
    // The same of quotients that may be no numbers.  Infinite ones: the largest code.  NaN: 0 in int8, NaN in e4m3.
    __device__ static uint2 pack_any(uint64_t (&y)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float z[2];
            unpack2(y[k], z[0], z[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (z[e] != z[e] && !E4M3) z[e] = 0.f;
                if (fabsf(z[e]) > kTop) z[e] = copysignf(kTop, z[e]);
            }
            y[k] = pack2(z[0], z[1]);
        }
        return pack(y);
    }
    __device__ static void unpack(uint2 c, float (&y)[8]) {
        const uint32_t r[2] = {c.x, c.y};
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (E4M3) {
                uint32_t lo, hi;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                    : "=r"(lo), "=r"(hi)
                    : "r"(r[k]));
                const float2 a = unpack_half2(lo), b = unpack_half2(hi);
                y[4 * k] = a.x, y[4 * k + 1] = a.y, y[4 * k + 2] = b.x, y[4 * k + 3] = b.y;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 * k + e] = (float)(signed char)(r[k] >> (8 * e));
            }
    }
};

// The largest finite magnitude of two packed fp16 values, as their bits.
__device__ __forceinline__ uint32_t finite_bits(uint32_t v) {
    const uint32_t m = v & 0x7fff7fffu;
    return m & __vcmpltu2(m, 0x7c007c00u);
}

constexpr int kVecs = 8;  // vectors of 8 elements per thread
// Threads of a CTA, 64, 128 and 256: four prompts 15.7, 15.7 and 16.2 us, 64 single tokens 4.4, 4.4 and 4.6.
constexpr int kLeastWriteThreads = 128;
template <int TILE>
constexpr int kWriteThreads = TILE > kLeastWriteThreads ? TILE : kLeastWriteThreads;

// TILE threads per tile.
template <bool E4M3, int D, int TILE>
__global__ void __launch_bounds__(kWriteThreads<TILE>) write_q8_kernel(const __grid_constant__ WriteParams p) {
    constexpr int kPerRow = D / 8, kTiles = kWriteThreads<TILE> / TILE;
    constexpr float kTop = Codes<E4M3>::kTop;
    __shared__ uint32_t tops[kWriteThreads<TILE> / 32];
    touched_ask(p.t);
    grid_dependency_wait();
    launch_dependents();
    touched_check(p.t);
    const int in = threadIdx.x % TILE;
    const int64_t tile = (int64_t)blockIdx.x * kTiles + threadIdx.x / TILE;
    // tiles of one block side by side: its heads' keys, then its heads' values
    const int64_t unit = div_nonneg(tile, 2 * p.num_kv_heads);
    const int rest = (int)(tile - unit * 2 * p.num_kv_heads);
    const int which = rest >= p.num_kv_heads, head = rest - which * p.num_kv_heads;
    TouchedBlock b = {-1, 0, 0, 0};
    if (tile < p.tiles) b = touched_block(p.t, unit, in == 0 && rest == 0);
    const int64_t at = (int64_t)b.phys * p.num_kv_heads + head;
    float *scale = p.scale[which] + (int64_t)b.phys * p.scale_stride + head;
    uint2 *codes = reinterpret_cast<uint2 *>(p.cache[which]) + (at << p.t.block_shift) * kPerRow;
    const __half *src = p.rows[which] + (b.token - b.lo) * p.stride[which] + (int64_t)head * D;

    // thread `in` has vector in % kPerRow of the rows in / kPerRow + i kStep (a tile's vectors side by side)
    constexpr int kStep = TILE / kPerRow;
    static_assert(TILE % kPerRow == 0, "whole rows");
    const int64_t stride = p.stride[which];
    const __half *at_row = src + in / kPerRow * stride + in % kPerRow * 8;
    uint4 x[kVecs];
    uint32_t top = 0, all = 0;  // largest finite magnitudes, all bits of the magnitudes
    float before = 0.f;
    if (b.phys >= 0) {
        if (b.lo > 0) before = *scale;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int r = (i * TILE + in) / kPerRow;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r >= b.lo && r < b.hi) x[i] = *reinterpret_cast<const uint4 *>(at_row);
            at_row += kStep * stride;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t m[4] = {x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu};
            all = __vmaxu2(all, __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3])));
        }
        top = all;
        if (__vcmpgtu2(all, 0x7bff7bffu)) {  // not all are finite
            top = 0;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(finite_bits(x[i].x), finite_bits(x[i].y)),
                                             __vmaxu2(finite_bits(x[i].z), finite_bits(x[i].w))));
        }
        top = max(top & 0xffffu, top >> 16);
    }
#pragma unroll
    for (int d = (TILE < 32 ? TILE : 32) / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, d));
    if (TILE > 32) {
        constexpr int kW = TILE < 32 ? 1 : TILE / 32;
        if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
        __syncthreads();  // also: every thread has read the scale
        const int w0 = threadIdx.x / TILE * kW;
#pragma unroll
        for (int w = 0; w < kW; ++w) top = max(top, tops[w0 + w]);
    } else {
        __syncwarp();
    }
    if (b.phys < 0) return;

    // a0: what the scale stands for; one that is negative or no number counts as 0
    float a0 = __half2float(__float2half_rn(before * kTop));
    if (!(a0 > 0.f)) a0 = 0.f;
    a0 = fminf(a0, 65504.f);
    const float a = fmaxf(a0, __half2float(__ushort_as_half((unsigned short)top)));
    const bool grown = b.lo > 0 && a > a0;
    if (in == 0 && (b.lo == 0 || grown)) *scale = a / kTop;
    const float by = a > 0.f ? kTop / a : kTop, again = a > 0.f ? a0 / a : 0.f;
    const bool odd = __vcmpgtu2(all, 0x7bff7bffu) != 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = i * TILE + in, r = v / kPerRow;
        const bool fresh = r >= b.lo && r < b.hi;
        if (!fresh && !(grown && r < b.lo)) continue;
        uint64_t y[4];
        if (fresh) {
            const uint32_t h[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = unpack_half2(h[k]);
                y[k] = mul2(pack2(f.x, f.y), pack2(by, by));
            }
        } else {
            float f[8];
            Codes<E4M3>::unpack(codes[v], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = mul2(pack2(f[2 * k], f[2 * k + 1]), pack2(again, again));
        }
        codes[v] = odd && fresh ? Codes<E4M3>::pack_any(y) : Codes<E4M3>::pack(y);
    }
}

// block_size * D / 64 threads per tile: D / 8 at block size 8, to 16 times as many at 128.
template <bool E4M3, int D>
const void *write_kernel(int block_size) {
    switch (block_size) {
        case 8: return reinterpret_cast<const void *>(&write_q8_kernel<E4M3, D, D / 8>);
        case 16: return reinterpret_cast<const void *>(&write_q8_kernel<E4M3, D, D / 4>);
        case 32: return reinterpret_cast<const void *>(&write_q8_kernel<E4M3, D, D / 2>);
        case 64: return reinterpret_cast<const void *>(&write_q8_kernel<E4M3, D, D>);
        default: return reinterpret_cast<const void *>(&write_q8_kernel<E4M3, D, 2 * D>);
    }
}

// ---- the key bounds ----

struct BoundsParams {
    TouchedParams t;
    const unsigned char *cache;
    const float *scale;
    __half *bounds;
    int64_t tiles;
    int num_kv_heads;
    int scale_stride;
};

// A warp per (block, KV head): lanes take 8 channels each of 4 (head_dim 64) or 2
// rows at a time, eight loads ahead.  Nothing meets in shared memory: what the lanes
// of one channel have is joined by shuffles.  Bound by HBM for prompts, whose blocks'
// rows are read once, and its latency: those of two prompts of 8000 and 16384 tokens,
// 8 heads of 128, fp16, 11.5 us, 4590 GB/s, 0.68 of the copy bandwidth (int8 10.6, e4m3
// 9.1); the last blocks of 64 sequences 3.8 us (4.8, 4.3).
// Threads of a CTA, 32, 64, 128 and 256: prompts 11.4, 11.5, 11.9 and 12.1 us, single tokens 3.7, 3.7, 3.9 and 4.1.
constexpr int kBoundsThreads = 64;

template <int TYPE, int D>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int kPerRow = D / 8, kRows = 32 / kPerRow, kAhead = 8;
    touched_ask(p.t);
    grid_dependency_wait();
    launch_dependents();
    touched_check(p.t);
    const int lane = threadIdx.x % 32, row = lane / kPerRow, col = lane % kPerRow;
    const int64_t tile = (int64_t)blockIdx.x * (kBoundsThreads / 32) + threadIdx.x / 32;
    if (tile >= p.tiles) return;
    const int64_t unit = div_nonneg(tile, p.num_kv_heads);
    const int head = (int)(tile - unit * p.num_kv_heads);
    const TouchedBlock b = touched_block(p.t, unit, lane == 0 && head == 0);
    if (b.phys < 0) return;
    const int64_t at = (int64_t)b.phys * p.num_kv_heads + head;
    const int64_t first = (at << p.t.block_shift) * kPerRow + col;
    __half2 hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hi[k] = __halves2half2(__ushort_as_half(0xfc00), __ushort_as_half(0xfc00));
        lo[k] = __hneg2(hi[k]);
    }
    for (int r0 = row; r0 < b.hi; r0 += kRows * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kRows;
            if (r < b.hi) {
                if (TYPE == PKV_CACHE_F16) {
                    x[i] = reinterpret_cast<const uint4 *>(p.cache)[first + (int64_t)r * kPerRow];
                } else {
                    const uint2 c = reinterpret_cast<const uint2 *>(p.cache)[first + (int64_t)r * kPerRow];
                    float y[8];
                    Codes<TYPE == PKV_CACHE_E4M3>::unpack(c, y);
                    x[i] = pack8(y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (r0 + i * kRows < b.hi) {
                const __half2 *h = reinterpret_cast<const __half2 *>(&x[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    hi[k] = __hmax2_nan(hi[k], h[k]);
                    lo[k] = __hmin2_nan(lo[k], h[k]);
                }
            }
    }
#pragma unroll
    for (int d = kPerRow; d < 32; d <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hi[k] = __hmax2_nan(hi[k], __shfl_xor_sync(kFullMask, hi[k], d));
            lo[k] = __hmin2_nan(lo[k], __shfl_xor_sync(kFullMask, lo[k], d));
        }
    if (row < 2) {  // one row of lanes writes the maxima, the next the minima
        uint4 y;
        __half2 *h = reinterpret_cast<__half2 *>(&y);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = row ? lo[k] : hi[k];
        if (TYPE != PKV_CACHE_F16) {
            const float s = p.scale[(int64_t)b.phys * p.scale_stride + head];
            float f[8];
            unpack8(y, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s;
            y = pack8(f);
        }
        reinterpret_cast<uint4 *>(p.bounds)[(at * 2 + row) * kPerRow + col] = y;
    }
}

template <int D>
const void *bounds_kernel(int type) {
    return type == PKV_CACHE_F16    ? reinterpret_cast<const void *>(&key_bounds_kernel<PKV_CACHE_F16, D>)
           : type == PKV_CACHE_INT8 ? reinterpret_cast<const void *>(&key_bounds_kernel<PKV_CACHE_INT8, D>)
                                    : reinterpret_cast<const void *>(&key_bounds_kernel<PKV_CACHE_E4M3, D>);
}

bool good_block_size(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128; }

// What both calls check of the sequences; PKV_OK fills t.
int sequences(TouchedParams &t, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
              const int32_t *query_starts, int num_tokens, int num_seqs, int num_kv_heads, int head_dim,
              int block_size, int num_blocks, int32_t *dev_status) {
    if (num_tokens < 0 || num_seqs < 0 || num_seqs > 4096 || max_blocks_per_seq < 1 || num_blocks < 1 ||
        num_kv_heads < 1 || num_kv_heads > (1 << 16) || block_size < 1 || head_dim < 1)
        return PKV_ERR_INVALID_ARG;
    if (!block_tables || !context_lens || (!query_starts && num_tokens != num_seqs)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > (1 << 30)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads > (INT64_C(1) << 31) / block_size) return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || !good_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
    t.block_tables = block_tables;
    t.context_lens = context_lens;
    t.query_starts = query_starts;
    t.status = dev_status;
    t.num_tokens = num_tokens;
    t.num_seqs = num_seqs;
    t.max_blocks_per_seq = max_blocks_per_seq;
    t.num_blocks = num_blocks;
    t.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
    return PKV_OK;
}

int launch(const void *fn, int64_t blocks, int threads, void **args, pkv_stream_t stream) {
    if (blocks > INT32_MAX) return PKV_ERR_INVALID_ARG;
    if (launch_pdl(fn, dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_reshape_and_cache_q8(const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                                        void *key_cache, void *value_cache, float *key_scale, float *value_scale,
                                        int scale_stride, const int32_t *block_tables, int max_blocks_per_seq,
                                        const int32_t *context_lens, const int32_t *query_starts, int num_tokens,
                                        int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                        int cache_type, int32_t *dev_status, pkv_stream_t stream) {
    if (num_tokens == 0 || num_seqs == 0) return PKV_OK;
    if (cache_type != PKV_CACHE_INT8 && cache_type != PKV_CACHE_E4M3) return PKV_ERR_INVALID_ARG;
    if (!key || !value || !key_cache || !value_cache || !key_scale || !value_scale) return PKV_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache))
        return PKV_ERR_INVALID_ARG;
    WriteParams p = {};
    const int rc = sequences(p.t, block_tables, max_blocks_per_seq, context_lens, query_starts, num_tokens, num_seqs,
                             num_kv_heads, head_dim, block_size, num_blocks, dev_status);
    if (rc != PKV_OK) return rc;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (key_stride < row || key_stride % 8 || value_stride < row || value_stride % 8 ||
        scale_stride < num_kv_heads)
        return PKV_ERR_INVALID_ARG;
    p.rows[0] = static_cast<const __half *>(key);
    p.rows[1] = static_cast<const __half *>(value);
    p.stride[0] = key_stride;
    p.stride[1] = value_stride;
    p.cache[0] = static_cast<unsigned char *>(key_cache);
    p.cache[1] = static_cast<unsigned char *>(value_cache);
    p.scale[0] = key_scale;
    p.scale[1] = value_scale;
    p.scale_stride = scale_stride;
    p.num_kv_heads = num_kv_heads;
    p.tiles = touched_units(num_tokens, num_seqs, p.t.block_shift, query_starts != nullptr) * 2 * num_kv_heads;
    const int tile = block_size * head_dim / 64;
    const bool e4m3 = cache_type == PKV_CACHE_E4M3;
    const void *fn = head_dim == 64 ? (e4m3 ? write_kernel<true, 64>(block_size) : write_kernel<false, 64>(block_size))
                                    : (e4m3 ? write_kernel<true, 128>(block_size) : write_kernel<false, 128>(block_size));
    void *args[] = {&p};
    const int threads = tile > kLeastWriteThreads ? tile : kLeastWriteThreads, per = threads / tile;
    return launch(fn, (p.tiles + per - 1) / per, threads, args, stream);
}

extern "C" int pkv_block_key_bounds(void *key_bounds, const void *key_cache, const float *key_scale,
                                    int scale_stride, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                    const int32_t *query_starts, int num_tokens, int num_seqs, int num_kv_heads,
                                    int head_dim, int block_size, int num_blocks, int cache_type,
                                    int32_t *dev_status, pkv_stream_t stream) {
    if (num_tokens == 0 || num_seqs == 0) return PKV_OK;
    if (cache_type != PKV_CACHE_F16 && cache_type != PKV_CACHE_INT8 && cache_type != PKV_CACHE_E4M3)
        return PKV_ERR_INVALID_ARG;
    if (!key_bounds || !key_cache || (cache_type != PKV_CACHE_F16 && (!key_scale || scale_stride < num_kv_heads)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(key_bounds) || !aligned16(key_cache)) return PKV_ERR_INVALID_ARG;
    BoundsParams p = {};
    const int rc = sequences(p.t, block_tables, max_blocks_per_seq, context_lens, query_starts, num_tokens, num_seqs,
                             num_kv_heads, head_dim, block_size, num_blocks, dev_status);
    if (rc != PKV_OK) return rc;
    p.cache = static_cast<const unsigned char *>(key_cache);
    p.scale = key_scale;
    p.scale_stride = scale_stride;
    p.bounds = static_cast<__half *>(key_bounds);
    p.num_kv_heads = num_kv_heads;
    p.tiles = touched_units(num_tokens, num_seqs, p.t.block_shift, query_starts != nullptr) * num_kv_heads;
    void *args[] = {&p};
    constexpr int64_t per = kBoundsThreads / 32;
    return launch(head_dim == 64 ? bounds_kernel<64>(cache_type) : bounds_kernel<128>(cache_type),
                  (p.tiles + per - 1) / per, kBoundsThreads, args, stream);
}
