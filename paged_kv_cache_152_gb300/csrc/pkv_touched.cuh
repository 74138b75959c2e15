// pkv_touched.cuh -- the blocks that hold a batch's new tokens, found by number:
// what the 8-bit cache write and the key bounds go over.
//
// Sequence s has n(s) new tokens, the last ones of its L(s) positions, in the
// rows starts[s] .. starts[s + 1] - 1 (starts NULL: one each, row s).  They lie
// in at most n(s) / block_size + 2 blocks, so the numbers from
// floor(starts[s] / block_size) + 2 s up to the next sequence's are enough for
// them; numbers without a block do nothing.
#ifndef PKV_TOUCHED_CUH
#define PKV_TOUCHED_CUH

#include "pkv_device.cuh"

namespace pkv {

struct TouchedParams {
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_starts;  // nullable
    int32_t *status;
    int num_tokens;
    int num_seqs;
    int max_blocks_per_seq;
    int num_blocks;
    int block_shift;
};

// Numbers to go over (host).
inline int64_t touched_units(int num_tokens, int num_seqs, int block_shift, bool with_starts) {
    return with_starts ? (num_tokens >> block_shift) + 2 * (int64_t)num_seqs : num_seqs;
}

struct TouchedBlock {
    int phys;       // physical block, -1: none
    int lo, hi;     // rows lo .. hi - 1 of it are new
    int64_t token;  // row lo's token
};

__device__ __forceinline__ int touched_start(const TouchedParams &p, int s) {
    return min(max(__ldg(p.query_starts + s), 0), p.num_tokens);
}

// Asks into L2, while the kernel before still runs (nothing is read), what the blocks are found by.
__device__ __forceinline__ void touched_ask(const TouchedParams &p) {
    const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    auto ask = [&](const void *at, int64_t bytes) {
        if (first * 128 < bytes) prefetch_l2(static_cast<const char *>(at) + first * 128);
    };
    ask(p.context_lens, (int64_t)p.num_seqs * 4);
    if (p.query_starts) ask(p.query_starts, ((int64_t)p.num_seqs + 1) * 4);
    ask(p.block_tables, (int64_t)p.num_seqs * p.max_blocks_per_seq * 4);
}

// Reports query_starts that decrease or leave the rows, of each sequence by a thread of its own: where they do, the
// numbers may lead past a sequence.  For grids of at least num_seqs threads.
__device__ __forceinline__ void touched_check(const TouchedParams &p) {
    const int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (!p.query_starts || s >= p.num_seqs) return;
    const int start = __ldg(p.query_starts + s), end = __ldg(p.query_starts + s + 1);
    if (start < 0 || end < start || end > p.num_tokens) report(p.status, PKV_ERR_OUT_OF_RANGE);
}

// Block number u.  `first`: one thread per number, which reports what is wrong.
__device__ __forceinline__ TouchedBlock touched_block(const TouchedParams &p, int64_t u, bool first) {
    TouchedBlock t = {-1, 0, 0, 0};
    int s = (int)u, start = s, n = 1;
    int64_t j = 0;
    if (p.query_starts) {
        // the last s whose first number is not past u: seven of them looked at at a time
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int step = (hi - lo + 7) >> 3;
            int begin[7], before = 0;
#pragma unroll
            for (int k = 0; k < 7; ++k) begin[k] = touched_start(p, min(lo + (k + 1) * step, p.num_seqs - 1));
#pragma unroll
            for (int k = 0; k < 7; ++k) {
                const int at = lo + (k + 1) * step;
                before += at < hi && (begin[k] >> p.block_shift) + 2 * (int64_t)at <= u;
            }
            lo += before * step;
            hi = min(hi, lo + step);
        }
        s = lo;
        start = touched_start(p, s);
        n = max(touched_start(p, s + 1) - start, 0);
        j = u - ((start >> p.block_shift) + 2 * (int64_t)s);
    }
    const int64_t reach = (int64_t)p.max_blocks_per_seq << p.block_shift;
    const int len = __ldg(p.context_lens + s);
    bool bad = j == 0 && (len < 0 || len > reach || (p.query_starts && n > max(len, 0)));
    const int64_t pos0 = (int64_t)max(len, 0) - n;              // the first new token's position
    const int64_t from = max(pos0, (int64_t)0), end = min((int64_t)max(len, 0), reach);
    const int64_t block = (from >> p.block_shift) + j;
    const int64_t row0 = block << p.block_shift;
    if (j >= 0 && row0 < end && from < end) {
        const int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + block);
        if (phys < 0 || phys >= p.num_blocks) {
            bad = true;
        } else {
            t.phys = phys;
            t.lo = (int)(max(from, row0) - row0);
            t.hi = (int)(min(end, row0 + (int64_t(1) << p.block_shift)) - row0);
            t.token = start + (row0 + t.lo - pos0);
        }
    }
    if (bad && first) report(p.status, PKV_ERR_OUT_OF_RANGE);
    return t;
}

}  // namespace pkv

#endif  // PKV_TOUCHED_CUH
