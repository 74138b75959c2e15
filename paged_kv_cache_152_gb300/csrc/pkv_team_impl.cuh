// pkv_team_impl.cuh -- the team decode: single-token attention over a cache of
// 8-bit codes with a scale per (block, KV head), or over listed blocks.
//
// For each (sequence, KV head) and query head h of its group, over the rows t
// (all of the context, or those of the listed blocks):
//
//     x_t = c k_b (q_h . K_t),   out = sum_t e^{x_t} v_b V_t / sum_t e^{x_t}
//
// with K, V the codes (exact in fp16), k_b, v_b the scales of t's block (1 for
// an fp16 cache) and c the softmax scale.  With m the running maximum of x and 2^e
// the running least power of two above the scales v, the weights e^{x_t - m} v_b 2^-e
// are at most 1 whatever the scores and the scales; the sum runs over e^{x_t - m}.
//
// Bound by HBM: a row is read once for all query heads of its group.  8-bit rows
// halve the bytes, so the work per byte doubles: the split and the layout are
// chosen for few instructions per row and few meetings of the warps.
//  * The warps of a CTA (four; eight over fp16) work on one segment's piece
//    together, a step of 32 rows (16 of 256 bytes) each in turn, with a ring of
//    their own (16 KB per warp, 128 KB per SM in flight) that runs on into the next
//    pieces.  Their outputs meet in shared memory, those of up to eight short
//    pieces between two barriers (64 sequences over 50 to 900, 32 heads, int8, "chats",
//    49.8 us now: 48.3 then, 59.4 with barriers at every piece).  Four warps with steps
//    of 32 rows, two CTAs per SM, took 48.8 us there, eight warps with steps of 16 rows
//    53.9; a grouped batch 176 and 180 (178 now).
//  * Copies by cp.async: a lane copies the 16 bytes that its place in the swizzled
//    tile wants, from the block that its row lies in, and rows past the end come
//    as zeros; the block table's entries of 32 steps are looked up at once, a batch
//    ahead.  With the arithmetic and the joining left out, the copies alone take 39.8
//    us of the chats' and 56.0 of the 62 for 8 long contexts.
//  * mma.sync m16n8k16 with the rows on M and the heads on N for the scores
//    (8 heads fill N; a 16-row tile takes D/16 instructions), and the dims on M
//    and the heads on N for the output, transposed: the codes come from shared
//    memory by ldmatrix (.trans for V) as pairs of bytes, whose dims are taken
//    in the order that the fragments want them (queries and outputs follow it),
//    so that widening to fp16 is all that is done to them.  The weights turn
//    from the scores' layout to the product's by movmatrix.  (One group's heads are
//    16 rows at most: tcgen05's tiles of 64 or 128 would stay empty.  The tensor pipe
//    is active 22 to 25% of the time, the integer pipe, which widens, 36 to 41%.)
//  * int8 codes widen to fp16 exactly: a byte with 0x64 above it is 1024 more than
//    itself, off which one subtraction takes 1152 (the byte is code + 128).  Taking
//    the 128 off the sums instead, 128 times the queries' sum at the scores' start,
//    costs as much time (chats 49.8 us, 8 long contexts 62.9 and 63.0) and the digits
//    of scores whose large queries meet codes near zero.
//  * A weight goes into its product as two fp16 terms, after a factor of 2^15: 22
//    significant bits down to 2^-18, 11 down to 2^-29, where 1 is a weight of the
//    largest score and the largest scale.  (One term: 1.4 times the error of an output
//    rounded once, and the chats 48.0 instead of 49.8 us, the others level.)
//  * A piece that is a whole segment is divided and written by the CTA; one that
//    a CTA boundary cuts leaves (maximum, sum, output) in the workspace for the
//    joining kernel, which runs behind it with its launch hidden (2.3 us).
//
// Measured (us, GB/s, of the copy bandwidth): 64 sequences over 50 to 900, 32 heads,
// int8 49.8, 4890, 0.72; 256 over 256 to 4096, 32 heads and 8 KV heads, e4m3 178,
// 6520, 0.96; 8 over 8000 to 32768, int8 63.0, 5830, 0.86; 64 blocks of 32 rows of
// each of these, fp16 19.2, 3480, 0.51 (of a latency of three look-ups in a row), int8
// 14.8, e4m3 14.0; 128 blocks of 16 for 64 sequences, fp16 89 to 90, 6000, 0.88, int8
// 53.3, 5060, 0.75, e4m3 52.5, 5140, 0.76.
#ifndef PKV_TEAM_IMPL_CUH
#define PKV_TEAM_IMPL_CUH

#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_team_params.h"
#include "pkv_team_schedule.h"

namespace pkv {

enum TeamKind { kTeamF16, kTeamInt8, kTeamE4m3 };

// What goes with a step's tiles: the key and value scales of its groups, and the
// groups' rows in use.
template <int GROUPS>
struct alignas(16) TeamMeta {
    float2 scale[GROUPS];
    int rows[GROUPS];
};

template <int KIND, int D, int NT>
struct TeamConfig {
    static constexpr bool kWide = KIND == kTeamF16;
    static constexpr int kRowBytes = D * (kWide ? 2 : 1);
    static constexpr int kRows = kRowBytes <= 128 ? 32 : 16;  // of a step
    static constexpr int kTiles = kRows / 16;
    static constexpr int kGroups = kRows / 8;                // a group of 8 rows lies in one block
    static constexpr int kUnits = kRowBytes / 16;            // 16-byte units of a row
    static constexpr int kTileBytes = kRows * kRowBytes;
    static constexpr int kWarps = kWide ? 8 : 4;             // of a CTA
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kCtas = 8 / kWarps;                 // per SM
    static constexpr int kStages = 16384 / (2 * kTileBytes); // 16 KB per warp in flight, 128 KB per SM
    static constexpr int kGroupCopies = kUnits / 4;          // of a lane, per cache and group
    static constexpr int kPitch = D + 8;                     // floats between heads of a warp's output
    // [warps][stages][K, V tiles] [warps][stages] TeamMeta
    // [warps][8 rows] (maximum, sum, output's unit), [warps][8 rows][pitch] floats (a row is a head of
    // one of the pieces in hold), then by sequence: cum
    static constexpr size_t kMeta = (size_t)kWarps * kStages * 2 * kTileBytes;
    static constexpr size_t kMl = kMeta + (size_t)kWarps * kStages * sizeof(TeamMeta<kGroups>);
    static constexpr size_t kRed = kMl + (size_t)kWarps * 8 * 16;
    static constexpr size_t kCum = kRed + (size_t)kWarps * 8 * kPitch * 4;
};

// Byte of 16-byte unit u of row r in a tile whose rows are RB bytes: eight
// consecutive rows' unit u lie in eight different 16-byte columns of the banks.
template <int RB>
__device__ __forceinline__ int team_swizzle(int r, int u) {
    if (RB == 64) return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
    return r * RB + ((u ^ (r & 7)) << 4);
}

// Four codes in a register -> the fp16 pairs (b0, b1), (b2, b3), or with PAIRED
// (b0, b2), (b1, b3).  The byte code ^ 0x80 below 0x64 is fp16's 1024 + 128 + code,
// off which 1152 is taken, exactly.
template <int KIND, bool PAIRED>
__device__ __forceinline__ void team_widen(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    if (KIND == kTeamInt8) {
        const uint32_t u = codes ^ 0x80808080u, bias = 0x64806480u;
        lo = __byte_perm(u, 0x64646464u, PAIRED ? 0x4240 : 0x4140);
        hi = __byte_perm(u, 0x64646464u, PAIRED ? 0x4341 : 0x4342);
        const __half2 b = *reinterpret_cast<const __half2 *>(&bias);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&lo), b);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&hi), b);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        const uint32_t c = PAIRED ? __byte_perm(codes, 0, 0x3120) : codes;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(c));
    }
}

__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_16_of(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 2^x; 2^-inf = 0.
__device__ __forceinline__ float team_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr int kTeamPlace = 15;      // weights are stored times 2^15
constexpr int kTeamLeastExp = -100;  // the least e
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((e + 127) << 23); }

// A warp's attention state: lane (g, t) = (lane / 4, lane % 4) has heads 2t and
// 2t + 1 of each tile of eight: m their maximum (the same on all g), l the sum
// over the rows that this lane has seen, o[i] the output of the fragment's dims.
template <int D, int NT>
struct TeamState {
    float m[NT][2], l[NT][2];
    float o[NT][D / 16][4];
    int e;           // the outputs are in units of 2^e
    __device__ __forceinline__ void clear() {
        e = kTeamLeastExp;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -CUDART_INF_F;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }
    }
};

// One step: tiles at kt, vt (shared addresses).
template <int KIND, int D, int NT>
__device__ __forceinline__ void team_step(uint32_t kt, uint32_t vt,
                                          const TeamMeta<TeamConfig<KIND, D, NT>::kGroups> &meta,
                                          const uint32_t (&q)[NT][D / 16][2], float scale_log2, int group, TeamState<D, NT> &st, int lane) {
    using C = TeamConfig<KIND, D, NT>;
    constexpr int RB = C::kRowBytes;
    const int g = lane >> 2;
    // ldmatrix: this lane's row and which of two units; a pair's two lie 16 bytes
    // apart but for the swizzle, so unit u's place is unit 0's with u's bits flipped
    const int row16 = (lane & 7) + ((lane >> 3) & 1) * 8;
    uint32_t place[C::kUnits / 2];
#pragma unroll
    for (int u = 0; u < C::kUnits; u += 2) place[u / 2] = team_swizzle<RB>(row16, u + (lane >> 4));

    float s[C::kTiles][NT][4];
#pragma unroll
    for (int r = 0; r < C::kTiles; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r][n][e] = 0.f;
#pragma unroll
    for (int u = 0; u < C::kUnits; u += 2)
#pragma unroll
        for (int r = 0; r < C::kTiles; ++r) {
            uint32_t x0, x1, x2, x3;  // rows 0-7, rows 8-15 of unit u, the same of unit u + 1
            ldsm_x4(kt + place[u / 2] + r * 16 * RB, x0, x1, x2, x3);
            if constexpr (C::kWide) {
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816(s[r][n], x0, x1, x2, x3, q[n][u / 2][0], q[n][u / 2][1]);
            } else {
                uint32_t a0, a1, a2, a3;
                team_widen<KIND, false>(x0, a0, a2);
                team_widen<KIND, false>(x1, a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816(s[r][n], a0, a1, a2, a3, q[n][u][0], q[n][u][1]);
                team_widen<KIND, false>(x2, a0, a2);
                team_widen<KIND, false>(x3, a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816(s[r][n], a0, a1, a2, a3, q[n][u + 1][0], q[n][u + 1][1]);
            }
        }

    // scores in log2 units
    float vs[C::kGroups];
    float top[NT][2];
    int e_to = C::kWide ? 0 : st.e;
#pragma unroll
    for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -CUDART_INF_F;
#pragma unroll
    for (int r = 0; r < C::kTiles; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = 2 * r + h;
            const bool live = g < meta.rows[j];
            const float2 scale = C::kWide ? make_float2(1.f, 1.f) : meta.scale[j];
            const float f = C::kWide ? scale_log2 : scale_log2 * scale.x;
            vs[j] = scale.y;
            if (!C::kWide) e_to = max(e_to, (int)((__float_as_uint(scale.y) & 0x7fffffffu) >> 23) - 126);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[r][n][2 * h + e];
                    x = live ? x * f : -CUDART_INF_F;
                    top[n][e] = fmaxf(top[n][e], x);
                }
        }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(kFullMask, top[n][e], d));

    // (heads past the group, whose queries are zeros, and states that are empty
    // still need no rescaling)
    bool moved = false;
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float was = st.m[n][e], to = fmaxf(top[n][e], was);
            f[n][e] = team_exp2(was - (to == -CUDART_INF_F ? 0.f : to));
            moved |= (to > was || e_to > st.e) && was != -CUDART_INF_F && n * 8 + 2 * (lane & 3) + e < group;
            st.m[n][e] = to;
            st.l[n][e] *= f[n][e];
        }
    if (__any_sync(kFullMask, moved)) {
        const float unit = C::kWide ? 1.f : power_of_2(max(st.e - e_to, -126));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f[n][0] *= unit, f[n][1] *= unit;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[n][i][0] *= f[n][0];
                st.o[n][i][1] *= f[n][1];
                st.o[n][i][2] *= f[n][0];
                st.o[n][i][3] *= f[n][1];
            }
        }
    }
    st.e = e_to;
    const float placed = power_of_2(kTeamPlace - e_to);
    uint32_t w[C::kGroups][NT][2];  // a weight as two fp16 terms
#pragma unroll
    for (int j = 0; j < C::kGroups; ++j) vs[j] *= placed;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float ref[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) ref[e] = st.m[n][e] == -CUDART_INF_F ? 0.f : st.m[n][e];
#pragma unroll
        for (int r = 0; r < C::kTiles; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = team_exp2(s[r][n][2 * h] - ref[0]), p1 = team_exp2(s[r][n][2 * h + 1] - ref[1]);
                st.l[n][0] += p0;
                st.l[n][1] += p1;
                const float w0 = p0 * vs[2 * r + h], w1 = p1 * vs[2 * r + h];
                const uint32_t hi = pack_half2(w0, w1);
                const float2 back = unpack_half2(hi);
                w[2 * r + h][n][0] = transpose_8x8(hi);
                w[2 * r + h][n][1] = transpose_8x8(pack_half2(w0 - back.x, w1 - back.y));
            }
    }

#pragma unroll
    for (int r = 0; r < C::kTiles; ++r)
#pragma unroll
        for (int u = 0; u < C::kUnits; u += 2) {
            uint32_t x0, x1, x2, x3;
            ldsm_x4_trans(vt + place[u / 2] + r * 16 * RB, x0, x1, x2, x3);
            if constexpr (C::kWide) {  // x0, x1: rows 0-7 and 8-15 of dims 0-7; x2, x3: of dims 8-15
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mma_16816(st.o[n][u / 2], x0, x2, x1, x3, w[2 * r][n][e], w[2 * r + 1][n][e]);
            } else {
                uint32_t a0, a1, a2, a3;
                team_widen<KIND, true>(x0, a0, a1);
                team_widen<KIND, true>(x1, a2, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mma_16816(st.o[n][u], a0, a1, a2, a3, w[2 * r][n][e], w[2 * r + 1][n][e]);
                team_widen<KIND, true>(x2, a0, a1);
                team_widen<KIND, true>(x3, a2, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mma_16816(st.o[n][u + 1], a0, a1, a2, a3, w[2 * r][n][e], w[2 * r + 1][n][e]);
            }
        }
}

// Up to 32 steps of a warp (every kWarps-th of a piece's) in one segment: lane
// j looks up the block table's entry j of theirs, all at once and a batch ahead of
// their use.
struct TeamBatch {
    int seg, s;     // the segment and its sequence
    int c;          // the first step
    int lo, end;    // the piece
    int rot;        // the warp that takes the piece's first step
    int count;      // steps of the batch, 0: none
    int phys;       // lane j: physical block of entry j
    int rows;       //         its rows in use
    int64_t at;     //         where they are in the caches, in bytes (fixed when the batch's turn comes)
};

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(TeamConfig<KIND, D, NT>::kThreads, TeamConfig<KIND, D, NT>::kCtas)
    team_kernel(const __grid_constant__ TeamParams p) {
    using C = TeamConfig<KIND, D, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    float4 *ml = reinterpret_cast<float4 *>(smem + C::kMl);
    float *red = reinterpret_cast<float *>(smem + C::kRed);
    int64_t *cum = reinterpret_cast<int64_t *>(smem + C::kCum);
    __shared__ int64_t warp_sum[C::kWarps];
    __shared__ int4 held[8];  // a piece: segment, the warp of its first step, its warps, 0 / 1 / 2: part 0 / part 1 / whole
    __shared__ TeamPlace share[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int heads = p.num_kv_heads, bs = 1 << p.block_shift;
    const int64_t reach = (int64_t)p.max_blocks_per_seq << p.block_shift;
    auto context = [&](int s) {
        const int len = __ldg(p.context_lens + s);
        return len < 0 ? 0 : len > reach ? (int)reach : len;
    };
    auto steps_of = [&](int s) {
        return team_steps(team_rows(context(s), p.block_shift, p.selected ? p.max_selected : -1), C::kRows);
    };

    // While the kernel before still runs nothing is read, but what will be read one after the other is asked into
    // L2 (which its writes go through): contexts, tables, lists and queries, up to 1 MB of each.
    {
        const int first = blockIdx.x * C::kThreads + tid, step = gridDim.x * C::kThreads;
        auto ask = [&](const void *at, int64_t bytes) {
            const int lines = (int)(min(bytes, (int64_t)1 << 20) + 127 >> 7);
            for (int i = first; i < lines; i += step) prefetch_l2(static_cast<const char *>(at) + (int64_t)i * 128);
        };
        ask(p.context_lens, (int64_t)p.num_seqs * 4);
        ask(p.block_tables, (int64_t)p.num_seqs * p.max_blocks_per_seq * 4);
        if (p.selected) {
            ask(p.num_selected, (int64_t)p.num_seqs * heads * 4);
            ask(p.selected, (int64_t)p.num_seqs * heads * p.max_selected * 4);
        }
        ask(p.query, (int64_t)p.num_seqs * p.num_heads * D * 2);
    }
    grid_dependency_wait();
    launch_dependents();

    // The prefix sums of the sequences' steps.
    {
        const int per = (p.num_seqs + C::kThreads - 1) / C::kThreads;
        const int first = min(tid * per, p.num_seqs), end = min(first + per, p.num_seqs);
        int64_t mine = 0;
        for (int s = first; s < end; ++s) mine += team_units(steps_of(s));
        int64_t sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(kFullMask, sum, d);
            if (lane >= d) sum += x;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int64_t at = sum - mine;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
        for (int s = first; s < end; ++s) {
            cum[s] = at;
            at += team_units(steps_of(s));
        }
        if (tid == C::kThreads - 1) cum[p.num_seqs] = at;
        __syncthreads();
    }
    const int64_t T = cum[p.num_seqs] * heads;
    const int64_t ctas = team_ctas(T, gridDim.x);
    if (tid < 2) share[tid] = team_start(cum, p.num_seqs, heads, min((int64_t)blockIdx.x + tid, ctas), ctas);
    __syncthreads();
    // The share: segments from.seg, from step from.step on, to to.seg, before to.step.
    const TeamPlace from = share[0], to = share[1];
    auto more = [&](int seg) { return seg < to.seg || (seg == to.seg && to.step > 0); };
    auto piece_end = [&](int seg, int s) { return seg < to.seg ? team_steps_of(cum, s) : to.step; };
    const bool any = more(from.seg) && !(from.seg == to.seg && from.step >= to.step);
    int2 cut = make_int2(-1, -1);

    // ---- the ring ----
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * 2 * C::kTileBytes;
    TeamMeta<C::kGroups> *meta = reinterpret_cast<TeamMeta<C::kGroups> *>(smem + C::kMeta) + warp * C::kStages;
    // a step's rows lie in `entries` blocks, 2^span_shift rows in each
    const int span_shift = min(p.block_shift, C::kRows == 32 ? 5 : 4);
    const int entries = C::kRows >> span_shift;
    const int room = 32 / entries;  // steps of a batch
    // The entries of the batch that begins at step c of the piece.
    auto look_up = [&](TeamBatch &x) {
        x.rows = x.phys = 0;
        x.count = min(room, (x.end - x.c + C::kWarps - 1) / C::kWarps);
        if (lane >= x.count * entries) return;
        const int64_t v = (int64_t)(x.c + lane / entries * C::kWarps) * C::kRows + (lane % entries << span_shift);
        int64_t block = v >> p.block_shift;
        const int len = context(x.s);
        bool bad = false, there = true;
        if (p.selected) {
            const int64_t seg = x.seg;
            const int blocks = (len + bs - 1) >> p.block_shift;
            const int most = min(blocks, p.max_selected);
            int count = __ldg(p.num_selected + seg);
            // (a row past max_selected is that of a step past the list)
            const int listed = __ldg(p.selected + seg * p.max_selected + min(block, (int64_t)p.max_selected - 1));
            bad = (count < 0 || count > most) && v == 0;
            count = min(count, most);
            there = block < count;
            if (there) {
                block = listed;
                if (block < 0 || block >= blocks) bad = true, there = false;
            }
        }
        if (there) {
            const int64_t pos = (block << p.block_shift) + (v & (bs - 1));
            x.rows = (int)max((int64_t)0, min((int64_t)1 << span_shift, len - pos));
            if (x.rows > 0) x.phys = __ldg(p.block_tables + (int64_t)x.s * p.max_blocks_per_seq + block);
        }
        if (bad) report(p.status, PKV_ERR_OUT_OF_RANGE);
    };
    // The next batch: the piece's, or the next piece's in which this warp has a step.
    auto follow = [&](const TeamBatch &x, TeamBatch &y) {
        y = x;
        y.c += x.count * C::kWarps;
        y.count = 0;
#pragma unroll 1
        while (y.c >= y.end) {
            y.seg = team_next(cum, p.num_seqs, heads, y.seg, y.s);
            if (!more(y.seg)) return;
            y.rot = (y.rot + y.end - y.lo) % C::kWarps;
            y.lo = 0;
            y.c = (warp - y.rot) & (C::kWarps - 1);
            y.end = piece_end(y.seg, y.s);
        }
        look_up(y);
    };
    // A batch's turn: its table entries, loaded a batch ago, are looked at.
    auto settle = [&](TeamBatch &x) {
        if (x.rows > 0 && (x.phys < 0 || x.phys >= p.num_blocks)) {
            report(p.status, PKV_ERR_OUT_OF_RANGE);
            x.phys = 0;
        }
        const int row = (x.c + lane / entries * C::kWarps) * C::kRows + (lane % entries << span_shift);
        x.at = ((((int64_t)x.phys * heads + (x.seg - x.s * heads)) << p.block_shift) + (row & (bs - 1))) * C::kRowBytes;
    };
    TeamBatch now, then;
    now.count = then.count = 0;
    int k = 0;  // the next step to issue in `now`
    const int first_s = any ? from.seg / heads : 0;
    if (any) {
        then.seg = from.seg, then.s = first_s, then.rot = 0;
        then.lo = from.step, then.c = from.step + warp, then.end = piece_end(from.seg, first_s);
        follow(then, now);
        if (now.count > 0) {
            follow(now, then);
            settle(now);
        }
    }
    const unsigned char *kc = static_cast<const unsigned char *>(p.key_cache) + lane * 16;
    const unsigned char *vc = static_cast<const unsigned char *>(p.value_cache) + lane * 16;
    // lanes 2 j, 2 j + 1: the key and the value scale of group j
    const float *sc = lane & 1 ? p.value_scale : p.key_scale;
    uint32_t places[C::kGroupCopies];
#pragma unroll
    for (int i = 0; i < C::kGroupCopies; ++i)
        places[i] = team_swizzle<C::kRowBytes>((i * 32 + lane) / C::kUnits, (i * 32 + lane) % C::kUnits);
    auto issue = [&](int stage) {
        if (now.count > 0) {
            const uint32_t kt = ring + stage * 2 * C::kTileBytes;
            if (entries == 1) {  // one block
                const int64_t at = __shfl_sync(kFullMask, now.at, k);
                const int rows = __shfl_sync(kFullMask, now.rows, k);
                const unsigned char *ks = kc + at, *vs = vc + at;
                if (rows == C::kRows) {
#pragma unroll
                    for (int j = 0; j < C::kGroups; ++j)
#pragma unroll
                        for (int i = 0; i < C::kGroupCopies; ++i) {
                            const int off = (j * C::kGroupCopies + i) * 512;
                            cp_async_16_of(kt + places[i] + j * 8 * C::kRowBytes, ks + off);
                            cp_async_16_of(kt + places[i] + j * 8 * C::kRowBytes + C::kTileBytes, vs + off);
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < C::kGroups; ++j)
#pragma unroll
                        for (int i = 0; i < C::kGroupCopies; ++i) {
                            const bool live = j * 8 + (i * 32 + lane) / C::kUnits < rows;
                            const int off = live ? (j * C::kGroupCopies + i) * 512 : 0;
                            cp_async_16_or_zero(kt + places[i] + j * 8 * C::kRowBytes, ks + off, live);
                            cp_async_16_or_zero(kt + places[i] + j * 8 * C::kRowBytes + C::kTileBytes, vs + off, live);
                        }
                }
            } else {
#pragma unroll
                for (int j = 0; j < C::kGroups; ++j) {
                    const int entry = k * entries + (j * 8 >> span_shift), in = j * 8 & ((1 << span_shift) - 1);
                    const int64_t at = __shfl_sync(kFullMask, now.at, entry) + in * C::kRowBytes;
                    const int rows = __shfl_sync(kFullMask, now.rows, entry) - in;
#pragma unroll
                    for (int i = 0; i < C::kGroupCopies; ++i) {
                        const bool live = (i * 32 + lane) / C::kUnits < rows;
                        const int64_t off = live ? at + i * 512 : 0;
                        cp_async_16_or_zero(kt + places[i] + j * 8 * C::kRowBytes, kc + off, live);
                        cp_async_16_or_zero(kt + places[i] + j * 8 * C::kRowBytes + C::kTileBytes, vc + off, live);
                    }
                }
            }
            const int entry = k * entries + ((lane >> 1) * 8 >> span_shift);
            const int rows = __shfl_sync(kFullMask, now.rows, entry) - ((lane >> 1) * 8 & ((1 << span_shift) - 1));
            const int block = C::kWide ? 0 : __shfl_sync(kFullMask, now.phys, entry);
            if (lane < 2 * C::kGroups) {
                TeamMeta<C::kGroups> &m = meta[stage];
                m.rows[lane >> 1] = rows;
                if (!C::kWide)
                    cp_async_4_or_zero(smem_addr(m.scale) + lane * 4,
                                       sc + (int64_t)block * p.scale_stride + (now.seg - now.s * heads), rows > 0);
            }
            if (++k == now.count) {
                k = 0;
                now = then;
                if (now.count > 0) {
                    follow(now, then);
                    settle(now);
                }
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < C::kStages; ++i) issue(i);

    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
        const int len = __ldg(p.context_lens + s);
        if ((len < 0 || len > reach) && tid == 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
        if (cum[s + 1] == cum[s]) {  // no position: zeros, and no entry of a list can count
            for (int i = tid; i < p.num_heads * D / 8; i += C::kThreads)
                reinterpret_cast<uint4 *>(p.out + (int64_t)s * p.num_heads * D)[i] = make_uint4(0, 0, 0, 0);
            if (p.selected)
                for (int i = tid; i < heads; i += C::kThreads)
                    if (__ldg(p.num_selected + (int64_t)s * heads + i) != 0) report(p.status, PKV_ERR_OUT_OF_RANGE);
        }
    }

    // ---- pieces, some in hold: their outputs stay apart until a barrier for all ----
    const int g = lane >> 2, t = lane & 3;
    TeamState<D, NT> st;
    uint32_t q[NT][D / 16][2];
    const int red_heads = min(8, p.group), hold = 8 / red_heads;
    auto load_q = [&](int seg) {
        const __half *rows_q = p.query + (int64_t)seg * p.group * D;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + g;
            const bool live = h < p.group;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                // fp16: dims 2t, 2t + 1 and 8 further; codes: dims 4t to 4t + 3
                const __half *src = rows_q + h * D + 16 * i + (C::kWide ? 2 * t : 4 * t);
                uint2 x = make_uint2(0u, 0u);
                if (live) {
                    if (C::kWide) {
                        x.x = __ldg(reinterpret_cast<const uint32_t *>(src));
                        x.y = __ldg(reinterpret_cast<const uint32_t *>(src + 8));
                    } else {
                        x = __ldg(reinterpret_cast<const uint2 *>(src));
                    }
                }
                q[n][i][0] = x.x, q[n][i][1] = x.y;
            }
        }
    };
    // Dims d and d + 1 of a row of the outputs that a piece's warps hold: to the output, or to the workspace.
    auto join = [&](int row, int head, int d, const int4 &piece) {
        float top = -CUDART_INF_F, l = 0.f;
        float4 x[C::kWarps];
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            x[w] = make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
            if (((w - piece.y) & (C::kWarps - 1)) < piece.z) x[w] = ml[w * 8 + row];
            top = fmaxf(top, x[w].x);
        }
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            if (((w - piece.y) & (C::kWarps - 1)) >= piece.z) continue;
            const float f = team_exp2(x[w].x - ref), fo = f * x[w].z * (1.f / (1 << kTeamPlace));
            const float2 y = *reinterpret_cast<const float2 *>(red + (w * 8 + row) * C::kPitch + d);
            l = fmaf(x[w].y, f, l);
            o.x = fmaf(y.x, fo, o.x);
            o.y = fmaf(y.y, fo, o.y);
        }
        if (piece.w == 2) {
            const float inv = l == 0.f ? 0.f : 1.f / l;  // no row: zeros
            *reinterpret_cast<__half2 *>(p.out + ((int64_t)piece.x * p.group + head) * D + d) =
                __floats2half2_rn(o.x * inv, o.y * inv);
        } else {
            const int64_t part = ((int64_t)blockIdx.x * 2 + piece.w) * p.group + head;
            if (d == 0) p.part_ml[part] = make_float2(top, l);
            *reinterpret_cast<float2 *>(p.part_o + part * D + d) = o;
        }
    };

    int stage = 0;
    int seg = from.seg, s = first_s, lo = from.step, rot = 0;
    bool on = any;
    if (on) load_q(seg);
    while (on) {
        int pieces = 0;
        for (; pieces < hold && on; ++pieces) {
            const int j = pieces, end = piece_end(seg, s), live_warps = min(C::kWarps, end - lo);
            const bool whole = lo == 0 && end == team_steps_of(cum, s);
            const int mine = (warp - rot) & (C::kWarps - 1);
            if (!whole) (lo > 0 ? cut.x : cut.y) = seg;
            if (tid == 0) held[j] = make_int4(seg, rot, live_warps, whole ? 2 : lo > 0 ? 0 : 1);
            if (mine < live_warps) {
                st.clear();
                for (int c = lo + mine; c < end; c += C::kWarps) {
                    cp_async_wait<C::kStages - 1>();
                    __syncwarp();
                    const uint32_t kt = ring + stage * 2 * C::kTileBytes;
                    team_step<KIND, D, NT>(kt, kt + C::kTileBytes, meta[stage], q, p.scale_log2, p.group, st, lane);
                    __syncwarp();
                    issue(stage);
                    if (++stage == C::kStages) stage = 0;
                }
            }
            rot = (rot + end - lo) % C::kWarps;
            seg = team_next(cum, p.num_seqs, heads, seg, s);
            lo = 0;
            on = more(seg);
            if (on) load_q(seg);  // the next piece's queries come while this one's outputs go
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int live = min(8, p.group - n * 8);
                if (mine < live_warps) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float l = st.l[n][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(kFullMask, l, d);
                        const int h = 2 * t + e;
                        if (h < live) {
                            const int at = warp * 8 + j * red_heads + h;
                            if (g == 0) ml[at] = make_float4(st.m[n][e], l, power_of_2(st.e), 0.f);
                            float *dst = red + at * C::kPitch;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                if (C::kWide) {
                                    dst[16 * i + g] = st.o[n][i][e];
                                    dst[16 * i + g + 8] = st.o[n][i][2 + e];
                                } else {
                                    *reinterpret_cast<float2 *>(dst + 16 * i + 2 * g) =
                                        make_float2(st.o[n][i][e], st.o[n][i][2 + e]);
                                }
                            }
                        }
                    }
                }
                if (NT > 1) {  // a piece at a time, eight heads at a time
                    __syncthreads();
                    for (int i = tid; i < live * (D / 2); i += C::kThreads)
                        join(i / (D / 2), n * 8 + i / (D / 2), i % (D / 2) * 2, held[0]);
                    if (n + 1 < NT) __syncthreads();
                }
            }
        }
        if (NT == 1) {
            __syncthreads();
            for (int i = tid; i < pieces * red_heads * (D / 2); i += C::kThreads) {
                const int row = i / (D / 2), j = row / red_heads;
                join(row, row - j * red_heads, i % (D / 2) * 2, held[j]);
            }
        }
        __syncthreads();
    }
    if (tid == 0) p.cut[blockIdx.x] = cut;
}

// Joins the parts of segments that CTA boundaries cut: block (c, h) takes head h
// of the segment whose first part is CTA c's last piece.
constexpr int kTeamJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kTeamJoinThreads) team_join_kernel(const __grid_constant__ TeamParams p) {
    constexpr int kWarps = kTeamJoinThreads / 32, kPer = D / 32;
    __shared__ float2 ml[kWarps];
    __shared__ float out[kWarps][D];
    grid_dependency_wait();
    launch_dependents();
    const int c = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A warp's part i: CTA c's last piece, then the first pieces of the CTAs behind it.
    float2 x;
    float y[kPer];
    auto load = [&](int i) {
        const int64_t part = ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * p.group + h;
        x = p.part_ml[part];
#pragma unroll
        for (int k = 0; k < kPer; ++k) y[k] = p.part_o[part * D + k * 32 + lane];
    };
    // The first ones are loaded along with what tells whether they are any.
    const bool in = c + warp < (int)gridDim.x;
    if (in) load(warp);
    const int seg = p.cut[c].y;
    int i = c + 1 + (int)threadIdx.x;
    int more = i < (int)gridDim.x ? p.cut[i].x : -1;
    if (seg < 0) return;
    int parts = 1;
    while (true) {
        const int n = __syncthreads_count(more == seg);
        parts += n;
        if (n < kTeamJoinThreads) break;
        i += kTeamJoinThreads;
        more = i < (int)gridDim.x ? p.cut[i].x : -1;
    }
    float top = -CUDART_INF_F, l = 0.f, o[kPer] = {};
    for (int i = warp; i < parts; i += kWarps) {
        if (i != warp) load(i);
        const float to = fmaxf(top, x.x), ref = to == -CUDART_INF_F ? 0.f : to;
        const float f = team_exp2(top - ref), fx = team_exp2(x.x - ref);
        top = to;
        l = l * f + x.y * fx;
#pragma unroll
        for (int k = 0; k < kPer; ++k) o[k] = o[k] * f + y[k] * fx;
    }
    if (lane == 0) ml[warp] = make_float2(top, l);
#pragma unroll
    for (int k = 0; k < kPer; ++k) out[warp][k * 32 + lane] = o[k];
    __syncthreads();
    if (threadIdx.x < D) {
        float all = -CUDART_INF_F, sum = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all = fmaxf(all, ml[w].x);
        const float ref = all == -CUDART_INF_F ? 0.f : all;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = team_exp2(ml[w].x - ref);
            sum = fmaf(ml[w].y, f, sum);
            y = fmaf(out[w][threadIdx.x], f, y);
        }
        const int64_t row = (int64_t)seg * p.group + h;
        p.out[row * D + threadIdx.x] = __float2half_rn(sum == 0.f ? 0.f : y / sum);
    }
}

template <int KIND, int D, int NT>
TeamKernel team_kernel_info_of() {
    using C = TeamConfig<KIND, D, NT>;
    TeamKernel k;
    k.fn = reinterpret_cast<const void *>(&team_kernel<KIND, D, NT>);
    k.smem_fixed = C::kCum + 8;
    k.threads = C::kThreads;
    k.ctas_per_sm = C::kCtas;
    k.step_rows = C::kRows;
    return k;
}

template <int KIND, int D>
TeamKernel team_kernel_info(int group) {
    return group <= 8 ? team_kernel_info_of<KIND, D, 1>() : team_kernel_info_of<KIND, D, 2>();
}

}  // namespace pkv

#endif  // PKV_TEAM_IMPL_CUH
