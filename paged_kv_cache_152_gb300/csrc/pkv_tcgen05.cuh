// pkv_tcgen05.cuh -- wrappers of the 5th-generation tensor-core instructions
// (tcgen05): tensor memory, matrix products, commits and fences.
#ifndef PKV_TCGEN05_CUH
#define PKV_TCGEN05_CUH

#include <stdint.h>

namespace pkv {

// Tensor memory: 128 lanes x 512 columns of 32 bits per SM.  An address holds
// the lane in bits 16-31 and the column in bits 0-15.  One whole warp
// allocates and frees.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_result, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
}

// Shared-memory matrix descriptor of a 128-byte-swizzled tile, its halves: the
// start address and the leading byte offset in units of 16 bytes (low), the
// stride byte offset, version 1 (bit 46) and swizzle mode 2 (bits 61-63) (high).
__device__ __forceinline__ uint32_t umma_desc_low(uint32_t addr, uint32_t leading_bytes) {
    return (addr & 0x3ffffu) >> 4 | (leading_bytes >> 4) << 16;
}
__host__ __device__ constexpr uint32_t umma_desc_high(uint32_t stride_bytes) { return stride_bytes >> 4 | 1u << 14 | 2u << 29; }

// Instruction descriptor of kind::f16 with fp16 operands and fp32
// accumulators: bit 4 the accumulator type, bit 16 set where B is stored with
// its N dimension contiguous, N / 8 at bit 17, M / 16 at bit 24.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int m, int n, bool b_n_major) {
    return 1u << 4 | (b_n_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(m / 16) << 24;
}

// The products are issued by one elected lane, but called by a whole converged
// warp with the same arguments, a chain of them in one statement: the
// descriptors can then stay in uniform registers, which the instruction reads,
// and the election is made once (from inside a one-lane branch each product
// cost 70 to 120 cycles to issue, more than it takes to compute).

#define PKV_MMA_HEAD                                                                                    \
    "{\n\t.reg .pred p, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\t" \
    "setp.ne.u32 p, %4, 0;\n\t"
// One product of the chain at offsets XA, XB of the operands' low words; the first adds to D only if asked.
#define PKV_MMA_SS(XA, XB, P)                                                              \
    "add.u32 x, %1, " XA ";\n\tadd.u32 y, %2, " XB ";\n\t"                                \
    "mov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"                                     \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " P ";\n\t"
#define PKV_MMA_TS(XA, XB, P)                                                              \
    "add.u32 x, %1, " XA ";\n\tadd.u32 y, %2, " XB ";\n\tmov.b64 b, {y, %5};\n\t"       \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, " P ";\n\t"

// S (tensor memory) = Q (shared) . K^T (shared) over D = 64 or 128 dims, 16 at a
// time: 32 bytes apart inside a half of 64 dims, halves 16 KB apart.
template <int D>
__device__ __forceinline__ void umma_scores(uint32_t s, uint32_t q, uint32_t k, uint32_t idesc) {
    constexpr uint32_t high = umma_desc_high(1024);
    if (D == 64)
        asm volatile(PKV_MMA_HEAD PKV_MMA_SS("0", "0", "p") "setp.eq.u32 p, 0, 0;\n\t" PKV_MMA_SS("2", "2", "p")
                         PKV_MMA_SS("4", "4", "p") PKV_MMA_SS("6", "6", "p") "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(0), "r"(high)
                     : "memory");
    else
        asm volatile(PKV_MMA_HEAD PKV_MMA_SS("0", "0", "p") "setp.eq.u32 p, 0, 0;\n\t" PKV_MMA_SS("2", "2", "p")
                         PKV_MMA_SS("4", "4", "p") PKV_MMA_SS("6", "6", "p") PKV_MMA_SS("1024", "1024", "p")
                             PKV_MMA_SS("1026", "1026", "p") PKV_MMA_SS("1028", "1028", "p")
                                 PKV_MMA_SS("1030", "1030", "p") "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(0), "r"(high)
                     : "memory");
}

// O (tensor memory) = P (tensor memory) . V (shared) (+ O) over 64 rows of V,
// 16 at a time: 8 columns of P (fp16 pairs), 2048 bytes of V.
__device__ __forceinline__ void umma_weighted(uint32_t o, uint32_t p, uint32_t v, uint32_t idesc, bool add) {
    asm volatile(PKV_MMA_HEAD PKV_MMA_TS("0", "0", "p") "setp.eq.u32 p, 0, 0;\n\t" PKV_MMA_TS("8", "128", "p")
                     PKV_MMA_TS("16", "256", "p") PKV_MMA_TS("24", "384", "p") "}" ::"r"(o),
                 "r"(p), "r"(v), "r"(idesc), "r"((uint32_t)add), "r"(umma_desc_high(1024))
                 : "memory");
}

// One arrival on the barrier once every product the elected lane has issued so
// far is complete.  Called by the whole warp as well.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// A plain arrival by the elected lane.
__device__ __forceinline__ void umma_arrive(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define PKV_OUT32(v)                                                                                          \
    "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),           \
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), \
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]),            \
        "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),            \
        "=r"(v[30]), "=r"(v[31])
#define PKV_IN32(v)                                                                                         \
    "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),      \
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),      \
        "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),     \
        "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
#define PKV_LIST32                                                                                          \
    "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, " \
    "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}"

// 32 columns of the warp's 32 lanes (lanes 32 * (warp % 4) and up): thread i
// holds lane i's.  The values are there after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " PKV_LIST32 ", [%32];" : PKV_OUT32(v) : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " PKV_LIST32 ";" ::PKV_IN32(v), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Keeps every use of v behind the wait that precedes this in program order.
__device__ __forceinline__ void tmem_pin32(uint32_t (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}

// One 32-byte store of eight 32-bit words; dst 32-byte aligned.
__device__ __forceinline__ void store_32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Two fp32 values in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x, 2 ulp (the hardware's ex2; subnormal results become zero).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace pkv

#endif  // PKV_TCGEN05_CUH
