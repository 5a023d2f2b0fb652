// tcgen05, TMA and mbarrier helpers of the prompt kernels (sm_103a).
#pragma once

#include "qevict_internal.cuh"

namespace qevict {

__device__ __forceinline__ void tc_mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void tc_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool tc_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// A wait that every role of a CTA shares a way out of: it gives up when another
// role has (the flag in shared memory) or when about two seconds have passed,
// and then raises the flag itself. False: the role must stop.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int *stop) {
    if (tc_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc_try_wait(bar, parity)) {
        if (*stop) return false;
        if (clock64() - t0 > kDefaultWaitCycles) {
            *stop = 1;
            return false;
        }
    }
    return true;
}

// Two or three barriers; where all are through already, for the price of one.
__device__ __forceinline__ bool tc_wait2(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, volatile int *stop) {
    const bool x = tc_try_wait(a, pa), y = tc_try_wait(b, pb);
    return (x || tc_wait(a, pa, stop)) && (y || tc_wait(b, pb, stop));
}
__device__ __forceinline__ bool tc_wait3(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, uint32_t c, uint32_t pc,
                                         volatile int *stop) {
    const bool x = tc_try_wait(a, pa), y = tc_try_wait(b, pb), z = tc_try_wait(c, pc);
    return (x || tc_wait(a, pa, stop)) && (y || tc_wait(b, pb, stop)) && (z || tc_wait(c, pc, stop));
}

__device__ __forceinline__ void tc_tma_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int u,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
}

// the descriptor of a tensor map into the cache, ahead of its first copy
__device__ __forceinline__ void tc_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ bool tc_elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 512 or fewer tensor-memory columns (a power of two), the address to *slot in
// shared memory; one whole warp calls each of the two.
template <int COLS>
__device__ __forceinline__ void tc_alloc(uint32_t slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void tc_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle, as their low words (the
// high word is kDescHi). K-major: rows of 64 channels (128 B), 8-row groups 1024
// B apart. MN-major (rows run along K): 8-row groups along K 1024 B apart,
// blocks of 64 along M or N `lead` B apart.
constexpr uint32_t kDescHi = (1u << 14) | (2u << 29) | (1024u >> 4);
__device__ __forceinline__ uint32_t tc_desc_k(uint32_t addr) { return (1u << 16) | ((addr & 0x3ffff) >> 4); }
__device__ __forceinline__ uint32_t tc_desc_mn(uint32_t addr, uint32_t lead) {
    return ((lead >> 4) << 16) | ((addr & 0x3ffff) >> 4);
}
// Instruction descriptor: bf16 x bf16 -> fp32, M = 128; B MN-major or K-major.
__host__ __device__ constexpr uint32_t tc_idesc(bool b_mn, uint32_t n = 128) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// D (+)= A B over K = 16, A in shared (ss) or tensor (ts) memory. The elected lane
// issues them in a warp whose lanes otherwise keep step (they wait for the same
// barriers and hold the same operands): the operands then come out of uniform
// registers, and an issue keeps ahead of the 64 cycles that a 128 x 128 x 16
// product takes (from a branch of one thread an issue took 80 to 97 cycles).
// Keeping step is also a condition of correctness. All lanes of the issuing warp wait
// for the same barriers (each polls, then a vote over the whole warp); the issue is
// a plain branch on the flag that tc_elect gave, with nothing between the wait and it
// that only some lanes run; a __syncwarp follows it. The operands lie in registers that
// the warp shares: forms in which lanes could run ahead (the elected lane polling for the
// others; lanes polling unlike barriers, the instruction itself predicated) ended in an
// illegal memory access.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
        : "memory");
}
// a 128 x N x 128 product of two tiles in shared memory, halves of 64 channels 128 and N rows apart
template <int N>
__device__ __forceinline__ void tc_mma_tile(uint32_t d, uint32_t a, uint32_t b) {
    const uint32_t da = tc_desc_k(a), db = tc_desc_k(b), ha = 128 * 128 / 16, hb = N * 128 / 16;
#pragma unroll
    for (int s = 0; s < 8; ++s)
        tc_mma_ss(d, da + (s >> 2) * ha + (s & 3) * 2, db + (s >> 2) * hb + (s & 3) * 2, tc_idesc(false, N), s > 0);
}
// all products issued so far arrive on `bar` when they have ended
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_ld32(uint32_t addr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"f"(r[0]),
        "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]),
        "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]),
        "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
        "f"(r[29]), "f"(r[30]), "f"(r[31]), "r"(addr)
        : "memory");
}
// 16 columns (32 packed bf16) of this warp's 32 lanes
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// ties loaded registers to the wait before it, so that no use is scheduled above
__device__ __forceinline__ void tc_tie(float (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile(""
                     : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]),
                       "+f"(r[i + 6]), "+f"(r[i + 7]));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Dynamic scheduling: a running CTA takes over the next CTA of its grid that has not
// started. The request's answer (16 bytes) completes on `bar`; after a false
// answer there is nothing left to ask for.
__device__ __forceinline__ void tc_ask(uint32_t answer, uint32_t bar) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the last answer has been read
    tc_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
        "r"(bar)
        : "memory");
}
__device__ __forceinline__ bool tc_answer(uint32_t answer, uint32_t &block) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(ok), "=r"(block)
        : "r"(answer)
        : "memory");
    return ok != 0;
}

// pairs of fp32 in one register pair
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// clusters: the same shared-memory address in another CTA, and loads from it
__device__ __forceinline__ uint32_t cl_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cl_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 cl_ld2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
// the pair at `p` of CTA `rank`; its type has to promise the alignment that the load needs
template <class T>
__device__ __forceinline__ uint2 cl_pair(const T *p, uint32_t rank) {
    static_assert(sizeof(T) == 8 && alignof(T) >= 8, "a pair of words on an 8-byte boundary");
    const float2 x = cl_ld2(cl_addr(smem_u32(p), rank));
    return make_uint2(__float_as_uint(x.x), __float_as_uint(x.y));
}
__device__ __forceinline__ float cl_ld1(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int cl_ldi(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cl_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float tc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace qevict
