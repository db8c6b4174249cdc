// Pieces of the kernels on the tcgen05 tensor cores (sm_103a): barriers and their bounded waits, TMA
// copies, products with operands in shared memory or TMEM, TMEM loads and stores, and the operands'
// descriptors and swizzle.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---- PTX -------------------------------------------------------------------------------

__device__ __forceinline__ unsigned smem_u32(const void *p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(unsigned bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One arrival for the whole warp: the barrier counts warps (an arrival of every thread would be
// 32 updates of one word, one after the other).
__device__ __forceinline__ void warp_arrive(unsigned bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// A wait gives up after this many ns: longer than any call's CTA waits for another's state.
constexpr unsigned long long kGiveUp = 10000000000;

// Waits for the barrier's phase of `parity`; false where it gave up.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity) {
    unsigned long long start = 0;
    while (true) {
        unsigned done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        unsigned long long now;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
        if (!start) start = now;
        if (now - start > kGiveUp) return false;
    }
}

// The same as straight-line code, which leaves a warp's control flow uniform as the compiler sees it:
// `dead` becomes nonzero where the wait gave up (after 40 million looks: 1.3 s, measured), and waits
// no more where it was.  For waits on the CTA's own work alone.  (Looks, and not try_wait, whose
// suspended threads come back some 30 cycles later: 3 % of the delta rule's prompts.)
__device__ __forceinline__ void mbar_pass(unsigned bar, unsigned parity, unsigned &dead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "@p bra OUT;\n\t"
        "AGAIN:\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra OUT;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, 40000000;\n\t"
        "@q bra AGAIN;\n\t"
        "mov.u32 %0, 1;\n\t"
        "OUT:\n\t}"
        : "+r"(dead)
        : "r"(bar), "r"(parity)
        : "memory");
}

// One lane of a whole warp: nonzero there.
__device__ __forceinline__ unsigned elect_one() {
    unsigned leader;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(leader));
    return leader;
}

__device__ __forceinline__ void tma_load(unsigned dst, const CUtensorMap *map, unsigned bar, int x,
                                         int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, unsigned src, int x, int y,
                                          int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 columns of the thread's TMEM lane.
__device__ __forceinline__ void tc_load16(unsigned addr, unsigned (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tc_store16(unsigned addr, const unsigned (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tc_store8(unsigned addr, const unsigned (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

// d (+)= a b, a and b in shared memory.
__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b,
                                       unsigned idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// d (+)= a b, a in TMEM.
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned idesc,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// The same, and the commit, by the one lane that elect_one() named, in code that the whole warp runs:
// operands are then uniform to the compiler, and a product takes 23 cycles to issue (52 from one
// lane's own branch: as long as an MMA of N = 64 runs).
__device__ __forceinline__ void mma_ts_of(unsigned leader, unsigned d, unsigned a,
                                          unsigned long long b, unsigned idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tc_commit_of(unsigned leader, unsigned bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar),
        "r"(leader)
        : "memory");
}

// Shared-memory operand in rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart.
// Read along the rows (K-major) it is [rows][64 k]; read across them (MN-major) it is
// [64 mn][rows k], further blocks of 64 mn `block_bytes` apart.
__device__ __forceinline__ unsigned long long operand(unsigned addr, unsigned block_bytes) {
    return static_cast<unsigned long long>((addr >> 4) & 0x3fff) |
           (static_cast<unsigned long long>(block_bytes >> 4) << 16) |
           (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: bf16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr unsigned instruction(int n, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn_major ? 1u << 15 : 0u) |
           (b_mn_major ? 1u << 16 : 0u) | (static_cast<unsigned>(n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// Address of 16-byte piece `piece` of row `row` of a swizzled tile.
__device__ __forceinline__ unsigned swizzled(unsigned tile, int row, int piece) {
    return tile + row * 128 + ((piece ^ (row & 7)) << 4);
}

__device__ __forceinline__ uint4 load_smem16(unsigned addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void store_smem16(unsigned addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void widen16(const uint4 &w, float (&v)[8]) {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// 2^x by the hardware's approximation (2 ulp), results below 2^-126 as 0: for weights that are
// rounded to bf16 next, or kept to 2^-17 in two parts.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace
