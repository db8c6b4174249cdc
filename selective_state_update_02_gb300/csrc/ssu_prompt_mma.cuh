// Prompts in chunked matrix form on the tcgen05 tensor cores (sm_103a), instantiated by
// ssu_prompt.cu beside the token-by-token kernel of ssu_prompt.cuh.
//
// Mathematics.  Over a chunk of Q = 128 tokens with a_t = dtv_t A and s(j, i] = a_{j+1} + .. +
// a_i, the recurrence S_t = exp(a_t) S_{t-1} + dtv_t x_t (x) B_t, y_t = S_t C_t + D x_t reads
//
//   y_i = sum_{j <= i} (C_i . B_j) exp(s(j, i]) dtv_j x_j  +  exp(s(0, i]) C_i S  +  D x_i
//   S'  = exp(s(0, Q]) S  +  sum_j (exp(s(j, Q]) dtv_j x_j) (x) B_j
//
// that is four matrix products per chunk and head: G = C B^T [Q x Q], I = C S^T [Q x P],
// Y = M X [Q x P] with M = G times the masked decays plus D on the diagonal, and U = B^T W [N x P]
// with W the weighted tokens.  A column is 64 rows of one head's state; a CTA takes two columns of
// one group through a prompt's stretch, chunk after chunk, so that G and every read of B and C are
// shared, and I and U of both are one product 128 wide (an MMA of N = 128 takes 63 cycles where two
// of N = 64 take 96: those read the first operand from shared memory twice).  The states stay in
// registers (thread n holds column n of the 64 rows).  G, I, Y and U accumulate in TMEM (all 512
// columns with M, which goes back there as Y's first operand), so a CTA has its SM to itself.
//
// Precision.  C, B and X are bf16 and exact.  M and the state that enters I are rounded to bf16
// (2^-9 of a term in the mean square, as much as the bf16 readout itself carries).  W decides
// the state that is carried on, so it enters as the sum of three bf16 parts (24 bits: all of an
// fp32 value; with two a head's state is up to 3e-6 off in the 2-norm, with three below 4.4e-7)
// where the state is kept in fp32, of two where it is rounded to bf16 in the end, and runs in fp32
// either way.
// Exponents are sums over short runs that never cross a chunk: within blocks of 32 tokens
// prefix and suffix sums, between blocks the block totals, so no exponent is a difference of
// two large sums except inside the diagonal block, whose weights are rounded to bf16 anyway.
// An a_t beyond +-256 (log2) is cut there: exp is then 0 (or infinite) all the same, and a cut
// sum stays small enough to be exact.  A NaN stays one, and with it all that comes after its token.
//
// Stretches.  A prompt that is long for the device is cut into stretches.  A first pass (kFirst)
// runs U alone over every stretch but a prompt's last, the first from the prompt's state and the
// others from zero; the second pass starts a stretch from the results of those before it.  Where
// there are more stretches than SMs, CTAs share their chunks along a line (below).
//
// What bounds it: the chain of a chunk's steps.  Of some 8,300 cycles per pair of columns and chunk
// (measured inside the kernel; 8 prompts of 4096 tokens through 64 heads: 264 us, 2.2 TB/s, 0.3 of
// the tensor pipe) M takes 2,000, W 2,000, Y and U 2,600 with the decays and the readout under
// them, I 500 and the state 650; the tensor pipe is busy for 3,300 of them, issue slots for a
// third.
// Products that run under M or the readout slow their TMEM loads by more than they hide: M a chunk
// ahead measured 1.11 of the time, W before M 1.14, sixteen warps 1.04 to 1.12, one column per CTA
// and two CTAs per SM 1.34.  A stretch costs 5 us on top (first loads and decays, the state in and
// out).

#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssu_prompt.cuh"

namespace {

constexpr int kChunk = 128;      // tokens per chunk: the MMA's M
constexpr int kSlab = 64;        // state rows per CTA: the MMA's N
constexpr int kPair = 2;         // columns (a head's 64-row slab) per CTA, of one group
constexpr int kCompute = kPair * kChunk;       // threads of the elementwise work: a row each
constexpr int kPromptThreads = kCompute + 96;  // one warp to issue, two to look x over and store
constexpr int kTileBytes = kChunk * 128;  // a 64-column bf16 tile of 128 rows
constexpr float kLog2e = 1.4426950408889634f;

struct PromptMmaParams {
    PromptParams q;
    int seg;              // chunks per stretch
    int slabs;            // headdim / 64
    int after_first;      // a first pass was launched before the second
    float *hand;          // [CTA of the line][column of the pair][64 p][N]: states handed on
    unsigned *turn;       // CTAs of the line begun; then per CTA whether its state is handed on
    float *local;         // [stretch][head * slabs + slab][64 p][N]
    float *decay;         // [stretch][head * slabs + slab]: log2 of the stretch's decay
};

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
           (static_cast<unsigned>(kChunk >> 4) << 24);
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
// rounded to bf16 next.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- the kernel ------------------------------------------------------------------------

// Shared memory: tiles first (1024-byte aligned), then the per-token values.  x, S and W hold one
// tile per column, side by side, as the two blocks of an operand 128 wide.  B has two places (the
// next chunk's G is formed before this one's U is done); W's second part takes S's place, which
// I has read by then, and gives it back when U is done; readouts leave from x's place.  W's third
// part has half a tile per column for tokens 64 .. 127; for tokens 0 .. 63, where dstate is 128 and
// no room is left, it takes the upper columns of C's place, which the next C gets once those
// products (U's first) are done.
template <int N>
struct PromptSmem {
    static constexpr int kBlocks = N / 64;  // 64-column tiles of B and C
    static constexpr int kC = 0;
    static constexpr int kB = kC + kBlocks * kTileBytes;
    static constexpr int kX = kB + 2 * kBlocks * kTileBytes;
    static constexpr int kW1 = kX + kPair * kTileBytes;
    static constexpr int kW2 = kW1 + kPair * kTileBytes;  // also S: bf16 [n][64 p]
    static constexpr int kW3 = kW2 + kPair * kTileBytes;  // tokens 64 .. 127
    static constexpr int kW3First = N == 128 ? kC + kTileBytes : kW3 + kTileBytes;  // 0 .. 63
    static constexpr int kVec = kW3 + (N == 128 ? 1 : 2) * kTileBytes;
    // floats of a chunk's tokens: v0 (128), pairs (prefix, dtv) (256), block totals (4), the
    // head's dt_bias, A log2 e and D (4); for this chunk and the next, for each column
    static constexpr int kConst = 3 * kChunk + 4;
    static constexpr int kVecFloats = kConst + 4;
    static constexpr int kBars = kVec + 2 * kPair * kVecFloats * 4;
    // per column, for this chunk and the next: whether x holds infinities or NaN, and from which
    // token of the chunk on each state row is lost to them
    static constexpr int kLost = kBars + 128;
    static constexpr int kLostInts = 4 + kSlab;
    static constexpr int kTotal = kLost + 2 * kPair * kLostInts * 4;
};

// A copy of v that the compiler takes for another value.
__device__ __forceinline__ unsigned opaque(unsigned v) {
    asm volatile("" : "+r"(v));
    return v;
}

// Where a CTA works.
struct Stretch {
    long long b;       // prompt; -1: past the last stretch
    long long g;       // the stretch's number in the call
    int index, count;  // of the prompt's stretches
};

// Prompts that overlap.  The workspace has room for the stretches of prompts that do not, so a
// prompt that begins before the end of a good one before it is a bad one too.  That takes offsets
// that run backwards somewhere, and is looked for only where some do.

// The largest of the ends of the thread's earlier prompts (`seen`, of all threads) and of those of
// the threads before it (`end`; 0: none); all threads call it, and `scan` is free afterwards.
__device__ __forceinline__ int end_before(int end, int seen, long long *scan) {
    constexpr int kWarps = kPromptThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = end;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl = max(incl, o);
    }
    const int earlier = __reduce_max_sync(0xffffffffu, seen);
    __syncthreads();
    if (lane == 31) scan[warp] = static_cast<long long>(earlier) << 32 | incl;
    __syncthreads();
    int most = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) most = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        most = max(most, static_cast<int>(scan[w] >> 32));
        if (w < warp) most = max(most, static_cast<int>(scan[w]));
    }
    __syncthreads();
    return most;
}

// The same question about one prompt that begins at `begin`, by one thread.
template <bool kIdx64>
__device__ __forceinline__ bool begins_early(const PromptParams &q, long long b, long long begin) {
    long long slot, lo, hi;
#pragma unroll 1
    for (long long j = 0; j < b; ++j)
        if (load_prompt<kIdx64>(q, j, false, slot, lo, hi) && lo < hi && begin < hi) return true;
    return false;
}

// The stretch that is the `at`-th of the call, or (kFirst) of those that are not their prompt's
// last; all threads get the answer.  With `all`, every prompt is looked at and the bad ones
// counted.
template <bool kIdx64, bool kFirst>
__device__ __forceinline__ Stretch find_stretch(const PromptMmaParams &m, long long at, bool all,
                                                long long *scan) {
    constexpr int kWarps = kPromptThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned per = static_cast<unsigned>(m.seg) * kChunk;  // at most 2^30
    long long before = 0;  // stretches of the prompts before: all << 32 | those not the last
    bool backwards = false;  // offsets that run backwards, up to these prompts
    int seen = 0;            // the largest end of the thread's earlier prompts
    if (tid == 0) scan[kWarps] = -1;
    auto pick = [](long long v) { return kFirst ? v & 0xffffffffll : v >> 32; };
#pragma unroll 1
    for (long long b0 = 0; b0 < m.q.p.batch && (all || at >= pick(before)); b0 += kPromptThreads) {
        const long long b = b0 + tid;
        long long n = 0, slot, lo = 0, hi = 0;
        bool good = b < m.q.p.batch && load_prompt<kIdx64>(m.q, b, all, slot, lo, hi);
        backwards = __syncthreads_or(backwards || lo > hi);
        const int ends = good && lo < hi ? static_cast<int>(hi) : 0;
        if (backwards && end_before(ends, seen, scan) > lo && ends) {
            good = false;
            if (all) record_skip(m.q.p, b);
        }
        seen = max(seen, ends);
        if (good) {
            n = (static_cast<unsigned>(hi - lo) + per - 1) / per;  // tokens fit 31 bits
            if (n == 0 && m.q.fresh && m.q.fresh[b]) n = 1;  // only clears the slot
        }
        const long long mine = n << 32 | (n > 1 ? n - 1 : 0);
        long long incl = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long start = before + incl - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) start += scan[w];
            before += scan[w];
        }
        const long long index = at - pick(start);
        if (index >= 0 && index < pick(mine)) {
            scan[kWarps] = b;
            scan[kWarps + 1] = (start >> 32) + index;
            scan[kWarps + 2] = index << 32 | n;
        }
    }
    __syncthreads();
    return Stretch{scan[kWarps], scan[kWarps + 1], static_cast<int>(scan[kWarps + 2] >> 32),
                   static_cast<int>(scan[kWarps + 2])};
}

// The passes: over every stretch but a prompt's last, for the states alone; over every stretch,
// one or (along the line) several parts of them per CTA.
enum class Pass { kFirst, kSecond, kLine };

// What a CTA is working on: chunks c0 .. c1 - 1 of a stretch (c1 < 0: to its end), for the `cta`-th
// pair of columns.
struct Part {
    long long b, g;    // as in Stretch
    int index, count;
    int cta, c0, c1;
    int more;          // 0: no part
    int turn;          // the CTA's place among those of the line
    // where the part's stretch begins in the line, and the CTA's share of the line
    long long at, begin, end;
    int chunks;        // of the stretch
    int mixed;         // some prompt's offsets run backwards
};

// Chunks and stretches of prompt b (tokens lo .. hi - 1), packed as chunks << 32 | stretches; none
// for one that is bad by itself.
template <bool kIdx64>
__device__ __forceinline__ unsigned long long prompt_extent(const PromptMmaParams &m, long long b,
                                                            bool counts, long long &lo,
                                                            long long &hi) {
    long long slot;
    lo = hi = 0;
    if (b >= m.q.p.batch || !load_prompt<kIdx64>(m.q, b, counts, slot, lo, hi)) return 0;
    const unsigned chunks = static_cast<unsigned>((hi - lo + kChunk - 1) / kChunk);
    unsigned n = (chunks + m.seg - 1) / m.seg;
    if (n == 0 && m.q.fresh && m.q.fresh[b]) n = 1;  // only clears the slot
    return static_cast<unsigned long long>(chunks) << 32 | n;
}

__device__ __forceinline__ int stretch_chunks(const PromptMmaParams &m, unsigned long long extent,
                                              int index) {
    const int n = static_cast<int>(extent), chunks = static_cast<int>(extent >> 32);
    return index == n - 1 ? chunks - index * m.seg : m.seg;
}

// The line: every stretch `ctas` times (once per pair of columns), two places per chunk and one
// for what a part costs before its first chunk and after its last; cut evenly, wherever that
// falls, so that CTAs end together (8 prompts of 32 chunks, 32 pairs, 152 CTAs: 264 us, 0.9 of
// the time of whole stretches in two rounds).  A CTA goes through its share backwards: a stretch cut by its end
// first, whose state goes to the next CTA, and the one that the CTA before began last, when that
// one has long handed its state on.  Turns are given out as CTAs begin, so a CTA waits for those
// alone that run already.
__device__ __forceinline__ void set_chunks(Part &w) {
    w.c0 = w.begin > w.at ? static_cast<int>((w.begin - w.at + 1) / 2) : 0;
    w.c1 = static_cast<int>(min((w.end - w.at + 1) / 2, 1ll << 30));
    if (w.c1 >= w.chunks) w.c1 = -1;
}

// The part before, in the line, that has something to do (one thread).
template <bool kIdx64>
__device__ __forceinline__ void step_back(const PromptMmaParams &m, Part &w, int ctas) {
    do {
        w.more = w.at > w.begin;
        if (!w.more) return;
        if (--w.cta < 0) {
            w.cta = ctas - 1;
            --w.g;
            if (--w.index < 0) {
                unsigned long long extent;
                do {
                    long long lo, hi;
                    extent = prompt_extent<kIdx64>(m, --w.b, false, lo, hi);
                    if (w.mixed && lo < hi && extent && begins_early<kIdx64>(m.q, w.b, lo))
                        extent = 0;
                } while (static_cast<unsigned>(extent) == 0);
                w.count = static_cast<int>(extent);
                w.index = w.count - 1;
                w.chunks = stretch_chunks(m, extent, w.index);
            } else {
                w.chunks = m.seg;  // not its prompt's last
            }
        }
        w.at -= 2 * w.chunks + 1;
        set_chunks(w);
    } while (w.chunks && (w.c1 < 0 ? w.chunks : w.c1) <= w.c0);
}

// The last part of the CTA's share; all threads call it.
template <bool kIdx64>
__device__ __forceinline__ void find_line(const PromptMmaParams &m, int ctas, Part &w,
                                          long long *scan) {
    constexpr int kWarps = kPromptThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto places = [&](unsigned long long v) {
        return (2 * static_cast<long long>(v >> 32) + static_cast<unsigned>(v)) * ctas;
    };
    if (tid == 0) {
        w.more = 0;
        w.turn = static_cast<int>(atomicAdd(m.turn, 1u));
    }
    // the extent of a prompt that does not overlap with one before it, all threads side by side
    auto apart = [&](long long b, int &seen, bool counts) {
        long long lo, hi;
        unsigned long long extent = prompt_extent<kIdx64>(m, b, false, lo, hi);
        const int ends = extent && lo < hi ? static_cast<int>(hi) : 0;
        if (end_before(ends, seen, scan) > lo && ends) {
            extent = 0;
            if (counts) record_skip(m.q.p, b);
        }
        seen = max(seen, ends);
        return extent;
    };
    unsigned long long all;
    bool mixed = false;
    while (true) {
        bool backwards = false;
        int seen = 0;
        all = 0;
#pragma unroll 1
        for (long long b0 = 0; b0 < m.q.p.batch; b0 += kPromptThreads) {
            if (mixed) {
                all += apart(b0 + tid, seen, blockIdx.x == 0);
            } else {
                long long lo, hi;
                all += prompt_extent<kIdx64>(m, b0 + tid, blockIdx.x == 0, lo, hi);
                backwards |= lo > hi;
            }
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
        if (lane == 0) scan[warp] = static_cast<long long>(all);
        if (!__syncthreads_or(backwards && !mixed)) break;
        mixed = true;  // again, without those that overlap
    }
    all = 0;
#pragma unroll 1
    for (int k = 0; k < kWarps; ++k) all += static_cast<unsigned long long>(scan[k]);
    const long long total = places(all);
    // at least two places, so that every share has some chunk's first
    const long long each = max((total + gridDim.x - 1) / gridDim.x, 2ll);
    const long long begin = w.turn * each, end = min(begin + each, total);
    if (begin >= end) return;
    unsigned long long before = 0;
    int seen = 0;
#pragma unroll 1
    for (long long b0 = 0; end > places(before); b0 += kPromptThreads) {
        long long lo, hi;
        const unsigned long long mine = mixed ? apart(b0 + tid, seen, false)
                                              : prompt_extent<kIdx64>(m, b0 + tid, false, lo, hi);
        unsigned long long incl = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = static_cast<long long>(incl);
        __syncthreads();
        unsigned long long start = before + incl - mine;
#pragma unroll 1
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) start += static_cast<unsigned long long>(scan[k]);
            before += static_cast<unsigned long long>(scan[k]);
        }
        if (end > places(start) && end <= places(start + mine)) {
            const long long stretch = (2ll * m.seg + 1) * ctas;  // places of a whole one
            long long o = end - 1 - places(start);
            w.b = b0 + tid;
            w.count = static_cast<int>(mine);
            w.index = static_cast<int>(min(o / stretch, w.count - 1ll));
            w.g = static_cast<unsigned>(start) + w.index;
            w.chunks = stretch_chunks(m, mine, w.index);
            o -= w.index * stretch;
            w.cta = static_cast<int>(o / (2 * w.chunks + 1));
            w.at = end - 1 - (o - static_cast<long long>(w.cta) * (2 * w.chunks + 1));
            w.begin = begin, w.end = end;
            w.mixed = mixed;
            w.more = 1;
            set_chunks(w);
            if (w.chunks && (w.c1 < 0 ? w.chunks : w.c1) <= w.c0) step_back<kIdx64>(m, w, ctas);
        }
    }
}

// Decay sums of one chunk, by the four warps of one warpgroup (one token per thread, `row`): the
// token's weight up to the end of its 32 tokens, its prefix within them, dtv, the blocks' totals.
__device__ __forceinline__ void chunk_decays(float *vec, bool live, float dt, float bias, float A2,
                                             int row, int lane) {
    float dtv = 0.0f, a = 0.0f;
    if (live) {
        dtv = softplus_f32(dt + bias);
        a = dtv * A2;
        a = a < -256.0f ? -256.0f : a > 256.0f ? 256.0f : a;  // NaN stays: fminf would drop it
    }
    float up = a, down = a;  // inclusive prefix and suffix
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, x);
        const float d = __shfl_down_sync(0xffffffffu, down, x);
        if (lane >= x) up += u;
        if (lane + x < 32) down += d;
    }
    float after = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 31) after = 0.0f;
    vec[row] = dtv * exp2f(after);
    reinterpret_cast<float2 *>(vec + kChunk)[row] = make_float2(up, dtv);
    if (lane == 31) vec[3 * kChunk + row / 32] = up;
}

// Waits until the CTA whose flag it is has handed its state on; false where it gave up.
__device__ __forceinline__ bool handed_on(const unsigned *flag, int lane) {
    bool done = true;
    if (lane == 0) {
        unsigned long long start, now;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(start));
        while (true) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
            if (v) break;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
            done = now - start < kGiveUp;
            if (!done) break;
            __nanosleep(200);
        }
    }
    __syncwarp();  // what lane 0 has acquired is there for all lanes (a shuffle orders no memory)
    return __shfl_sync(0xffffffffu, done, 0);
}

// The CTA's place in the call, of which threads hold as little as they can: a group's columns (one
// is 64 rows of a head: column c is head c / slabs, slab c % slabs) go to CTAs in pairs, an odd
// last one alone (its CTA works on it twice and keeps one result).
__device__ __forceinline__ int columns_per_group(const PromptMmaParams &m) {
    return static_cast<int>(opaque(m.q.p.heads_per_group)) * m.slabs;
}

__device__ __forceinline__ int ctas_per_stretch(const PromptMmaParams &m) {
    return m.q.p.nheads / m.q.p.heads_per_group * ((columns_per_group(m) + 1) / 2);
}

__device__ __forceinline__ unsigned tiles_at(const unsigned char *raw) {
    return (opaque(smem_u32(raw)) + 1023u) & ~1023u;
}

constexpr int kIssuer = kCompute / 32;  // the issuing warp; the next one stores
constexpr int kBars = 13;

__device__ __forceinline__ void init_barriers(unsigned bars) {
    for (int i = 0; i < 7; ++i) mbar_init(bars + 8 * i, 1);
    for (int i = 7; i < 11; ++i) mbar_init(bars + 8 * i, kCompute / 32);
    mbar_init(bars + 88, 1);
    mbar_init(bars + 96, kPair);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

template <int N>
__device__ __forceinline__ int *lost_of(unsigned char *raw, unsigned phase) {
    using Smem = PromptSmem<N>;
    return reinterpret_cast<int *>(raw + (tiles_at(raw) - smem_u32(raw)) + Smem::kLost) +
           phase * (kPair * Smem::kLostInts);
}

__device__ __forceinline__ unsigned load_smem2(unsigned at) {
    unsigned short u;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
    return u;
}

__device__ __forceinline__ void store_smem2(unsigned at, unsigned v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<unsigned short>(v))
                 : "memory");
}

// Whether `valid` tokens' rows of a tile of x hold infinities or NaN (one warp, under M).
__device__ __forceinline__ bool look_over(unsigned x, int valid, int lane) {
    constexpr int kLoads = kTileBytes / 512;  // 4 rows each
    __nv_bfloat162 sum[4] = {};
    const __nv_bfloat162 zero{};
#pragma unroll 16
    for (int k = 0; k < kLoads; ++k) {
        const uint4 v = load_smem16(x + k * 512 + lane * 16);
        if (4 * k + lane / 8 >= valid) continue;  // no token of this prompt
        sum[0] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.x), zero, sum[0]);
        sum[1] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.y), zero, sum[1]);
        sum[2] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.z), zero, sum[2]);
        sum[3] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.w), zero, sum[3]);
    }
    sum[0] = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
    return __any_sync(0xffffffffu,
                      (reinterpret_cast<const unsigned &>(sum[0]) & 0x7fff7fffu) != 0);
}

// Takes them out; `lost` says from which token on a state row is lost to them.
__device__ __forceinline__ void take_out(unsigned x, int *lost, int valid, int lane) {
    for (int p = lane; p < kSlab; p += 32) lost[4 + p] = kChunk;
    __syncwarp();
#pragma unroll 1
    for (int row = lane; row < valid; row += 32)
#pragma unroll 1
        for (int p = 0; p < kSlab; ++p) {
            const unsigned at = swizzled(x, row, p / 8) + 2 * (p % 8);
            if ((load_smem2(at) & 0x7f80) != 0x7f80) continue;
            store_smem2(at, 0);
            atomicMin(lost + 4 + p, row);
        }
    fence_async_smem();
}

// One part, by all threads; false in those whose wait gave up.
//
// Roles.  One thread starts the loads and the products as their inputs become ready, another the
// stores.  Eight warps do the elementwise work, four per column, a thread per row (token of the
// chunk, TMEM lane, column n of the state).  Per chunk, with the barrier that each hand-over uses:
//
//   issue:    next B; [done] I -> i; [i] next C; [m, v] Y -> y; [w] U -> 3, u; [3] rest of C;
//             [b, c] next G -> g
//   compute:  [g] M, [i] I scaled -> m; [x] W -> w; the next chunk's decays; [y] readout into x's
//             place -> r; [u] S advanced and published -> done
//   store:    (two warps, a column each) [x] x looked over -> v; one: [r] readout out, then next x
//
// so Y runs under W, U under the decays and the readout, I and the loads under M.  (Readouts
// stored by the threads themselves kept the shared-memory pipe busy for thousands of cycles per
// chunk: 32 lines per instruction.)
template <int N, typename ST, bool kIdx64, Pass kPass>
__device__ __forceinline__ bool run_part(const PromptMmaParams &m, const CUtensorMap &map_x,
                                         const CUtensorMap &map_b, const CUtensorMap &map_c,
                                         const CUtensorMap &map_out, const Part &part, Part &next,
                                         unsigned char *raw, unsigned tmem) {
    constexpr bool kFirst = kPass == Pass::kFirst, line = kPass == Pass::kLine;
    using Smem = PromptSmem<N>;
    constexpr int kBlocks = Smem::kBlocks;
    constexpr int kParts = sizeof(ST) == 4 ? 3 : 2;  // bf16 parts of W
    const SsuParams &p = m.q.p;
    bool alive = true;
    const int tid = opaque(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const unsigned base = tiles_at(raw);
    const unsigned sC = base + Smem::kC, sB = base + Smem::kB, sX = base + Smem::kX;
    const unsigned sW1 = base + Smem::kW1, sW2 = base + Smem::kW2;
    const unsigned sS = sW2;
    const unsigned bars = base + Smem::kBars;
    const unsigned bar_b = bars, bar_c = bars + 8, bar_x = bars + 16, bar_g = bars + 24,
                   bar_i = bars + 32, bar_u = bars + 40, bar_y = bars + 48, bar_w = bars + 56,
                   bar_m = bars + 64, bar_done = bars + 72, bar_r = bars + 80, bar_3 = bars + 88,
                   bar_v = bars + 96;
    // TMEM columns: G (both columns'), M, I and then Y, U (each one after the other)
    const unsigned tG = opaque(tmem), tM = tG + 128, tY = tG + 256, tU = tG + 384;
    const int per_group = columns_per_group(m), pairs = (per_group + 1) / 2;
    const int columns = p.nheads * m.slabs;
    const int grp = part.cta / pairs;
    const int first_column = grp * per_group + 2 * (part.cta - grp * pairs);
    const bool paired = 2 * (part.cta - grp * pairs) + 1 < per_group;
    const long long b = part.b, g = part.g;
    long long slot, begin, end;
    load_prompt<kIdx64>(m.q, b, false, slot, begin, end);
    // tokens fit 31 bits
    const int start = static_cast<int>(begin) + part.index * m.seg * kChunk;
    const int from = start + part.c0 * kChunk;
    const bool last = part.index == part.count - 1 && part.c1 < 0;
    const int to = part.c1 >= 0 ? start + part.c1 * kChunk
                   : last       ? static_cast<int>(end)
                                : start + m.seg * kChunk;

    constexpr int kBBytes = kBlocks * kTileBytes;  // one place of B
    auto load_x = [&](int tok) {
        mbar_expect(bar_x, kPair * kTileBytes);
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
            const int c = first_column + (paired ? k : 0);
            tma_load(sX + k * kTileBytes, &map_x, bar_x, c % m.slabs * kSlab, c / m.slabs, tok);
        }
    };
    if (warp == kIssuer) {
        if (lane == 0) {
            auto load_b = [&](int tok, unsigned place) {
                mbar_expect(bar_b, kBBytes);
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
                    tma_load(sB + place * kBBytes + k * kTileBytes, &map_b, bar_b, k * 64, grp,
                             tok);
            };
            auto load_c = [&](int tok, int k) {
                if (k == 0) mbar_expect(bar_c, kBBytes);
                tma_load(sC + k * kTileBytes, &map_c, bar_c, k * 64, grp, tok);
            };
            constexpr bool kShared = kParts == 3 && N == 128;  // W3 and C's upper columns
            // Shared-memory address of a tile, from an opaque copy of the base: the operands' many
            // descriptors are worked out where they are used instead of held in registers.
            auto tile = [&](int offset) {
                unsigned at = base;
                asm volatile("" : "+r"(at));
                return at + offset;
            };
            auto product_g = [&](unsigned place) {
                const unsigned c = tile(Smem::kC), b = tile(Smem::kB) + place * kBBytes;
#pragma unroll
                for (int k = 0; k < N / 16; ++k) {
                    const unsigned off = (k / 4) * kTileBytes + (k % 4) * 32;
                    mma_ss(tG, operand(c + off, 0), operand(b + off, 0),
                           instruction(kChunk, false, false), k > 0);
                }
                tc_commit(bar_g);
            };
            if (from < to) {
                load_b(from, 0);
                if (!kFirst)
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k) load_c(from, k);
                load_x(from);
                if (!kFirst) {
                    alive = mbar_wait(bar_b, 0);
                    if (alive) alive = mbar_wait(bar_c, 0);
                    product_g(0);
                }
            }
            if constexpr (line) {  // the part to come, whose first tiles are then in L2
                next = part;
                step_back<kIdx64>(m, next, ctas_per_stretch(m));
                if (next.more) {
                    long long slot_, first, end_;
                    load_prompt<kIdx64>(m.q, next.b, false, slot_, first, end_);
                    const int at = static_cast<int>(first) +
                                   (next.index * m.seg + next.c0) * kChunk;
                    const int group = next.cta / pairs;
                    const int c = group * per_group + 2 * (next.cta - group * pairs);
                    for (int k = 0; k < kBlocks && at < end_; ++k) {
                        tma_prefetch(&map_b, k * 64, group, at);
                        tma_prefetch(&map_c, k * 64, group, at);
                    }
                    for (int k = 0; k < kPair && at < end_; ++k)
                        tma_prefetch(&map_x, min(c + k, columns - 1) % m.slabs * kSlab,
                                     min(c + k, columns - 1) / m.slabs, at);
                }
            }
            unsigned phase = 0;
            for (int tok = from; tok < to; tok += kChunk, phase ^= 1) {
                const bool more = tok + kChunk < to;
                // the next B takes the place that the chunk before this one's U has left
                if (kFirst && alive) alive = mbar_wait(bar_b, phase);
                if (more) load_b(tok + kChunk, phase ^ 1);
                if (!kFirst) {
                    if (tok + 2 * kChunk < to) {  // from HBM into L2 long before it is waited for
#pragma unroll
                        for (int k = 0; k < kPair; ++k) {
                            const int c = first_column + (paired ? k : 0);
                            tma_prefetch(&map_x, c % m.slabs * kSlab, c / m.slabs,
                                         tok + 2 * kChunk);
                        }
                    }
                    if (alive) alive = mbar_wait(bar_done, phase);  // S published, Y and U read
                    tc_fence_after();
                    const unsigned c_now = tile(Smem::kC), s_now = tile(Smem::kW2);
#pragma unroll
                    for (int k = 0; k < N / 16; ++k) {
                        const unsigned off = (k / 4) * kTileBytes + (k % 4) * 32;
                        mma_ss(tY, operand(c_now + off, 0), operand(s_now + k * 2048, N * 128),
                               instruction(kPair * kSlab, false, true), k > 0);
                    }
                    tc_commit(bar_i);
                    if (alive) alive = mbar_wait(bar_i, phase);
                    if (more)
#pragma unroll
                        for (int k = 0; k < (kShared ? 1 : kBlocks); ++k) load_c(tok + kChunk, k);
                    if (alive) alive = mbar_wait(bar_m, phase);
                    if (alive) alive = mbar_wait(bar_v, phase);
                    tc_fence_after();
                    const unsigned x_now = tile(Smem::kX);
#pragma unroll
                    for (int c = 0; c < kPair; ++c)
#pragma unroll
                        for (int k = 0; k < kChunk / 16; ++k)
                            mma_ts(tY + c * kSlab, tM + c * 64 + 8 * k,
                                   operand(x_now + c * kTileBytes + k * 2048, 0),
                                   instruction(kSlab, false, true), true);
                    tc_commit(bar_y);
                }
                if (alive) alive = mbar_wait(bar_w, phase);
                tc_fence_after();
                const unsigned b_now = tile(Smem::kB) + phase * kBBytes;
                const unsigned w1 = tile(Smem::kW1), w2 = tile(Smem::kW2), w3 = tile(Smem::kW3),
                               w3_first = tile(Smem::kW3First);
                auto product_u = [&](unsigned w, int kk, unsigned block, bool more_of_it) {
                    mma_ss(tU, operand(b_now + kk * 2048, N == 128 ? kTileBytes : 0),
                           operand(w, block), instruction(kPair * kSlab, true, true), more_of_it);
                };
                if constexpr (kParts == 3) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        product_u(w3_first + k * 2048, k, kTileBytes / 2, k > 0);
                    if (kShared && !kFirst) tc_commit(bar_3);
#pragma unroll
                    for (int k = 4; k < 8; ++k)
                        product_u(w3 + (k - 4) * 2048, k, kTileBytes / 2, true);
                }
                if (kShared && !kFirst) {  // (under the products just given)
                    if (alive) alive = mbar_wait(bar_3, phase);
                    if (more) load_c(tok + kChunk, 1);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k)  // the small parts first: sums lose less
                    product_u((k < 8 ? w2 : w1) + k % 8 * 2048, k % 8, kTileBytes,
                              kParts == 3 || k > 0);
                tc_commit(bar_u);
                if (!kFirst && more) {  // every reader of G has passed m
                    if (alive) alive = mbar_wait(bar_b, phase ^ 1);
                    if (alive) alive = mbar_wait(bar_c, phase ^ 1);
                    product_g(phase ^ 1);
                }
                if (kFirst && more) load_x(tok + kChunk);  // x is in registers, or past them
                if (alive) alive = mbar_wait(bar_u, phase);
            }
        }
        __syncwarp();
    } else if (warp > kIssuer) {
        // Looks x over before Y reads it; then whole chunks go out as tiles (the compute threads
        // store a prompt's last, shorter one).
        if (!kFirst) {
            unsigned phase = 0;
            for (int tok = from; tok < to; tok += kChunk, phase ^= 1) {
                const int valid = to - tok < kChunk ? to - tok : kChunk;
                if (alive) alive = mbar_wait(bar_x, phase);
                // In the product with M a token's x meets the weights of all rows, zeros before the
                // token, and zero times an infinity or NaN is NaN: those are taken out of x
                // once W has been made of it, and the readouts that they spoil are spoilt by
                // hand.  (5 % of the largest call, as Y waits for it: one warp for both columns
                // 8 %, the compute threads each their row 8 %.)
                const int column = warp - kIssuer - 1;
                const unsigned tile = sX + column * kTileBytes;
                int *const lost = lost_of<N>(raw, phase) + column * Smem::kLostInts;
                const bool any = look_over(tile, valid, lane);
                if (lane == 0) lost[0] = any;
                if (any) {
                    if (alive) alive = mbar_wait(bar_w, phase);
                    take_out(tile, lost, valid, lane);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_v);
                    if (column == 0 && valid == kChunk) {
                        if (alive) alive = mbar_wait(bar_r, phase);
#pragma unroll
                        for (int k = 0; k < kPair; ++k) {
                            const int c = first_column + k;
                            if (k == 0 || paired)
                                tma_store(&map_out, sX + k * kTileBytes, c % m.slabs * kSlab,
                                          c / m.slabs, tok);
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        if (tok + kChunk < to) load_x(tok + kChunk);
                    }
                }
                __syncwarp();
            }
            if (!line && warp == kIssuer + 1 && lane == 0)
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncwarp();
    } else {
        const int which = warp >> 2, quarter = warp & 3;
        const int row = 32 * quarter + lane;
        // The thread's place in the call, worked out again where it is needed rather than held in
        // registers through the loop.
        struct Place {
            int column, h, slab;
            bool keeps;  // whether the thread's results are kept
        };
        auto place = [&]() {
            const int c = opaque(part.cta), per_group = columns_per_group(m);
            const int pairs = (per_group + 1) / 2, of_group = 2 * (c % pairs);
            const bool paired = of_group + 1 < per_group;
            Place at;
            at.column = c / pairs * per_group + of_group + (paired ? which : 0);
            at.h = at.column / m.slabs, at.slab = at.column - at.h * m.slabs;
            at.keeps = which == 0 || paired;
            return at;
        };
        const Place here = place();
        const unsigned lanes = static_cast<unsigned>(quarter) << 21;  // (32 quarter) << 16
        const unsigned myX = sX + which * kTileBytes, myS = sS + which * N * 128;
        const unsigned myW3 = base + (row < 64 ? Smem::kW3First : Smem::kW3) +
                              which * (kTileBytes / 2);
        const unsigned myY = tY + which * kSlab + lanes;
        const unsigned myU = tU + which * kSlab + lanes;
        float *const vecs =
            reinterpret_cast<float *>(raw + (base - smem_u32(raw)) + Smem::kVec) +
            which * 2 * Smem::kVecFloats;
        auto column_sync = [&]() {
            asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "n"(kCompute / kPair) : "memory");
        };
        float *const head = vecs + Smem::kConst;
        if (row == 0) head[2] = __ldg(p.D + here.h * p.D_h);
        // The decays are worked out a chunk ahead.  dt waits as raw bits: a conversion right behind
        // its load would wait for it.
        const unsigned short *const dt_col =
            reinterpret_cast<const unsigned short *>(p.dt) + here.h * p.dt_h;
        unsigned dt_next = 0;
        {
            unsigned dt = 0;
            if (from + row < to) dt = dt_col[(from + row) * p.dt_b];
            if (from + kChunk + row < to) dt_next = dt_col[(from + kChunk + row) * p.dt_b];
            const float bias = __ldg(p.dt_bias + here.h * p.bias_h);
            const float A2 = __ldg(p.A + here.h * p.A_h) * kLog2e;
            if (row == 0) head[0] = bias, head[1] = A2;
            chunk_decays(vecs, from + row < to, __uint_as_float(dt << 16), bias, A2, row, lane);
        }

        // The state a stretch starts from: the thread holds S[0 ..][row].
        float S[kSlab];
        const bool own = row < N;
        auto state_at = [&](const Place &at, int i) {
            return static_cast<ST *>(p.state) + slot * p.st_pool + at.h * p.st_head +
                   static_cast<long long>(at.slab * kSlab + i) * p.st_row + row;
        };
#pragma unroll
        for (int i = 0; i < kSlab; ++i) S[i] = 0.0f;
        // A prompt's state before a stretch: its slot's (or zeros) before the first, which a first
        // pass also puts by where the last stretch would have its result, as the last one of the
        // second pass overwrites the slot while the first may not have begun; what the first pass
        // leaves of the stretches before any other.
        auto kept = [&](long long k) {
            return m.local + (k * columns + here.column) * (kSlab * N) + row;
        };
        const int index = part.index, count = part.count;
        const long long g0 = g - index;  // the prompt's first stretch
        if (!kFirst && count > 1 && m.after_first) pdl_wait();
        if (line && part.c0 > 0) {
            if (alive) alive = handed_on(m.turn + part.turn, lane);
            if (own) {
                const float *const hand =
                    m.hand + ((part.turn - 1ll) * kPair + which) * (kSlab * N) + row;
#pragma unroll
                for (int i = 0; i < kSlab; ++i) S[i] = __ldcg(hand + i * N);
            }
        } else if (own && index == 0) {
            if (!kFirst && count > 1) {
#pragma unroll
                for (int i = 0; i < kSlab; ++i) S[i] = __ldcg(kept(g0 + count - 1) + i * N);
            } else if (!(m.q.fresh && m.q.fresh[b] != 0)) {
#pragma unroll
                for (int i = 0; i < kSlab; ++i) S[i] = static_cast<float>(*state_at(here, i));
            }
            if (kFirst && here.keeps) {
#pragma unroll
                for (int i = 0; i < kSlab; ++i) __stcg(kept(g0 + count - 1) + i * N, S[i]);
            }
        }
        if (!kFirst && own && part.c0 == 0) {
            for (long long k = g0; k < g; ++k) {
                const float f = k == g0 ? 0.0f : exp2f(__ldcg(m.decay + k * columns + here.column));
#pragma unroll
                for (int i = 0; i < kSlab; ++i)
                    S[i] = k == g0 ? __ldcg(kept(k) + i * N)
                                   : fmaf(S[i], f, __ldcg(kept(k) + i * N));
            }
        }
        auto publish = [&]() {  // the state as the next chunk's bf16 operand
            if (own) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    store_smem16(swizzled(myS, row, c),
                                 make_uint4(f2_to_bf2(S[8 * c], S[8 * c + 1]),
                                            f2_to_bf2(S[8 * c + 2], S[8 * c + 3]),
                                            f2_to_bf2(S[8 * c + 4], S[8 * c + 5]),
                                            f2_to_bf2(S[8 * c + 6], S[8 * c + 7])));
            }
            fence_async_smem();
        };
        if (!kFirst) {
            publish();
            warp_arrive(bar_done, lane);
        }
        column_sync();  // the decays

        float stretch_decay = 0.0f;  // log2
        unsigned phase = 0;
        for (int tok = from; tok < to; tok += kChunk, phase ^= 1) {
            const int valid = to - tok < kChunk ? to - tok : kChunk;
            float *const v0 = vecs + phase * Smem::kVecFloats;
            const float2 *const pre = reinterpret_cast<const float2 *>(v0 + kChunk);
            if (valid < kChunk) {  // tokens of the next prompt: X and B must not bring them in
                if (alive) alive = mbar_wait(bar_x, phase);
                if (alive) alive = mbar_wait(bar_b, phase);
                if (row >= valid) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        store_smem16(swizzled(myX, row, c), make_uint4(0, 0, 0, 0));
                        if (which == 0)
#pragma unroll
                            for (int k = 0; k < kBlocks; ++k)
                                store_smem16(swizzled(sB + phase * kBBytes + k * kTileBytes, row,
                                                      c),
                                             make_uint4(0, 0, 0, 0));
                    }
                }
                fence_async_smem();
            }
            if (!kFirst) {
                const float up = pre[row].x;
                const float4 t = *reinterpret_cast<const float4 *>(v0 + 3 * kChunk);
                const float D = head[2];
                // M = G times decays, two blocks of 32 columns per warpgroup
                if (alive) alive = mbar_wait(bar_g, phase);
                __syncwarp();
                tc_fence_after();
                // (rolled loops: unrolled, with the cases of every block side by side, the code is
                // larger than the instruction cache and M took twice as long)
                const unsigned myM = tM + which * 64 + lanes;
#pragma unroll 1
                for (int col = 0; col < 32 * quarter; col += 32) {  // before the row's 32 tokens
                    unsigned gg[2][16], mm[2][8];
                    tc_load16(tG + lanes + col, gg[0]);
                    tc_load16(tG + lanes + col + 16, gg[1]);
                    // the blocks between the columns' and the row's
                    const float f = exp2f(up + ((col < 32 && quarter > 1 ? t.y : 0.0f) +
                                                (col < 64 && quarter > 2 ? t.z : 0.0f)));
                    const float4 *vv = reinterpret_cast<const float4 *>(v0 + col);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 q = vv[4 * k + j];
                            const float2 lo = __fmul2_rn(
                                make_float2(__uint_as_float(gg[k][4 * j]),
                                            __uint_as_float(gg[k][4 * j + 1])),
                                __fmul2_rn(make_float2(f, f), make_float2(q.x, q.y)));
                            const float2 hi = __fmul2_rn(
                                make_float2(__uint_as_float(gg[k][4 * j + 2]),
                                            __uint_as_float(gg[k][4 * j + 3])),
                                __fmul2_rn(make_float2(f, f), make_float2(q.z, q.w)));
                            mm[k][2 * j] = f2_to_bf2(lo.x, lo.y);
                            mm[k][2 * j + 1] = f2_to_bf2(hi.x, hi.y);
                        }
                        tc_store8(myM + col / 2 + 8 * k, mm[k]);
                    }
                }
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {  // the row's own 32 tokens
                    const int col = 32 * quarter + 16 * k;
                    unsigned gg[16], mm[8];
                    tc_load16(tG + lanes + col, gg);
                    const float4 *pp = reinterpret_cast<const float4 *>(pre + col);
                    const int edge = lane - 16 * k;  // the last column kept
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 q = pp[j];  // (prefix, dtv) of two columns
                        const float e0 =
                            exp2_ftz(up - q.x) * (q.y * __uint_as_float(gg[2 * j]));
                        const float e1 =
                            exp2_ftz(up - q.z) * (q.w * __uint_as_float(gg[2 * j + 1]));
                        // on the diagonal, D x of the token itself
                        mm[j] = f2_to_bf2(2 * j < edge    ? e0
                                          : 2 * j == edge ? e0 + D
                                                          : 0.0f,
                                          2 * j + 1 < edge    ? e1
                                          : 2 * j + 1 == edge ? e1 + D
                                                              : 0.0f);
                    }
                    tc_store8(myM + col / 2, mm);
                }
#pragma unroll 1
                for (int cb = quarter + 1; cb < 4; ++cb) {
                    const unsigned zero[16] = {};
                    tc_store16(myM + 16 * cb, zero);
                }
                // The state's share of the readout, where Y will add to it
                const float fi = exp2f(up + ((quarter > 0 ? t.x : 0.0f) +
                                             (quarter > 1 ? t.y : 0.0f) +
                                             (quarter > 2 ? t.z : 0.0f)));
                if (alive) alive = mbar_wait(bar_i, phase);
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    unsigned ii[2][16];
                    tc_load16(myY + 32 * half, ii[0]);
                    tc_load16(myY + 32 * half + 16, ii[1]);
                    tc_wait_ld();
#pragma unroll
                    for (int piece = 0; piece < 2; ++piece) {
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 y =
                                __fmul2_rn(make_float2(fi, fi),
                                           make_float2(__uint_as_float(ii[piece][i]),
                                                       __uint_as_float(ii[piece][i + 1])));
                            ii[piece][i] = __float_as_uint(y.x);
                            ii[piece][i + 1] = __float_as_uint(y.y);
                        }
                        tc_store16(myY + 32 * half + 16 * piece, ii[piece]);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                warp_arrive(bar_m, lane);
            }
            {
                // the token's weight in the chunk's last state: from its own 32 tokens' end onwards
                const float4 t = *reinterpret_cast<const float4 *>(v0 + 3 * kChunk);
                const float w = v0[row] * exp2f((quarter < 1 ? t.y : 0.0f) +
                                                (quarter < 2 ? t.z : 0.0f) +
                                                (quarter < 3 ? t.w : 0.0f));
                if (alive) alive = mbar_wait(bar_x, phase);
#pragma unroll 2
                for (int c = 0; c < 8; ++c) {
                    float x[8];
                    widen16(load_smem16(swizzled(myX, row, c)), x);
                    unsigned bits[kParts][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 f =
                            __fmul2_rn(make_float2(w, w), make_float2(x[2 * i], x[2 * i + 1]));
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            bits[k][i] = f2_to_bf2(f.x, f.y);
                            f = __fadd2_rn(
                                f, make_float2(-__uint_as_float(bits[k][i] << 16),
                                               -__uint_as_float(bits[k][i] & 0xffff0000u)));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        store_smem16(
                            swizzled((k == 0 ? sW1 : sW2) + which * kTileBytes, row, c),
                            make_uint4(bits[k][0], bits[k][1], bits[k][2], bits[k][3]));
                    if constexpr (kParts == 3)
                        store_smem16(swizzled(myW3, row & 63, c),
                                     make_uint4(bits[2][0], bits[2][1], bits[2][2], bits[2][3]));
                }
            }
            fence_async_smem();
            warp_arrive(bar_w, lane);
            const float4 t = *reinterpret_cast<const float4 *>(v0 + 3 * kChunk);
            const float chunk_decay = (t.x + t.y) + (t.z + t.w), f = exp2f(chunk_decay);
            if (kFirst) stretch_decay += chunk_decay;
            if (tok + kChunk < to) {  // the next chunk's decays
                const float dt = __uint_as_float(dt_next << 16);
                if (tok + 2 * kChunk + row < to)
                    dt_next = dt_col[(tok + 2 * kChunk + row) * p.dt_b];
                chunk_decays(vecs + (phase ^ 1) * Smem::kVecFloats, tok + kChunk + row < to, dt,
                             head[0], head[1], row, lane);
            }
            column_sync();
            if (!kFirst) {
                if (alive) alive = mbar_wait(bar_y, phase);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    unsigned yy[2][16], o[16];
                    tc_load16(myY + 32 * half, yy[0]);
                    tc_load16(myY + 32 * half + 16, yy[1]);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = f2_to_bf2(__uint_as_float(yy[i / 8][2 * i % 16]),
                                         __uint_as_float(yy[i / 8][2 * i % 16 + 1]));
                    if (valid == kChunk) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            store_smem16(swizzled(myX, row, 4 * half + c),
                                         make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2],
                                                    o[4 * c + 3]));
                    } else if (const Place at = place(); at.keeps && row < valid) {
                        __nv_bfloat16 *const dst = p.out + (tok + row) * p.out_b +
                                                   at.h * p.out_h + at.slab * kSlab + 32 * half;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            reinterpret_cast<uint4 *>(dst)[c] = make_uint4(
                                o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                }
                const int *const lost = lost_of<N>(raw, phase) + which * Smem::kLostInts;
                if (__builtin_expect(lost[0], 0)) {
                    const Place at = place();
#pragma unroll 1
                    for (int i = 0; i < kSlab; ++i) {
                        if (lost[4 + i] > row) continue;
                        if (valid == kChunk)
                            store_smem2(swizzled(myX, row, i / 8) + 2 * (i % 8), 0x7fff);
                        else if (at.keeps && row < valid)
                            p.out[(tok + row) * p.out_b + at.h * p.out_h + at.slab * kSlab + i] =
                                __ushort_as_bfloat16(0x7fff);
                    }
                }
                if (valid == kChunk) {
                    fence_async_smem();
                    warp_arrive(bar_r, lane);
                }
            }
            if (alive) alive = mbar_wait(bar_u, phase);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                unsigned uu[2][16];
                tc_load16(myU + 32 * half, uu[0]);
                tc_load16(myU + 32 * half + 16, uu[1]);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float *const s = S + 32 * half + i;
                    const float2 v =
                        __ffma2_rn(make_float2(s[0], s[1]), make_float2(f, f),
                                   make_float2(__uint_as_float(uu[i / 16][i % 16]),
                                               __uint_as_float(uu[i / 16][i % 16 + 1])));
                    s[0] = v.x;
                    s[1] = v.y;
                }
            }
            tc_fence_before();
            if (!kFirst) {
                publish();
                warp_arrive(bar_done, lane);
            }
        }

        const Place at = place();
        if (own && at.keeps) {
            if (kFirst) {
                float *loc = m.local + (g * columns + at.column) * (kSlab * N) + row;
#pragma unroll
                for (int i = 0; i < kSlab; ++i) __stcg(loc + i * N, S[i]);
                if (row == 0) __stcg(m.decay + g * columns + at.column, stretch_decay);
            } else if (last) {
                slot = load_slot<kIdx64>(p, part.b);
#pragma unroll
                for (int i = 0; i < kSlab; ++i) {
                    if constexpr (sizeof(ST) == 4)
                        *state_at(at, i) = S[i];
                    else
                        *state_at(at, i) = __float2bfloat16(S[i]);
                }
            }
        }
        if (line && part.c1 >= 0) {
            if (own) {
                float *const hand =
                    m.hand + (part.turn * 1ll * kPair + which) * (kSlab * N) + row;
#pragma unroll
                for (int i = 0; i < kSlab; ++i) __stcg(hand + i * N, S[i]);
            }
            asm volatile("bar.sync %0, %1;" ::"n"(1 + kPair), "n"(kCompute) : "memory");
            if (tid == 0)
                asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(m.turn + 1 + part.turn),
                             "r"(1u)
                             : "memory");
        }
    }
    return alive;
}

template <int N, typename ST, bool kIdx64, Pass kPass>
__global__ void __launch_bounds__(kPromptThreads, 1)
    ssu_prompt_mma_kernel(const __grid_constant__ PromptMmaParams m,
                          const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ CUtensorMap map_b,
                          const __grid_constant__ CUtensorMap map_c,
                          const __grid_constant__ CUtensorMap map_out) {
    constexpr bool kFirst = kPass == Pass::kFirst;
    extern __shared__ unsigned char raw[];
    __shared__ long long scan[kPromptThreads / 32 + 3];
    __shared__ Part part, next;
    __shared__ unsigned tmem_slot;
    // A second pass behind a first is let in when the first has begun, so what came before the
    // first is complete; it waits for the first before it reads its results, and before it ends.
    if (kFirst || !m.after_first) pdl_wait();
    if (kFirst) pdl_trigger();
    const int tid = threadIdx.x;
    const int ctas = ctas_per_stretch(m);
    if constexpr (kPass == Pass::kLine) {
        find_line<kIdx64>(m, ctas, part, scan);
    } else {
        const long long nth = blockIdx.x / ctas;
        const Stretch my =
            find_stretch<kIdx64, kFirst>(m, nth, !kFirst && blockIdx.x == 0, scan);
        if (tid == 0) {
            part.b = my.b, part.g = my.g, part.index = my.index, part.count = my.count;
            part.cta = static_cast<int>(blockIdx.x - nth * ctas);
            part.c0 = 0, part.c1 = -1;
            part.more = my.b >= 0;
        }
    }
    __syncthreads();
    if (!part.more) {
        if (!kFirst && m.after_first) pdl_wait();
        return;
    }
    const unsigned bars = tiles_at(raw) + PromptSmem<N>::kBars;
    if (tid == 0) init_barriers(bars);
    if (tid / 32 == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    bool alive;
    while (true) {
        alive = run_part<N, ST, kIdx64, kPass>(m, map_x, map_b, map_c, map_out, part, next, raw,
                                               tmem_slot);
        tc_fence_before();
        if (__syncthreads_or(!alive) || kPass != Pass::kLine) break;
        if (tid == 0) {  // fresh barriers for the part before
            for (int i = 0; i < kBars; ++i)
                asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bars + 8 * i)
                             : "memory");
            init_barriers(bars);
            part = next;
        }
        __syncthreads();
        tc_fence_after();
        if (!part.more) break;
    }
    if (kPass == Pass::kLine && tid == 32 * (kIssuer + 1))
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!alive) {  // what is in flight lands long before this is over
        atomicOr(&m.q.p.err[2], 1u);
        __nanosleep(1000000);
    }
    if (!kFirst && m.after_first) pdl_wait();
    __syncthreads();
    if (tid / 32 == kIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot),
                     "r"(512)
                     : "memory");
    }
}

}  // namespace
