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
// Y = M X [Q x P] with M = G times the masked decays, and U = B^T W [N x P] with W the weighted
// tokens.  One CTA takes one head's stretch of a prompt, chunk after chunk, its state in
// registers (thread n holds column n of the P = 64 rows).  G, I, U and Y accumulate in TMEM
// (256 of the SM's 512 columns, so two CTAs share an SM and one's products run under the
// other's elementwise work); M goes back into TMEM as an A operand.
//
// Precision.  C, B and X are bf16 and exact.  M and the state that enters I are rounded to bf16
// (2^-9 of a term in the mean square, as much as the bf16 readout itself carries).  W decides
// the state that is carried on, so it enters as the sum of three bf16 parts (24 bits: all of an
// fp32 value; two parts measured 1.1e-6 of the state in the 2-norm, against 1e-7) where the state
// is kept in fp32, of two where it is rounded to bf16 in the end, and runs in fp32 either way.
// Exponents are sums over short runs that never cross a chunk: within blocks of 32 tokens
// prefix and suffix sums, between blocks the block totals, so no exponent is a difference of
// two large sums except inside the diagonal block, whose weights are rounded to bf16 anyway.
// An a_t beyond +-256 (log2) is cut there: exp is then 0 (or infinite) all the same, and a cut
// sum stays small enough to be exact.
//
// Stretches.  A prompt that is long for the device is cut into stretches of `seg` chunks.  A
// first pass (kFirst) runs U alone over every stretch but a prompt's last, from a zero state;
// the second pass starts a stretch from the prompt's own state advanced through the earlier
// stretches' results.
//
// What bounds it: ~1,800 cycles of tensor pipe per chunk and head (G 512, I, Y 256 each, U 768
// with its three parts) against 96 KB that a CTA brings in through L2.

#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssu_prompt.cuh"

namespace {

constexpr int kChunk = 128;      // tokens per chunk: the MMA's M
constexpr int kSlab = 64;        // state rows per CTA: the MMA's N
constexpr int kPromptThreads = 256 + 32;  // two warpgroups for the elementwise work, one warp to issue
constexpr int kHalf = kSlab / 2;  // a thread's share of its row: the two warpgroups halve it
constexpr int kTileBytes = kChunk * 128;  // a 64-column bf16 tile of 128 rows
constexpr float kLog2e = 1.4426950408889634f;

struct PromptMmaParams {
    PromptParams q;
    int seg;              // chunks per stretch
    int slabs;            // headdim / 64
    int out32;            // out's rows are 32-byte aligned
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

__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Waits for the barrier's phase of `parity`; gives up (false) after a bounded number of polls.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity) {
    for (int i = 0; i < (1 << 18); ++i) {
        unsigned done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}

__device__ __forceinline__ void tma_load(unsigned dst, const CUtensorMap *map, unsigned bar, int x,
                                         int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
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

// 32 columns of the thread's TMEM lane.
__device__ __forceinline__ void tc_load32(unsigned addr, unsigned (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
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

__device__ __forceinline__ void tc_store32(unsigned addr, const unsigned (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
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

// 32 bytes, one whole sector, by one thread.
__device__ __forceinline__ void store_sector(void *dst, unsigned a, unsigned b, unsigned c,
                                             unsigned d, unsigned e, unsigned f, unsigned g,
                                             unsigned h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a),
                 "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

// 2^x by the hardware's approximation (2 ulp), results below 2^-126 as 0: for weights that are
// rounded to bf16 next.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- the kernel ------------------------------------------------------------------------

// Shared memory: tiles first (1024-byte aligned), then the per-token values.  W's three parts take
// the places of C and S once G and I are done.
template <int N>
struct PromptSmem {
    static constexpr int kBlocks = N / 64;  // 64-column tiles of B and C
    static constexpr int kC = 0;            // also W's first two parts
    static constexpr int kB = 2 * kTileBytes;
    static constexpr int kX = kB + kBlocks * kTileBytes;
    static constexpr int kS = kX + kTileBytes;  // state, bf16 [n][64 p]; also W's third part
    static constexpr int kVec = kS + kTileBytes;
    // floats of a chunk's tokens: v0 (128), pairs (prefix, dtv) (256), block totals (4); two of
    // them, for this chunk and the next
    static constexpr int kVecFloats = 3 * kChunk + 4;
    static constexpr int kBars = kVec + 2 * kVecFloats * 4;
    static constexpr int kTotal = kBars + 64;
};

// The stretch `g` of the call: its prompt and first chunk.  All threads get the answer; false
// past the last stretch.  With `all`, every prompt is looked at and the bad ones counted.
template <bool kIdx64>
__device__ __forceinline__ bool find_stretch(const PromptMmaParams &m, long long g, bool all,
                                             long long *scan, long long &b, long long &index) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long before = 0;
    constexpr int kWarps = kPromptThreads / 32;
    if (tid == 0) scan[kWarps] = -1;
    for (long long b0 = 0; b0 < m.q.p.batch; b0 += kPromptThreads) {
        const long long bb = b0 + tid;
        long long n = 0;
        if (bb < m.q.p.batch) {
            long long slot, lo, hi;
            if (load_prompt<kIdx64>(m.q, bb, all, slot, lo, hi)) {
                const long long per = static_cast<long long>(m.seg) * kChunk;
                n = (hi - lo + per - 1) / per;
                if (n == 0 && m.q.fresh && m.q.fresh[bb]) n = 1;  // only clears the slot
            }
        }
        long long incl = n;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long base = before;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += scan[w];
            before += scan[w];
        }
        incl += base;
        if (g >= incl - n && g < incl) {
            scan[kWarps] = bb;
            scan[kWarps + 1] = g - (incl - n);
        }
        if (!all && g < before) break;
    }
    __syncthreads();
    b = scan[kWarps];
    index = scan[kWarps + 1];
    return b >= 0;
}

// Decay sums of one chunk, by the four warps of one warpgroup (one token per thread, `row`): the
// token's weight up to the end of its 32 tokens, its prefix within them, dtv, the blocks' totals.
__device__ __forceinline__ void chunk_decays(float *vec, bool live, float dt, float bias, float A2,
                                             int row, int lane) {
    float dtv = 0.0f, a = 0.0f;
    if (live) {
        dtv = softplus_f32(dt + bias);
        a = fminf(fmaxf(dtv * A2, -256.0f), 256.0f);
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

// Roles.  Warp 8 issues: one of its threads starts the copies and the products, as their inputs
// become ready.  Warps 0 .. 7 do the elementwise work; a thread's row (token of the chunk, TMEM
// lane, column n of the state) is the same in both warpgroups, which halve each row's columns.
// Per chunk, with the barrier that each hand-over uses:
//
//   issue:    [full, done] G, I -> [w] U -> next B, C -> [m] Y -> next X
//   compute:  [x] W's parts in registers -> [g] W into C and S -> w; I scaled, D x added; M -> m;
//             the next chunk's decays; [u] S advanced and published; [y] readout out -> done
//
// so U runs under M, and the copies under everything that does not need them.
template <int N, typename ST, bool kIdx64, bool kFirst>
__global__ void __launch_bounds__(kPromptThreads, 2)
    ssu_prompt_mma_kernel(const __grid_constant__ PromptMmaParams m,
                          const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ CUtensorMap map_b,
                          const __grid_constant__ CUtensorMap map_c) {
    using Smem = PromptSmem<N>;
    constexpr int kBlocks = Smem::kBlocks;
    constexpr int kParts = sizeof(ST) == 4 ? 3 : 2;  // bf16 parts of W
    constexpr int kCompute = 256;
    extern __shared__ unsigned char raw[];
    __shared__ long long scan[kPromptThreads / 32 + 2];
    __shared__ unsigned tmem_slot;
    pdl_wait();
    const SsuParams &p = m.q.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int columns = p.nheads * m.slabs;  // CTAs per stretch: heads and slabs
    const long long g = blockIdx.x / columns;
    const int column = static_cast<int>(blockIdx.x - g * columns);
    const int h = column / m.slabs, slab = column - h * m.slabs;
    long long b, index;
    if (!find_stretch<kIdx64>(m, g, !kFirst && blockIdx.x == 0, scan, b, index)) return;
    long long slot, begin, end;
    load_prompt<kIdx64>(m.q, b, false, slot, begin, end);
    const long long from = begin + index * m.seg * kChunk;
    long long to = from + static_cast<long long>(m.seg) * kChunk;
    const bool last = to >= end;
    if (last) to = end;
    if (kFirst && last) return;  // nothing continues after a prompt's last stretch

    const unsigned base = (smem_u32(raw) + 1023u) & ~1023u;
    const unsigned sC = base + Smem::kC, sB = base + Smem::kB, sX = base + Smem::kX;
    const unsigned sS = base + Smem::kS;
    float *const vecs = reinterpret_cast<float *>(raw + (base - smem_u32(raw)) + Smem::kVec);
    const unsigned bar_full = base + Smem::kBars, bar_x = bar_full + 8, bar_g = bar_full + 16,
                   bar_u = bar_full + 24, bar_y = bar_full + 32, bar_w = bar_full + 40,
                   bar_m = bar_full + 48, bar_done = bar_full + 56;

    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(bar_full + 8 * i, 1);
        for (int i = 5; i < 8; ++i) mbar_init(bar_full + 8 * i, kCompute);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(256)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = tmem_slot;
    // columns: G 0..127, U 128..191, I and then Y 192..255.  M takes G's place piece by piece: its
    // tokens 0..63 (bf16 pairs) columns 0..31, 64..127 columns 64..95, each written by the
    // warpgroup that has read the columns of G there.
    const unsigned tG = tmem, tU = tmem + 128, tY = tmem + 192;
    bool alive = true;

    if (warp == 8) {
        if (lane == 0) {
            const int grp = group_of(h, p.group_magic);
            auto load_bc = [&](long long tok) {
                const int t = static_cast<int>(tok);
                mbar_expect(bar_full, kTileBytes * kBlocks * (kFirst ? 1 : 2));
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    tma_load(sB + k * kTileBytes, &map_b, bar_full, k * 64, grp, t);
                    if (!kFirst) tma_load(sC + k * kTileBytes, &map_c, bar_full, k * 64, grp, t);
                }
            };
            auto load_x = [&](long long tok) {
                mbar_expect(bar_x, kTileBytes);
                tma_load(sX, &map_x, bar_x, slab * kSlab, h, static_cast<int>(tok));
            };
            if (from < to) {
                load_bc(from);
                load_x(from);
            }
            unsigned phase = 0;
            for (long long tok = from; tok < to; tok += kChunk, phase ^= 1) {
                const bool more = tok + kChunk < to;
                if (!kFirst) {
                    if (alive) alive = mbar_wait(bar_full, phase);
                    if (alive) alive = mbar_wait(bar_done, phase);  // S and TMEM: see below
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < N / 16; ++k) {
                        const unsigned off = (k / 4) * kTileBytes + (k % 4) * 32;
                        mma_ss(tG, operand(sC + off, 0), operand(sB + off, 0),
                               instruction(kChunk, false, false), k > 0);
                    }
#pragma unroll
                    for (int k = 0; k < N / 16; ++k) {
                        const unsigned off = (k / 4) * kTileBytes + (k % 4) * 32;
                        mma_ss(tY, operand(sC + off, 0), operand(sS + k * 2048, 0),
                               instruction(kSlab, false, true), k > 0);
                    }
                    tc_commit(bar_g);
                }
                if (alive) alive = mbar_wait(bar_w, phase);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kParts * kChunk / 16; ++k) {
                    const int which = k / (kChunk / 16), kk = k % (kChunk / 16);
                    mma_ss(tU, operand(sB + kk * 2048, N == 128 ? kTileBytes : 0),
                           operand((which < 2 ? sC + which * kTileBytes : sS) + kk * 2048, 0),
                           instruction(kSlab, true, true), k > 0);
                }
                tc_commit(bar_u);
                if (kFirst) {  // U alone reads the tiles (x went through registers)
                    if (more) load_x(tok + kChunk);
                    if (alive) alive = mbar_wait(bar_u, phase);
                    if (more) load_bc(tok + kChunk);
                    continue;
                }
                if (alive) alive = mbar_wait(bar_m, phase);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kChunk / 16; ++k)
                    mma_ts(tY, tG + (k < 4 ? 8 * k : 32 + 8 * k), operand(sX + k * 2048, 0),
                           instruction(kSlab, false, true), true);
                tc_commit(bar_y);
                if (alive) alive = mbar_wait(bar_u, phase);
                if (more) load_bc(tok + kChunk);
                if (alive) alive = mbar_wait(bar_y, phase);
                if (more) load_x(tok + kChunk);
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, part = warp >> 2, row = 32 * quarter + lane;
        const unsigned lanes = static_cast<unsigned>(quarter) << 21;  // (32 quarter) << 16
        const bool fresh = m.q.fresh && m.q.fresh[b] != 0;
        const float bias = __ldg(p.dt_bias + h * p.bias_h);
        const float A2 = __ldg(p.A + h * p.A_h) * kLog2e;
        const float D = __ldg(p.D + h * p.D_h);
        const __nv_bfloat16 *const dt_col = p.dt + h * p.dt_h;
        // The second warpgroup has less of M and works the decays out, a chunk ahead.
        float dt_next = 0.0f;
        if (part == 1) {
            float dt = 0.0f;
            if (from + row < to) dt = __bfloat162float(dt_col[(from + row) * p.dt_b]);
            if (from + kChunk + row < to)
                dt_next = __bfloat162float(dt_col[(from + kChunk + row) * p.dt_b]);
            chunk_decays(vecs, from + row < to, dt, bias, A2, row, lane);
        }

        // The state a stretch starts from: the thread holds S[32 part .. 32 part + 31][row].
        float S[kHalf];
        const bool own = row < N;
        ST *const state = static_cast<ST *>(p.state) + slot * p.st_pool + h * p.st_head +
                          static_cast<long long>(slab * kSlab + kHalf * part) * p.st_row + row;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) S[i] = 0.0f;
        if (!kFirst && own) {
            if (!fresh) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) S[i] = static_cast<float>(state[i * p.st_row]);
            }
            for (long long k = g - index; k < g; ++k) {
                const float *loc =
                    m.local + ((k * columns + column) * kSlab + kHalf * part) * N + row;
                const float f = exp2f(__ldcg(m.decay + k * columns + column));
#pragma unroll
                for (int i = 0; i < kHalf; ++i) S[i] = fmaf(S[i], f, __ldcg(loc + i * N));
            }
        }
        // The state as the next chunk's bf16 operand; then the issuing warp may use it and TMEM.
        auto publish = [&]() {
            if (own) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    store_smem16(swizzled(sS, row, 4 * part + c),
                                 make_uint4(f2_to_bf2(S[8 * c], S[8 * c + 1]),
                                            f2_to_bf2(S[8 * c + 2], S[8 * c + 3]),
                                            f2_to_bf2(S[8 * c + 4], S[8 * c + 5]),
                                            f2_to_bf2(S[8 * c + 6], S[8 * c + 7])));
            }
            fence_async_smem();
        };
        if (!kFirst) {
            publish();
            mbar_arrive(bar_done);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");  // the decays

        float stretch_decay = 0.0f;  // log2
        unsigned phase = 0;
        for (long long tok = from; tok < to; tok += kChunk, phase ^= 1) {
            const int valid = static_cast<int>(to - tok < kChunk ? to - tok : kChunk);
            float *const v0 = vecs + phase * Smem::kVecFloats;
            const float2 *const pre = reinterpret_cast<const float2 *>(v0 + kChunk);
            const float4 t4 = *reinterpret_cast<const float4 *>(v0 + 3 * kChunk);
            const float t[4] = {t4.x, t4.y, t4.z, t4.w};
            float later = 0.0f, earlier = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k > quarter) later += t[k];
                if (k < quarter) earlier += t[k];
            }
            const float up = pre[row].x;
            const float w = v0[row] * exp2f(later);  // the token's weight in the chunk's last state
            const float chunk_decay = (t[0] + t[1]) + (t[2] + t[3]);
            stretch_decay += chunk_decay;
            if (alive) alive = mbar_wait(bar_x, phase);
            uint4 xr[4];  // the thread's half of its token's x; zeros past the prompt's end
#pragma unroll
            for (int c = 0; c < 4; ++c)
                xr[c] = row < valid ? load_smem16(swizzled(sX, row, 4 * part + c))
                                    : make_uint4(0, 0, 0, 0);
            // C and S are W's to take once G and I are done
            if (alive) alive = mbar_wait(kFirst ? bar_full : bar_g, phase);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x[8];
                widen16(xr[c], x);
                unsigned bits[kParts][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 f = __fmul2_rn(make_float2(w, w), make_float2(x[2 * i], x[2 * i + 1]));
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        bits[k][i] = f2_to_bf2(f.x, f.y);
                        f = __fadd2_rn(f, make_float2(-__uint_as_float(bits[k][i] << 16),
                                                      -__uint_as_float(bits[k][i] & 0xffff0000u)));
                    }
                }
#pragma unroll
                for (int k = 0; k < kParts; ++k)
                    store_smem16(swizzled(k < 2 ? sC + k * kTileBytes : sS, row, 4 * part + c),
                                 make_uint4(bits[k][0], bits[k][1], bits[k][2], bits[k][3]));
            }
            if (row >= valid) {  // tokens of the next prompt: X and B must not bring them in
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    store_smem16(swizzled(sX, row, 4 * part + c), make_uint4(0, 0, 0, 0));
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k)
                        store_smem16(swizzled(sB + k * kTileBytes, row, 4 * part + c),
                                     make_uint4(0, 0, 0, 0));
                }
            }
            fence_async_smem();
            mbar_arrive(bar_w);
            if (!kFirst) {
                // The state's share of the readout and D x, where Y will add to them
                const float fi = exp2f(up + earlier);
                unsigned ii[32];
                tc_load32(tY + lanes + kHalf * part, ii);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[8];
                    widen16(xr[c], x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 y = __ffma2_rn(
                            make_float2(fi, fi),
                            make_float2(__uint_as_float(ii[8 * c + 2 * i]),
                                        __uint_as_float(ii[8 * c + 2 * i + 1])),
                            __fmul2_rn(make_float2(D, D), make_float2(x[2 * i], x[2 * i + 1])));
                        ii[8 * c + 2 * i] = __float_as_uint(y.x);
                        ii[8 * c + 2 * i + 1] = __float_as_uint(y.y);
                    }
                }
                tc_store32(tY + lanes + kHalf * part, ii);
                // M = G times decays, two blocks of 32 columns per warpgroup
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int cb = 2 * part + half;
                    unsigned mm[16];
                    if (cb <= quarter) {
                        unsigned gg[32];
                        tc_load32(tG + lanes + 32 * cb, gg);
                        tc_wait_ld();
                        if (cb < quarter) {
                            float between = 0.0f;
#pragma unroll
                            for (int k = 1; k < 4; ++k)
                                if (k > cb && k < quarter) between += t[k];
                            const float f = exp2f(up + between);
                            const float4 *vv = reinterpret_cast<const float4 *>(v0 + 32 * cb);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 q = vv[j];
                                const float2 lo = __fmul2_rn(
                                    make_float2(__uint_as_float(gg[4 * j]),
                                                __uint_as_float(gg[4 * j + 1])),
                                    __fmul2_rn(make_float2(f, f), make_float2(q.x, q.y)));
                                const float2 hi = __fmul2_rn(
                                    make_float2(__uint_as_float(gg[4 * j + 2]),
                                                __uint_as_float(gg[4 * j + 3])),
                                    __fmul2_rn(make_float2(f, f), make_float2(q.z, q.w)));
                                mm[2 * j] = f2_to_bf2(lo.x, lo.y);
                                mm[2 * j + 1] = f2_to_bf2(hi.x, hi.y);
                            }
                        } else {
                            const float4 *pp = reinterpret_cast<const float4 *>(pre + 32 * cb);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float4 q = pp[j];  // (prefix, dtv) of columns 2j, 2j + 1
                                const float e0 = exp2_ftz(up - q.x) *
                                                 (q.y * __uint_as_float(gg[2 * j]));
                                const float e1 = exp2_ftz(up - q.z) *
                                                 (q.w * __uint_as_float(gg[2 * j + 1]));
                                mm[j] = f2_to_bf2(2 * j <= lane ? e0 : 0.0f,
                                                  2 * j + 1 <= lane ? e1 : 0.0f);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) mm[j] = 0;
                    }
                    tc_store16(tG + lanes + 64 * part + 16 * half, mm);
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(bar_m);
            }
            if (part == 1 && tok + kChunk < to) {  // the next chunk's decays
                const float dt = dt_next;
                if (tok + 2 * kChunk + row < to)
                    dt_next = __bfloat162float(dt_col[(tok + 2 * kChunk + row) * p.dt_b]);
                chunk_decays(vecs + (phase ^ 1) * Smem::kVecFloats, tok + kChunk + row < to, dt,
                             bias, A2, row, lane);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
            const float f = exp2f(chunk_decay);
            if (alive) alive = mbar_wait(bar_u, phase);
            __syncwarp();
            tc_fence_after();
            {
                unsigned uu[32];
                tc_load32(tU + lanes + kHalf * part, uu);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < kHalf; i += 2) {
                    const float2 s = __ffma2_rn(
                        make_float2(S[i], S[i + 1]), make_float2(f, f),
                        make_float2(__uint_as_float(uu[i]), __uint_as_float(uu[i + 1])));
                    S[i] = s.x;
                    S[i + 1] = s.y;
                }
            }
            if (kFirst) continue;
            publish();
            if (alive) alive = mbar_wait(bar_y, phase);
            __syncwarp();
            tc_fence_after();
            unsigned yy[32];
            tc_load32(tY + lanes + kHalf * part, yy);
            tc_wait_ld();
            tc_fence_before();
            mbar_arrive(bar_done);
            if (row < valid) {
                unsigned o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = f2_to_bf2(__uint_as_float(yy[2 * i]), __uint_as_float(yy[2 * i + 1]));
                __nv_bfloat16 *const dst = p.out + (tok + row) * p.out_b + h * p.out_h +
                                           slab * kSlab + kHalf * part;
                if (m.out32) {
                    store_sector(dst, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
                    store_sector(dst + 16, o[8], o[9], o[10], o[11], o[12], o[13], o[14], o[15]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        reinterpret_cast<uint4 *>(dst)[c] =
                            make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            }
        }

        if (own) {
            if (kFirst) {
                float *loc = m.local + ((g * columns + column) * kSlab + kHalf * part) * N + row;
#pragma unroll
                for (int i = 0; i < kHalf; ++i) __stcg(loc + i * N, S[i]);
                if (tid == 0) __stcg(m.decay + g * columns + column, stretch_decay);
            } else if (last) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    if constexpr (sizeof(ST) == 4)
                        state[i * p.st_row] = S[i];
                    else
                        state[i * p.st_row] = __float2bfloat16(S[i]);
                }
            }
        }
    }
    if (!alive) atomicOr(&p.err[2], 1u);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256)
                     : "memory");
    }
}

}  // namespace
