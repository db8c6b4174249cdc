// The gated delta rule over prompts in chunks, on the tcgen05 tensor cores (sm_103a), instantiated by
// ssu_delta.cu beside the token-by-token kernel of ssu_delta.cuh.
//
// Mathematics.  Over a chunk of C = 64 tokens, with s_i the sum of the log decays up to token i, kn
// and qn the keys and queries at length one, and S the state [P, N] that the chunk begins with:
//
//   L_ij = beta_i e^{s_i - s_j} (kn_i . kn_j)  for j < i;      T = (I + L)^-1
//   U    = T R,  R_i = beta_i (v_i - e^{s_i} S kn_i)           (the corrections e_i of all tokens)
//   y_i  = e^{s_i} S qn_i + sum_{j <= i} (kn_j . qn_i) e^{s_i - s_j} U_j
//   S'   = e^{s_C} S + sum_j e^{s_C - s_j} U_j kn_j^T
//
// Three kernels.  A plan (one CTA; none for few prompts) lists the chunks of all prompts.  A first
// pass, parallel over chunks and heads, makes of keys and gates alone what a chunk needs beside its
// state: T, the masked M_ij = (k_j . qn_i) e^{s_i - s_j} and the tokens' factors.  A second pass
// takes a head's state (128 of its rows) through a prompt, chunk after chunk.
//
// The second pass holds everything transposed, with the state's 128 rows p as the MMA's M: then S, R
// and U are first operands, which come from TMEM, where the threads that made them put them, and the
// tiles of K, Q, T and M in shared memory, as they were copied, are the second ones:
//
//   S (K, Q)^T [128 x 128],  R T^T [128 x 64],  U M^T [128 x 64],  U K [128 x N]
//
// Two warpgroups share the rows' elementwise work, a thread holding 4 rows' 16 columns of S.
//
// Precision.  States, statistics and sums are fp32.  K and Q are bf16 and exact (their lengths are
// factors of tokens).  The other operands enter as sums of bf16 parts: for the state S, R and U three
// (24 bits; two for a state kept in bf16) and T two (1 on its diagonal is exact, the other elements are
// to 2^-17); for the readout U and M two each, three of the four products.  Readouts are then as far
// off as fp32 sums rounded once, 0.0017 in the 2-norm (with M in one part 0.0022, and 0.0102 where a
// head's keys are all the same and its corrections cancel).  fp32 states are 2e-7 to 5e-6 off with
// decays of up to thousands of tokens, as the fp32 recurrence's are (3e-7 to 1e-5: its decays'
// roundings add up); where all keys are the same T's second part shows, 2^-16.7 to 2^-14.3 (of 4000
// tokens with gates of 0.5 to 1).  T is worked out by inverting blocks of 16 along the diagonal row by
// row and joining them, T21 = -T22 L21 T11 (powers of L, as a product formula would have, grow like
// binomials where keys are alike).
//
// A chunk with an infinity, a NaN or growing decays (a zero weight times such an element is NaN) is
// taken token by token by the second pass, from the state in registers.
//
// What bounds it (8 prompts of 4096 tokens through 32 heads of 128 x 128: 541 us): the second pass (360
// of them) by the chain of a chunk's steps, 2.8 us or 5,500 cycles at one CTA per SM, of which more
// than half is products (24 MMAs of N = 128, 16 of N = 64 down to 16, 12 of N = 128) and the rest the
// elementwise work between a product's end and the next one's first operand (of R 430 cycles, 340 of
// them arithmetic); the first pass by shared memory and the chain of its own steps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssu_delta.cuh"
#include "ssu_tc.cuh"

namespace {

constexpr int kDeltaChunk = 64;  // tokens per chunk
constexpr int kDeltaRows = 128;  // state rows per CTA: the MMA's M
constexpr int kDeltaTile = kDeltaChunk * 128;  // 64 rows of 64 bf16

// What the first pass leaves of a chunk for one head: T's and M's two parts as the tiles of an operand,
// and the tokens' factors.  All four are lower triangles, in blocks of 16 x 16, of which products take
// no block above the diagonal (a step of 16 columns k has the rows from 16 k on).  So M's second part
// lies where the others have those blocks: its columns k = 1 .. 3 in M's tile, from row 0 on at the
// columns 4 - k, its first ones, rows 0 .. 47, in T's first part at the columns 3, the rest at 1.
struct DeltaRecord {
    enum : int {
        kT1 = 0,
        kT2 = kDeltaTile,
        kM = 2 * kDeltaTile,
        kVec = 3 * kDeltaTile,
        kBytes = kVec + 2048
    };
    enum : int {  // floats of kVec, 64 each
        kBeta = 0,     // beta
        kPast = 64,    // beta e^{s} / |k|: of S k in R
        kLeft = 128,   // e^{s_C - s} / |k|: of U in the next state
        kRead = 192,   // scale / |q|: of U M^T
        kReadS = 256,  // e^{s}: of S q
        kDecay = 320,  // the token's own decay
        kKey = 384,    // 1 / |k|
        kWhole = 448,  // e^{s_C}; then whether the chunk is to be taken token by token
        kSlow = 449
    };
};

// What the plan says of a prompt.
struct __align__(32) DeltaPrompt {
    int begin, end;  // tokens
    int first;       // chunk
    int starts;      // kNot: a bad prompt; else whether from zeros or from its slot
    long long slot;
    enum : int { kNot = 0, kSlot = 1, kZeros = 2 };
};

struct DeltaMmaParams {
    DeltaParams d;
    int idx64;              // the index type is int64
    int few;                // at most 32 prompts: without a plan
    int slabs;              // of 128 rows
    int per_cta;            // heads per CTA of the first pass
    int *total;             // chunks of the call
    DeltaPrompt *prompts;   // the longest first
    int2 *chunks;           // first token, tokens
    unsigned char *records;  // [chunk][head]
};

// ---- pieces of both passes ----------------------------------------------------------------

// TMEM in the fragments of an 8 x 8 matrix: of 16 lanes and 8 columns a thread holds columns 2 t and
// 2 t + 1 (t = lane % 4) of lanes g and g + 8 (g = lane / 4), and of packed pairs column t of 4.
// So V comes by ldmatrix and the readout goes by stmatrix, both transposed, with a pair of tokens
// per register (an element per load and store kept shared memory busy for 2,000 cycles per chunk).
__device__ __forceinline__ void tc_load_frag(unsigned addr, unsigned (&r)[16]) {  // 32 columns
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tc_load_frag(unsigned addr, unsigned (&r)[8]) {  // 16 columns
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tc_store_frag(unsigned addr, const unsigned (&r)[4]) {  // 8 columns
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void tc_store_frag(unsigned addr, const unsigned (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void load_trans4(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void store_trans4(unsigned addr, const unsigned (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// ---- the plan ----------------------------------------------------------------------------

constexpr int kPlanThreads = 256;
constexpr int kPlanSorted = 1024;  // prompts up to which the longest come first

// A prompt that begins before the end of a good one before it is a bad one too (offsets ran
// backwards): chunks never outnumber tokens / 64 + batch, which the workspace has room for.
template <bool kIdx64>
__global__ void __launch_bounds__(kPlanThreads) ssu_delta_plan_kernel(
    const __grid_constant__ DeltaMmaParams m) {
    pdl_wait();
    pdl_trigger();
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ int warp_end[kWarps], warp_chunks[kWarps], firsts[kPlanThreads];
    __shared__ int2 spans[kPlanThreads];
    __shared__ int lengths[kPlanSorted], chunks_of[kPlanSorted];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const SsuParams &p = m.d.m.p;
    int seen = 0, total = 0;  // the largest end and the chunks of the prompts before
    auto put = [&](long long at, long long b, bool good, int first) {
        DeltaPrompt d{0, 0, first, DeltaPrompt::kNot, 0};
        if (good) {
            long long lo, hi;
            load_prompt<kIdx64>(m.d.m, b, false, d.slot, lo, hi);
            d.begin = static_cast<int>(lo), d.end = static_cast<int>(hi);
            d.starts =
                m.d.m.fresh && m.d.m.fresh[b] != 0 ? DeltaPrompt::kZeros : DeltaPrompt::kSlot;
        }
        m.prompts[at] = d;
    };
    for (long long b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const long long b = b0 + tid;
        long long slot, lo = 0, hi = 0;
        bool good = b < p.batch && load_prompt<kIdx64>(m.d.m, b, true, slot, lo, hi);
        int end = good && lo < hi ? static_cast<int>(hi) : 0, most = end;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, most, x);
            if (lane >= x) most = max(most, o);
        }
        if (lane == 31) warp_end[warp] = most;
        __syncthreads();
        int before = __shfl_up_sync(0xffffffffu, most, 1);
        if (lane == 0) before = 0;
        before = max(before, seen);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before = max(before, warp_end[w]);
            seen = max(seen, warp_end[w]);
        }
        if (end && before > lo) {
            good = false;
            record_skip(p, b);
        }
        const int n = good ? static_cast<int>((hi - lo + kDeltaChunk - 1) / kDeltaChunk) : 0;
        int incl = n;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        if (lane == 31) warp_chunks[warp] = incl;
        __syncthreads();
        int first = total + incl - n;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) first += warp_chunks[w];
            total += warp_chunks[w];
        }
        if (p.batch <= kPlanSorted) {
            if (b < p.batch) lengths[b] = good ? static_cast<int>(hi - lo) : -1, chunks_of[b] = first;
        } else if (b < p.batch) {
            put(b, b, good, first);
        }
        firsts[tid] = first;
        spans[tid] = n ? make_int2(static_cast<int>(lo), static_cast<int>(hi)) : make_int2(0, 0);
        __syncthreads();
        const int these = static_cast<int>(min(p.batch - b0, static_cast<long long>(kPlanThreads)));
        for (int k = warp; k < these; k += kWarps) {
            const int2 span = spans[k];
            for (int i = lane; i < (span.y - span.x + kDeltaChunk - 1) / kDeltaChunk; i += 32) {
                const int at = span.x + i * kDeltaChunk;
                m.chunks[firsts[k] + i] = make_int2(at, min(kDeltaChunk, span.y - at));
            }
        }
        __syncthreads();
    }
    if (tid == 0) *m.total = total;
    if (p.batch > kPlanSorted) return;
    for (long long b = tid; b < p.batch; b += kPlanThreads) {
        const int mine = lengths[b];
        int rank = 0;
        for (int o = 0; o < static_cast<int>(p.batch); ++o)
            rank += lengths[o] > mine || (lengths[o] == mine && o < b);
        put(rank, b, mine >= 0, chunks_of[b]);
    }
}

// Of at most 32 prompts every CTA works out the same for itself, a prompt per lane of one warp (a plan
// in front costs a call 3 us); `chunks` is the number of the lane's prompt's.
__device__ __forceinline__ DeltaPrompt plan_lane(const DeltaMmaParams &m, bool counts, int lane,
                                                 int &chunks) {
    DeltaPrompt d{0, 0, 0, DeltaPrompt::kNot, 0};
    long long lo = 0, hi = 0;
    bool good = false;
    if (lane < m.d.m.p.batch)
        good = m.idx64 ? load_prompt<true>(m.d.m, lane, counts, d.slot, lo, hi)
                       : load_prompt<false>(m.d.m, lane, counts, d.slot, lo, hi);
    const int end = good && lo < hi ? static_cast<int>(hi) : 0;
    int most = end;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, most, x);
        if (lane >= x) most = max(most, o);
    }
    const int before = __shfl_up_sync(0xffffffffu, most, 1);
    if (lane > 0 && end && before > lo) {
        good = false;
        if (counts) record_skip(m.d.m.p, lane);
    }
    chunks = good ? static_cast<int>((hi - lo + kDeltaChunk - 1) / kDeltaChunk) : 0;
    d.first = chunks;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, d.first, x);
        if (lane >= x) d.first += o;
    }
    d.first -= chunks;
    if (good) {
        d.begin = static_cast<int>(lo), d.end = static_cast<int>(hi);
        d.starts =
            m.d.m.fresh && m.d.m.fresh[lane] != 0 ? DeltaPrompt::kZeros : DeltaPrompt::kSlot;
    }
    return d;
}

// The prompt that is the `rank`-th longest (lane 0's answer counts).
__device__ __forceinline__ DeltaPrompt few_ranked(const DeltaMmaParams &m, int rank, int lane) {
    int chunks;
    DeltaPrompt d = plan_lane(m, false, lane, chunks);
    const int mine = d.starts == DeltaPrompt::kNot ? -1 : d.end - d.begin;
    int before = 0;
    for (int o = 0; o < static_cast<int>(m.d.m.p.batch); ++o) {
        const int other = __shfl_sync(0xffffffffu, mine, o);
        before += other > mine || (other == mine && o < lane);
    }
    const unsigned found =
        __ballot_sync(0xffffffffu, lane < m.d.m.p.batch && before == rank);
    const int from = __ffs(found) - 1;
    d.begin = __shfl_sync(0xffffffffu, d.begin, from);
    d.end = __shfl_sync(0xffffffffu, d.end, from);
    d.first = __shfl_sync(0xffffffffu, d.first, from);
    d.starts = __shfl_sync(0xffffffffu, d.starts, from);
    d.slot = __shfl_sync(0xffffffffu, d.slot, from);
    return d;
}

// ---- the first pass ------------------------------------------------------------------------
//
// K K^T and Q K^T are one tcgen05 product of K and Q, 16 rows of each in turn, with themselves: then
// the four warps of a TMEM quarter each have 16 rows of both, and Q's lengths are on the diagonal.
// The blocks of T are joined by mma.sync of operands in two bf16 parts (three products, 2^-17).
//
// What bounds it: shared memory's bandwidth (68 % of it taken in calls of many waves) and the chain of
// its steps with 16 warps to an SM.  (Scalar joins, three shared loads for eight multiplications, took
// 2.1 times the pass's time; K K^T and Q K^T by mma.sync and joins of tf32 parts 1.1.)

constexpr int kPrepThreads = 128;
constexpr int kPrepHeads = 2;   // the most heads per CTA: a warp each makes their factors
constexpr int kPrepPitch = 72;  // floats per row of L and T: pairs of 8 rows on 32 banks
constexpr int kPrepColumns = 128;  // of TMEM

template <int N>
struct PrepSmem {
    static constexpr int kBlock = 128 * 128;  // 64 columns of K's and Q's rows
    static constexpr int kL = 0;              // over K and Q, when their products are done
    static constexpr int kT = kL + kDeltaChunk * kPrepPitch * 4;
    static constexpr int kTilesEnd = N / 64 * kBlock;
    static constexpr int kMatEnd = kT + kDeltaChunk * kPrepPitch * 4;
    static constexpr int kM = kTilesEnd > kMatEnd ? kTilesEnd : kMatEnd;
    static constexpr int kMFirst = kM + kDeltaTile;  // the first 16 columns of M's second part
    static constexpr int kLengths = kMFirst + kDeltaChunk * 32;  // 1 / |k|, scale / |q|
    static constexpr int kSums = kLengths + 2 * kDeltaChunk * 4;  // s in two floats, per head
    static constexpr int kVec = kSums + kPrepHeads * 2 * kDeltaChunk * 4;  // per head
    static constexpr int kBars = kVec + kPrepHeads * 2048;
    static constexpr int kTotal = kBars + 16;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const unsigned (&a)[4],
                                          const unsigned (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// A pair of fp32 values as two bf16 parts.
__device__ __forceinline__ void split_pair(float2 f, unsigned &hi, unsigned &lo) {
    hi = f2_to_bf2(f.x, f.y);
    lo = f2_to_bf2(f.x - __uint_as_float(hi << 16), f.y - __uint_as_float(hi & 0xffff0000u));
}

// d += A B over columns k0 .. k1 - 1 of A and those rows of B, both in rows of kPrepPitch floats: 16
// rows from `a`, kTiles times 8 columns from `b`.
template <int kMost, int kTiles>
__device__ __forceinline__ void block_product(float (&d)[kTiles][4], const float *a,
                                              const float *b, int k0, int k1, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float *const arow = a + g * kPrepPitch + 2 * t, *const brow = b + 2 * t * kPrepPitch + g;
    float small[2][kTiles][4] = {};  // the products side by side: a sum's MMAs are a chain
#pragma unroll
    for (int k = 0; k < kMost; k += 16) {
        if (k < k0 || k >= k1) continue;
        unsigned ah[4], al[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            split_pair(*reinterpret_cast<const float2 *>(arow + x % 2 * 8 * kPrepPitch + k +
                                                         x / 2 * 8),
                       ah[x], al[x]);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            unsigned bh[2], bl[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float *const at = brow + (k + 8 * x) * kPrepPitch + 8 * n;
                split_pair(make_float2(at[0], at[kPrepPitch]), bh[x], bl[x]);
            }
            mma_16816(small[0][n], al, bh);
            mma_16816(small[1][n], ah, bl);
            mma_16816(d[n], ah, bh);
        }
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[n][i] += small[0][n][i] + small[1][n][i];
}

// The product's 16 x 8 kTiles values, times `sign`, to rows of kPrepPitch floats from `to`.
template <int kTiles>
__device__ __forceinline__ void put_product(const float (&d)[kTiles][4], float *to, float sign,
                                            int lane) {
    float *const row = to + (lane >> 2) * kPrepPitch + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
        *reinterpret_cast<float2 *>(row + 8 * n) = make_float2(sign * d[n][0], sign * d[n][1]);
        *reinterpret_cast<float2 *>(row + 8 * kPrepPitch + 8 * n) =
            make_float2(sign * d[n][2], sign * d[n][3]);
    }
}

// Sums of log decays are pairs of floats, the second what rounding the first has lost: differences of
// neighbours stay exact behind long decays.  (In double, which this GPU has few units for, the sums of
// a chunk took 6,000 cycles.)
__device__ __forceinline__ float2 add_pairs(float2 a, float2 b) {
    const float sum = a.x + b.x, of_b = sum - a.x;
    const float lost = (a.x - (sum - of_b)) + (b.x - of_b) + (a.y + b.y);
    const float x = sum + lost;
    return make_float2(x, lost - (x - sum));
}

// One head's rates of the chunk's tokens, two per lane of one warp, before their keys' lengths are
// known; dt and gate as loaded.
struct DeltaRates {
    float beta[2], past[2], left[2];  // beta, e^s, e^{s_C - s}
    bool bad;
};

__device__ __forceinline__ DeltaRates delta_rates(const unsigned (&dt)[2], const unsigned (&gate)[2],
                                                  float bias, float A2, int valid, float *sums,
                                                  float *vec, int lane) {
    using R = DeltaRecord;
    DeltaRates r;
    r.bad = false;
    float a[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        a[k] = r.beta[k] = 0.0f;
        if (2 * lane + k >= valid) continue;
        a[k] = softplus_f32(__uint_as_float(dt[k] << 16) + bias) * A2;
        if (a[k] < -300.0f) a[k] = -300.0f;  // 2^-300 is 0; NaN stays
        r.beta[k] = 1.0f / (1.0f + expf(-__uint_as_float(gate[k] << 16)));
        r.bad |= !(a[k] < 60.0f) || !(r.beta[k] <= 1.0f);
    }
    float2 upto = add_pairs(make_float2(a[0], 0.0f), make_float2(a[1], 0.0f));
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const float2 o = make_float2(__shfl_up_sync(0xffffffffu, upto.x, x),
                                     __shfl_up_sync(0xffffffffu, upto.y, x));
        if (lane >= x) upto = add_pairs(o, upto);
    }
    float2 before = make_float2(__shfl_up_sync(0xffffffffu, upto.x, 1),
                                __shfl_up_sync(0xffffffffu, upto.y, 1));
    if (lane == 0) before = make_float2(0.0f, 0.0f);
    const float2 s[2] = {add_pairs(before, make_float2(a[0], 0.0f)), upto};
    const float2 whole = make_float2(__shfl_sync(0xffffffffu, upto.x, 31),
                                     __shfl_sync(0xffffffffu, upto.y, 31));
    r.bad |= !(s[0].x < 60.0f) || !(s[1].x < 60.0f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = 2 * lane + k;
        sums[i] = s[k].x;
        sums[kDeltaChunk + i] = s[k].y;
        r.past[k] = exp2f(s[k].x);
        r.left[k] = exp2f((whole.x - s[k].x) + (whole.y - s[k].y));
        vec[R::kBeta + i] = r.beta[k];
        vec[R::kReadS + i] = r.past[k];
        vec[R::kDecay + i] = exp2f(a[k]);
    }
    if (lane == 0) vec[R::kWhole] = exp2f(whole.x);
    return r;
}

// Grid: chunks, heads / per_cta (the heads of a CTA are of one key head).
template <int N>
__global__ void __launch_bounds__(kPrepThreads, 4)
    ssu_delta_prep_kernel(const __grid_constant__ DeltaMmaParams m,
                          const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_q) {
    using Smem = PrepSmem<N>;
    using R = DeltaRecord;
    extern __shared__ unsigned char unaligned[];
    __shared__ unsigned tmem_slot;
    __shared__ int2 found;
    const unsigned tiles = (smem_u32(unaligned) + 1023u) & ~1023u;
    unsigned char *const raw = unaligned + (tiles - smem_u32(unaligned));
    const unsigned bar_tiles = tiles + Smem::kBars, bar_product = bar_tiles + 8;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        mbar_init(bar_tiles, 1);
        mbar_init(bar_product, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(kPrepColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    auto free_tmem = [&]() {
        if (warp == 0)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kPrepColumns)
                         : "memory");
    };
    pdl_wait();
    pdl_trigger();
    int2 chunk;  // first token, tokens; of no chunk: no tokens
    if (m.few) {
        if (warp == 0) {
            int chunks;
            const DeltaPrompt d =
                plan_lane(m, blockIdx.x == 0 && blockIdx.y == 0, lane, chunks);
            const int at = static_cast<int>(blockIdx.x) - d.first;
            if (lane == 0) found = make_int2(0, 0);
            __syncwarp();
            if (at >= 0 && at < chunks)
                found = make_int2(d.begin + at * kDeltaChunk,
                                  min(kDeltaChunk, d.end - d.begin - at * kDeltaChunk));
        }
        __syncthreads();
        chunk = found;
    } else {
        chunk = m.chunks[blockIdx.x];  // (past the last one: of no use)
        if (static_cast<int>(blockIdx.x) >= *m.total) chunk.y = 0;
    }
    if (chunk.y == 0) {
        free_tmem();
        return;
    }
    const SsuParams &p = m.d.m.p;
    const int tok = chunk.x, valid = chunk.y;
    const int h0 = blockIdx.y * m.per_cta, grp = group_of(h0, p.group_magic);
    unsigned dead = 0;
    if (tid == 96) {
        mbar_expect(bar_tiles, N / 64 * Smem::kBlock);
#pragma unroll
        for (int k = 0; k < N / 64; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const unsigned to = tiles + k * Smem::kBlock + w * 4096;
                tma_load(to, &map_k, bar_tiles, k * 64, grp, tok + 16 * w);
                tma_load(to + 2048, &map_q, bar_tiles, k * 64, grp, tok + 16 * w);
            }
    }
    // the rates of the warp's own head
    unsigned dt[2] = {}, gate[2] = {};
    float bias = 0.0f, A2 = 0.0f;
    if (warp < m.per_cta) {
        const int h = h0 + warp;
        bias = __ldg(p.dt_bias + h * p.bias_h), A2 = __ldg(p.A + h * p.A_h) * kLog2e;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (2 * lane + k >= valid) continue;
            const long long t = static_cast<long long>(tok) + 2 * lane + k;
            dt[k] = reinterpret_cast<const unsigned short *>(p.dt)[t * p.dt_b + h * p.dt_h];
            gate[k] =
                reinterpret_cast<const unsigned short *>(m.d.beta)[t * m.d.beta_t + h * m.d.beta_h];
        }
    }
    // (under the copies)
    float *const my_vec = reinterpret_cast<float *>(raw + Smem::kVec) + warp * 512;
    DeltaRates rates{};
    if (warp < m.per_cta)
        rates = delta_rates(dt, gate, bias, A2, valid,
                            reinterpret_cast<float *>(raw + Smem::kSums) + warp * 2 * kDeltaChunk,
                            my_vec, lane);
    if (warp == 3) {
        const unsigned leader = elect_one();
        mbar_pass(bar_tiles, 0, dead);
        if (leader)
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
                const unsigned long long at =
                    operand(tiles + (k / 4) * Smem::kBlock + (k % 4) * 32, 0);
                mma_ss(tmem, at, at, instruction(128, false, false), k > 0);
            }
        tc_commit_of(leader, bar_product);
        __syncwarp();
    }
    // The warp's 16 rows are its TMEM quarter's: lanes 0 .. 15 have K's, the others Q's.
    const int block = warp;
    float *const lengths = reinterpret_cast<float *>(raw + Smem::kLengths);
    const int g = lane >> 2, t = lane & 3;
    mbar_pass(bar_product, 0, dead);
    __syncwarp();
    tc_fence_after();
    const unsigned k_rows = tmem + (static_cast<unsigned>(block) << 21);
    const unsigned q_rows = k_rows + (16u << 16);
    unsigned own[8], qq[8];  // the diagonals
    tc_load_frag(k_rows + 32 * block, own);
    tc_load_frag(q_rows + 32 * block + 16, qq);
    tc_wait_ld();
    bool bad = false;
    if (t == g >> 1) {  // the thread with rows g and g + 8 of the diagonals
        const bool unit = m.d.eps >= 0.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = 16 * block + g + 8 * half;
            const float k2 = __uint_as_float(g & 1 ? own[6 * half + 1] : own[6 * half]);
            const float q2 = __uint_as_float(g & 1 ? qq[6 * half + 1] : qq[6 * half]);
            const bool live = row < valid;
            const float rk = !live ? 0.0f : unit ? 1.0f / sqrtf(k2 + m.d.eps) : 1.0f;
            const float rq = !live ? 0.0f : unit ? m.d.scale / sqrtf(q2 + m.d.eps) : m.d.scale;
            lengths[row] = rk;
            lengths[kDeltaChunk + row] = rq;
            bad |= live && (!(k2 < INFINITY) || !(q2 < INFINITY) || !(rk < INFINITY) ||
                            !(fabsf(rq) < INFINITY));
        }
    }
    bad = __syncthreads_or(bad);
    if (__syncthreads_or(dead)) {  // what is in flight lands long before this is over
        if (tid == 0) atomicOr(&p.err[2], 1u);
        __nanosleep(1000000);
        tc_fence_before();
        __syncthreads();
        free_tmem();
        return;
    }
    if (warp < m.per_cta) {
        const bool slow = bad || __any_sync(0xffffffffu, rates.bad);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = 2 * lane + k;
            const float rk = lengths[i];
            my_vec[R::kPast + i] = rates.beta[k] * rates.past[k] * rk;
            my_vec[R::kLeft + i] = rates.left[k] * rk;
            my_vec[R::kRead + i] = lengths[kDeltaChunk + i];
            my_vec[R::kKey + i] = rk;
        }
        if (lane == 0) my_vec[R::kSlow] = slow ? 1.0f : 0.0f;
    }
    float *const L = reinterpret_cast<float *>(raw + Smem::kL);
    float *const T = reinterpret_cast<float *>(raw + Smem::kT);
#pragma unroll 1
    for (int k = 0; k < m.per_cta; ++k) {
        __syncthreads();  // the factors; the head before has left
        const float *const sums = reinterpret_cast<float *>(raw + Smem::kSums) + k * 2 * kDeltaChunk;
        const float *const vec = reinterpret_cast<float *>(raw + Smem::kVec) + k * 512;
        {
            const int i0 = 16 * block + g;
            const float hi[2] = {sums[i0], sums[i0 + 8]};
            const float lo[2] = {sums[kDeltaChunk + i0], sums[kDeltaChunk + i0 + 8]};
            const float f[2] = {vec[R::kBeta + i0] * lengths[i0],
                                vec[R::kBeta + i0 + 8] * lengths[i0 + 8]};
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
                if (nb > block) continue;
                unsigned kk[8], qk[8];
                tc_load_frag(k_rows + 32 * nb, kk);
                tc_load_frag(q_rows + 32 * nb, qk);
                tc_wait_ld();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int n = 2 * nb + x, j = 8 * n + 2 * t;
                    const float2 sh = *reinterpret_cast<const float2 *>(sums + j);
                    const float2 sl = *reinterpret_cast<const float2 *>(sums + kDeltaChunk + j);
                    const float2 rk = *reinterpret_cast<const float2 *>(lengths + j);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int i = i0 + 8 * half, at = 4 * x + 2 * half;
                        const float e0 = exp2_ftz((hi[half] - sh.x) + (lo[half] - sl.x)) * rk.x;
                        const float e1 = exp2_ftz((hi[half] - sh.y) + (lo[half] - sl.y)) * rk.y;
                        // (rows past the prompt's end hold anything)
                        *reinterpret_cast<float2 *>(L + i * kPrepPitch + j) =
                            i < valid ? make_float2(__uint_as_float(kk[at]) * (e0 * f[half]),
                                                    __uint_as_float(kk[at + 1]) * (e1 * f[half]))
                                      : make_float2(0.0f, 0.0f);
                        unsigned one, two;
                        split_pair(make_float2(j <= i ? __uint_as_float(qk[at]) * e0 : 0.0f,
                                               j + 1 <= i ? __uint_as_float(qk[at + 1]) * e1 : 0.0f),
                                   one, two);
                        *reinterpret_cast<unsigned *>(raw + Smem::kM + i * 128 +
                                                      ((n ^ (i & 7)) << 4) + 4 * t) = one;
                        const int to = nb == 0 ? Smem::kMFirst + i * 32 + x * 16
                                               : Smem::kM + (i - 16 * nb) * 128 +
                                                     (((2 * (4 - nb) + x) ^ (i & 7)) << 4);
                        *reinterpret_cast<unsigned *>(raw + to + 4 * t) = two;
                    }
                }
            }
        }
        __syncwarp();
        // the warp's block of 16 on the diagonal: a column of the inverse per lane (L's elements on
        // and above the diagonal are not looked at)
        if (lane < 16) {
            const float *const rows = L + 16 * block * (kPrepPitch + 1);
            float x[16];
            x[0] = lane == 0 ? 1.0f : 0.0f;
#pragma unroll
            for (int i = 1; i < 16; ++i) {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(rows + i * kPrepPitch + j);
                    sum = fmaf(l.x, x[j], sum);
                    if (j + 1 < i) sum = fmaf(l.y, x[j + 1], sum);
                    if (j + 2 < i) sum = fmaf(l.z, x[j + 2], sum);
                    if (j + 3 < i) sum = fmaf(l.w, x[j + 3], sum);
                }
                x[i] = i == lane ? 1.0f : i < lane ? 0.0f : -sum;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) T[(16 * block + i) * kPrepPitch + 16 * block + lane] = x[i];
        }
        __syncthreads();
        // joined to blocks of 32, then of 64: T21 = -T22 (L21 T11), the product in brackets in
        // L's free upper half
        {
            const int row0 = warp / 2 * 32, c = warp % 2 * 8;
            float y[1][4] = {};
            block_product<16, 1>(y, L + (row0 + 16) * kPrepPitch + row0,
                                 T + row0 * kPrepPitch + row0 + c, 0, 16, lane);
            put_product<1>(y, L + row0 * kPrepPitch + row0 + 16 + c, 1.0f, lane);
            __syncthreads();
            float z[1][4] = {};
            block_product<16, 1>(z, T + (row0 + 16) * kPrepPitch + row0 + 16,
                                 L + row0 * kPrepPitch + row0 + 16 + c, 0, 16, lane);
            put_product<1>(z, T + (row0 + 16) * kPrepPitch + row0 + c, -1.0f, lane);
        }
        __syncthreads();
        {
            const int r = warp % 2 * 16, c = warp / 2 * 16;
            float y[2][4] = {};
            // (T11 and T22 are zero above their diagonals)
            block_product<32, 2>(y, L + (32 + r) * kPrepPitch, T + c, c, 32, lane);
            put_product<2>(y, L + r * kPrepPitch + 32 + c, 1.0f, lane);
            __syncthreads();
            float z[2][4] = {};
            block_product<32, 2>(z, T + (32 + r) * kPrepPitch + 32, L + 32 + c, 0, r + 16, lane);
            put_product<2>(z, T + (32 + r) * kPrepPitch + c, -1.0f, lane);
        }
        __syncthreads();
        unsigned char *const to =
            m.records + (static_cast<long long>(blockIdx.x) * p.nheads + h0 + k) * R::kBytes;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int row = (tid + x * kPrepThreads) / 8, piece = tid % 8;
            const float4 *const f =
                reinterpret_cast<const float4 *>(T + row * kPrepPitch + piece * 8);
            // (half the lanes the other way round: 8 lanes' 16 bytes on 32 banks)
            const int turned = piece >> 2;
            const float4 first = f[turned], second = f[1 - turned];
            const float4 a = turned ? second : first, b = turned ? first : second;
            const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            unsigned one[4], two[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                one[i] = f2_to_bf2(v[2 * i], v[2 * i + 1]);
                two[i] = f2_to_bf2(v[2 * i] - __uint_as_float(one[i] << 16),
                                   v[2 * i + 1] - __uint_as_float(one[i] & 0xffff0000u));
            }
            const int at = row * 128 + ((piece ^ (row & 7)) << 4);
            uint4 first_part = make_uint4(one[0], one[1], one[2], one[3]);
            // M's second part, above T's diagonal
            const int of_m = piece / 2 == 3 && row < 48   ? row
                             : piece / 2 == 1 && row < 16 ? row + 48
                                                          : -1;
            if (of_m >= 0)
                first_part = *reinterpret_cast<const uint4 *>(raw + Smem::kMFirst + of_m * 32 +
                                                              piece % 2 * 16);
            *reinterpret_cast<uint4 *>(to + R::kT1 + at) = first_part;
            *reinterpret_cast<uint4 *>(to + R::kT2 + at) = make_uint4(two[0], two[1], two[2], two[3]);
            const int m_at = (tid + x * kPrepThreads) * 16;
            *reinterpret_cast<uint4 *>(to + R::kM + m_at) =
                *reinterpret_cast<const uint4 *>(raw + Smem::kM + m_at);
        }
        *reinterpret_cast<uint4 *>(to + R::kVec + tid * 16) =
            *reinterpret_cast<const uint4 *>(raw + Smem::kVec + k * 2048 + tid * 16);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    free_tmem();
}

// ---- the second pass -----------------------------------------------------------------------

constexpr int kDeltaCompute = 256;
// warps after the compute warps: one issues the products, one the copies, one looks values over,
// one stores
constexpr int kDeltaIssuer = kDeltaCompute / 32, kDeltaLoader = kDeltaIssuer + 1,
              kDeltaLooker = kDeltaIssuer + 2, kDeltaStorer = kDeltaIssuer + 3;
constexpr int kDeltaThreads = kDeltaCompute + 128;
constexpr int kDeltaStages = 3;

template <int N>
struct DeltaSmem {
    static constexpr int kBlocks = N / 64;
    static constexpr int kK = 0;           // K's and Q's blocks of 64 columns in turn: together
    static constexpr int kQ = kDeltaTile;  // they are an operand of 128 rows
    static constexpr int kBlock = 2 * kDeltaTile;
    static constexpr int kV = kBlocks * kBlock;  // the readout leaves from here
    static constexpr int kRecord = kV + 2 * kDeltaTile;
    static constexpr int kStage = kRecord + DeltaRecord::kBytes;
    static constexpr int kSwap = kDeltaStages * kStage;  // two floats per compute thread
    static constexpr int kFlags = kSwap + 2 * kDeltaCompute * 4;
    static constexpr int kBars = kFlags + 16;
    static constexpr int kTotal = kBars + 8 * (4 * kDeltaStages + 14);
    static_assert(kStage % 1024 == 0, "tiles start at 1024 bytes");
};

__device__ __forceinline__ void bulk_load(unsigned dst, const void *src, unsigned bytes,
                                          unsigned bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// f - (the bf16 halves of `bits`), exactly, in FMAs of mixed types: the same by masks and shifts is
// bound by the integer pipe, which has half their rate.
__device__ __forceinline__ float2 less_halves(float2 f, unsigned bits) {
    float2 r;
    asm("{\n\t.reg .b16 l, h, m;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "mov.b16 m, 0xbf80;\n\t"  // -1
        "fma.rn.f32.bf16 %0, l, m, %3;\n\t"
        "fma.rn.f32.bf16 %1, h, m, %4;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(bits), "f"(f.x), "f"(f.y));
    return r;
}

// Two values as bf16 parts; each part is what the ones before leave.
template <int kParts>
__device__ __forceinline__ void split2(float2 f, unsigned (&bits)[kParts]) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
        bits[k] = f2_to_bf2(f.x, f.y);
        if (k + 1 < kParts) f = less_halves(f, bits[k]);
    }
}

// Roles.  Per chunk, with the barrier of each hand-over ([r], [u], [w], [d], [q] and [m] only where
// the chunk is not taken token by token):
//
//   loader:  [empty] tiles and record -> full
//   looker:  [full] values looked over, a prompt's last chunk cut -> look
//   issuer:  [look, s] S (K, Q)^T -> p; [r] R T^T -> u; [w] U K -> d; [q] U M^T -> m, empty
//   compute: [look, p] R -> r; the last chunk's [m] readout into its V's place -> t, empty; [u] U ->
//            w; S Q^T with its decays to where U M^T adds to it, U for that -> q; [d] S -> s
//   storer:  [look, t] the readout's tile out -> empty
//
// S, R and U are handed over 16 columns of each warpgroup at a time, so that products of the first
// run while the next are made: of a product's MMAs only the last piece's are waited for.  K and Q
// are one operand, as an MMA of N = 128 takes little longer than one of N = 64.
template <int N, typename ST>
__global__ void __launch_bounds__(kDeltaThreads, 1)
    ssu_delta_mma_kernel(const __grid_constant__ DeltaMmaParams m,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ CUtensorMap map_out) {
    using Smem = DeltaSmem<N>;
    using R = DeltaRecord;
    constexpr int kParts = sizeof(ST) == 4 ? 3 : 2, kBlocks = Smem::kBlocks;
    constexpr int kCols = N / 2;           // of a row of S, per thread
    constexpr int kPieces = kCols / 16;    // of S; R and U have two
    extern __shared__ unsigned char raw[];
    __shared__ unsigned tmem_slot;
    __shared__ DeltaPrompt ranked;
    const SsuParams &p = m.d.m.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform to the compiler)
    const unsigned base = (smem_u32(raw) + 1023u) & ~1023u;
    unsigned char *const smem = raw + (base - smem_u32(raw));
    const unsigned bars = base + Smem::kBars;
    const unsigned full = bars, empty = bars + 8 * kDeltaStages, look = empty + 8 * kDeltaStages;
    const unsigned bar_t = look + 8 * kDeltaStages, bar_s = bar_t + 8 * kDeltaStages,
                   bar_r = bar_s + 32, bar_w = bar_r + 16, bar_q = bar_w + 16, bar_p = bar_q + 8,
                   bar_u = bar_p + 8, bar_d = bar_u + 8, bar_m = bar_d + 8, bar_x = bar_m + 8;
    if (tid == 0) {
        for (int i = 0; i < kDeltaStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kDeltaCompute / 32 + 2);
            mbar_init(look + 8 * i, 1);
            mbar_init(bar_t + 8 * i, kDeltaCompute / 32);
        }
        for (int i = 0; i < 9; ++i) mbar_init(bar_s + 8 * i, kDeltaCompute / 32);
        for (unsigned bar : {bar_p, bar_u, bar_d, bar_m}) mbar_init(bar, 1);
        mbar_init(bar_x, kDeltaCompute / 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kDeltaIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    // TMEM columns: S's parts, the third of which makes room for two of weighted U; the next state's
    // sum (before it, R's parts); S K^T, then U, then in its place weighted U's third part; S Q^T,
    // then U's parts for the readout; the readout's sum
    const unsigned tS = tmem, tW = tmem + 128, tD = tmem + 192, tP = tmem + 320, tQ = tmem + 384,
                   tM = tmem + 448;
    // U's weighted parts, k-step by k-step (16 tokens): two parts of 32 columns; the third in pieces
    auto weighted = [&](int part, int step) {
        return part < 2 ? tW + part * 32 + 8 * step
                        : tP + 32 * (step / 2) + 16 + 8 * (step % 2);
    };

    pdl_wait();
    const int columns = p.nheads * m.slabs;
    const int column = blockIdx.x % columns, h = column / m.slabs;
    const int row0 = (column - h * m.slabs) * kDeltaRows;
    if (m.few) {
        if (warp == 0) {
            const DeltaPrompt d = few_ranked(m, blockIdx.x / columns, lane);
            if (lane == 0) ranked = d;
        }
        __syncthreads();
    }
    const DeltaPrompt prompt = m.few ? ranked : m.prompts[blockIdx.x / columns];
    const bool good = prompt.starts != DeltaPrompt::kNot;
    const bool fresh = prompt.starts == DeltaPrompt::kZeros;
    const int begin = prompt.begin, end = prompt.end;
    const int chunks = __shfl_sync(
        0xffffffffu, good ? (end - begin + kDeltaChunk - 1) / kDeltaChunk : 0, 0);
    const int grp = group_of(h, p.group_magic);
    const int v_blocks = min(2, (p.headdim - row0 + 63) / 64);
    unsigned dead = 0;  // whether a wait gave up: what comes after it is not valid, nor waited for
    // the chunk's stage and the parity of its barriers
    int stage = 0;
    unsigned turn = 0;
    auto next_stage = [&]() {
        if (++stage == kDeltaStages) stage = 0, turn ^= 1;
    };
    auto flag = [&]() {
        return reinterpret_cast<const volatile int *>(smem + Smem::kFlags)[stage] != 0;
    };

    if (warp == kDeltaLoader) {
        if (lane == 0) {
            const unsigned bytes = (2 * kBlocks + v_blocks) * kDeltaTile + R::kBytes;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, next_stage()) {
                const unsigned to = base + stage * Smem::kStage, bar = full + 8 * stage;
                if (c >= kDeltaStages) mbar_pass(empty + 8 * stage, turn ^ 1, dead);
                if (dead) break;
                mbar_expect(bar, bytes);
                const int tok = begin + c * kDeltaChunk;
                for (int k = 0; k < kBlocks; ++k) {
                    tma_load(to + Smem::kK + k * Smem::kBlock, &map_k, bar, k * 64, grp, tok);
                    tma_load(to + Smem::kQ + k * Smem::kBlock, &map_q, bar, k * 64, grp, tok);
                }
                for (int k = 0; k < v_blocks; ++k)
                    tma_load(to + Smem::kV + k * kDeltaTile, &map_v, bar, row0 + k * 64, h, tok);
                bulk_load(to + Smem::kRecord,
                          m.records + (static_cast<long long>(prompt.first + c) * p.nheads + h) *
                                          R::kBytes,
                          R::kBytes, bar);
            }
        }
        __syncwarp();
    } else if (warp == kDeltaLooker) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, next_stage()) {
            mbar_pass(full + 8 * stage, turn, dead);
            const unsigned at = base + stage * Smem::kStage + Smem::kV;
            const int valid = min(kDeltaChunk, end - begin - c * kDeltaChunk);
            const __nv_bfloat162 zero{};
            __nv_bfloat162 sum[4] = {};
#pragma unroll 8
            for (int k = 0; k < v_blocks * kDeltaTile / 512; ++k) {  // 4 rows of a tile each
                const uint4 v = load_smem16(at + k * 512 + lane * 16);
                if ((4 * k + lane / 8) % kDeltaChunk >= valid) continue;
                sum[0] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.x), zero, sum[0]);
                sum[1] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.y), zero, sum[1]);
                sum[2] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.z), zero, sum[2]);
                sum[3] = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(v.w), zero, sum[3]);
            }
            sum[0] = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
            const bool any = __any_sync(
                0xffffffffu, (reinterpret_cast<const unsigned &>(sum[0]) & 0x7fff7fffu) != 0);
            if (valid < kDeltaChunk) {  // tokens of the next prompt, which products would meet
                for (int k = lane; k < (kDeltaChunk - valid) * 8; k += 32) {
                    const unsigned to =
                        base + stage * Smem::kStage + (valid + k / 8) * 128 + k % 8 * 16;
                    for (int t = 0; t < kBlocks; ++t)
                        store_smem16(to + Smem::kK + t * Smem::kBlock, make_uint4(0, 0, 0, 0));
                    for (int t = 0; t < v_blocks; ++t)
                        store_smem16(to + Smem::kV + t * kDeltaTile, make_uint4(0, 0, 0, 0));
                }
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                const float *const vec = reinterpret_cast<const float *>(
                    smem + stage * Smem::kStage + Smem::kRecord + R::kVec);
                reinterpret_cast<int *>(smem + Smem::kFlags)[stage] =
                    any || vec[R::kSlow] != 0.0f;
                mbar_arrive(look + 8 * stage);
            }
            __syncwarp();
        }
    } else if (warp == kDeltaStorer) {
        if (lane == 0) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, next_stage()) {
                const int tok = begin + c * kDeltaChunk;
                mbar_pass(look + 8 * stage, turn, dead);
                mbar_pass(bar_t + 8 * stage, turn, dead);
                if (dead) break;
                if (!flag() && tok + kDeltaChunk <= end) {
                    for (int k = 0; k < v_blocks; ++k)
                        tma_store(&map_out, base + stage * Smem::kStage + Smem::kV + k * kDeltaTile,
                                  row0 + k * 64, h, tok);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
                mbar_arrive(empty + 8 * stage);
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncwarp();
    } else if (warp == kDeltaIssuer) {
        const unsigned leader = elect_one();
        unsigned fast = 0;  // parity of the chunks not taken token by token
        bool any = false;
        // d, its tokens from `first` on, += a step of 16 tokens' a by a triangle's columns at b
        auto triangle = [&](unsigned d, unsigned a, unsigned b, int first, int tokens, bool add) {
            mma_ts_of(leader, d + first, a, operand(b, 0), instruction(tokens, false, false), add);
        };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, next_stage()) {
            const unsigned at = base + stage * Smem::kStage;
            mbar_pass(look + 8 * stage, turn, dead);
            if (__any_sync(0xffffffffu, flag())) {
                for (int x = 0; x < kPieces; ++x) mbar_pass(bar_s + 8 * x, c & 1, dead);
                if (leader) {
                    mbar_arrive(bar_p);
                    mbar_arrive(empty + 8 * stage);
                }
                __syncwarp();
                continue;
            }
            // U of the last such chunk has been read before its places are written
            if (any) mbar_pass(bar_m, fast ^ 1, dead);
            any = true;
#pragma unroll
            for (int x = 0; x < kPieces; ++x) {
                mbar_pass(bar_s + 8 * x, c & 1, dead);
                tc_fence_after();
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = x + half * kPieces;
                        mma_ts_of(leader, tP, tS + part * (N / 2) + 8 * k,
                                  operand(at + Smem::kK + (k / 4) * Smem::kBlock + (k % 4) * 32, 0),
                                  instruction(2 * kDeltaChunk, false, false),
                                  x > 0 || part < kParts - 1 || half > 0);
                    }
            }
            tc_commit_of(leader, bar_p);
            const unsigned t1 = at + Smem::kRecord + R::kT1, t2 = at + Smem::kRecord + R::kT2;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mbar_pass(bar_r + 8 * x, fast, dead);
                tc_fence_after();
                auto correct = [&](int part, unsigned t, bool add) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = x + 2 * half;
                        triangle(tP, tD + part * 32 + 8 * k, t + k * (2048 + 32), 16 * k, 64 - 16 * k,
                                 add || half > 0);
                    }
                };
                // small parts first: sums lose less
                if constexpr (kParts == 3) correct(2, t1, x > 0);
                correct(0, t2, kParts == 3 || x > 0);
                correct(1, t1, true);
                correct(0, t1, true);
            }
            tc_commit_of(leader, bar_u);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mbar_pass(bar_w + 8 * x, fast, dead);
                tc_fence_after();
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = x + 2 * half;
                        mma_ts_of(leader, tD, weighted(part, k),
                                  operand(at + Smem::kK + k * 2048, N == 128 ? Smem::kBlock : 0),
                                  instruction(N, false, true),
                                  x > 0 || part < kParts - 1 || half > 0);
                    }
            }
            tc_commit_of(leader, bar_d);
            mbar_pass(bar_q, fast, dead);
            tc_fence_after();
            const unsigned tile = at + Smem::kRecord + R::kM;
            auto u_at = [&](int part, int k) { return tQ + 32 * (k / 2) + 16 * part + 8 * (k % 2); };
            triangle(tM, u_at(0, 0), t1 + 3 * 32, 0, 48, true);
            triangle(tM, u_at(0, 0), t1 + 32, 48, 16, true);
#pragma unroll
            for (int k = 1; k < 4; ++k)
                triangle(tM, u_at(0, k), tile + (4 - k) * 32, 16 * k, 64 - 16 * k, true);
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    triangle(tM, u_at(part, k), tile + k * (2048 + 32), 16 * k, 64 - 16 * k, true);
            tc_commit_of(leader, empty + 8 * stage);
            tc_commit_of(leader, bar_m);
            fast ^= 1;
        }
        __syncwarp();
    } else {
        // A warp has 32 of the state's rows (TMEM lanes) and half of its columns, or half the tokens.
        // A thread has rows g + 8 e of its 16 lanes `hh`, columns 8 i + 2 t, + 1 of every block i.
        const int quarter = warp & 3, half = warp >> 2;
        const int g = lane >> 2, t = lane & 3;
        const unsigned lanes = static_cast<unsigned>(quarter) << 21;
        constexpr unsigned kLanes16 = 16u << 16;
        constexpr int kCol8 = kCols / 8;
        float2 S[kCol8][2][2];  // [block][hh][e]
        ST *const state = static_cast<ST *>(p.state) + prompt.slot * p.st_pool + h * p.st_head +
                          half * kCols + 2 * t;
        auto row_at = [&](int hh, int e) { return 32 * quarter + 16 * hh + 8 * e + g; };
        const bool reads = good && !fresh && chunks;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = row0 + row_at(hh, e);
                const ST *const from = state + row * p.st_row;
#pragma unroll
                for (int i = 0; i < kCol8; ++i) {
                    S[i][hh][e] = make_float2(0.0f, 0.0f);
                    if (!reads || row >= p.headdim) continue;
                    if constexpr (sizeof(ST) == 4) {
                        S[i][hh][e] = __ldcs(reinterpret_cast<const float2 *>(from + 8 * i));
                    } else {
                        const unsigned w = __ldcs(reinterpret_cast<const unsigned *>(from + 8 * i));
                        S[i][hh][e] = make_float2(__uint_as_float(w << 16),
                                                  __uint_as_float(w & 0xffff0000u));
                    }
                }
            }
        auto hand_over = [&](unsigned bar) {
            tc_wait_st();
            tc_fence_before();
            warp_arrive(bar, lane);
        };
        // Two blocks of pairs as bf16 parts, to the columns that `to(part)` names.
        auto put_parts = [&](auto parts, const float2 (&f)[2][2][2], auto to) {
            constexpr int kN = decltype(parts)::value;
            unsigned bits[kN][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        unsigned w[kN];
                        split2<kN>(f[i][hh][e], w);
#pragma unroll
                        for (int part = 0; part < kN; ++part) bits[part][hh][2 * i + e] = w[part];
                    }
#pragma unroll
            for (int part = 0; part < kN; ++part)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    tc_store_frag(to(part) + lanes + hh * kLanes16, bits[part][hh]);
        };
        auto publish = [&](int x) {  // 16 columns of S as the next products' operand
            const float2 f[2][2][2] = {
                {{S[2 * x][0][0], S[2 * x][0][1]}, {S[2 * x][1][0], S[2 * x][1][1]}},
                {{S[2 * x + 1][0][0], S[2 * x + 1][0][1]},
                 {S[2 * x + 1][1][0], S[2 * x + 1][1][1]}}};
            put_parts(std::integral_constant<int, kParts>(), f, [&](int part) { return tS + part * (N / 2) + half * (N / 4) + 8 * x; });
            hand_over(bar_s + 8 * x);
        };
        if (chunks)
#pragma unroll
            for (int x = 0; x < kPieces; ++x) publish(x);
        unsigned fast = 0;
        // Matrix k % 4 of 16 tokens and 16 rows `hh` in V's tiles, where ldmatrix and stmatrix take
        // their rows' addresses from lanes.
        auto v_at = [&](unsigned at, int x, int hh) {
            const int token = 32 * half + 16 * x + 8 * (lane >> 4) + (lane & 7);
            const int row = 32 * quarter + 16 * hh + 8 * (lane >> 3 & 1);
            return swizzled(at + Smem::kV + (row >> 6) * kDeltaTile, token, (row & 63) >> 3);
        };
        // the two tokens of block i (of the warpgroup's four) that the thread has
        auto factors = [&](const float *vec, int kind, int i) {
            return *reinterpret_cast<const float2 *>(vec + kind + 32 * half + 8 * i + 2 * t);
        };
        auto vec_of = [&](int stage) {
            return reinterpret_cast<const float *>(smem + stage * Smem::kStage + Smem::kRecord +
                                                   R::kVec);
        };
        // The readout of chunk c, the last one, whose products have been waited for by nobody yet.
        bool waits = false;
        auto read_out = [&](int c) {
            const int last = stage == 0 ? kDeltaStages - 1 : stage - 1;
            const unsigned at = base + last * Smem::kStage;
            const float *const vec = vec_of(last);
            const int tok = begin + c * kDeltaChunk, valid = min(kDeltaChunk, end - tok);
            mbar_pass(bar_m, fast ^ 1, dead);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                unsigned um[2][8], y[2][4];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    tc_load_frag(tM + lanes + hh * kLanes16 + 32 * half + 16 * x, um[hh]);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 read = factors(vec, R::kRead, 2 * x + i);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = 4 * i + 2 * e;
                            const float2 f = __fmul2_rn(
                                read, make_float2(__uint_as_float(um[hh][k]),
                                                  __uint_as_float(um[hh][k + 1])));
                            y[hh][2 * i + e] = f2_to_bf2(f.x, f.y);
                        }
                }
                if (valid == kDeltaChunk) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) store_trans4(v_at(at, x, hh), y[hh]);
                } else {
                    __nv_bfloat16 *const out = p.out + static_cast<long long>(tok) * p.out_b +
                                               h * p.out_h + row0;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int hh = k / 8, i = k / 4 % 2, e = k / 2 % 2, odd = k % 2;
                        const int token = 32 * half + 16 * x + 8 * i + 2 * t + odd;
                        const int row = row_at(hh, e);
                        if (token < valid && row0 + row < p.headdim)
                            out[token * p.out_b + row] =
                                __ushort_as_bfloat16(y[hh][2 * i + e] >> (16 * odd));
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(bar_t + 8 * last, lane);
            warp_arrive(empty + 8 * last, lane);
            waits = false;
        };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, next_stage()) {
            const unsigned at = base + stage * Smem::kStage;
            const int tok = begin + c * kDeltaChunk, valid = min(kDeltaChunk, end - tok);
            const float *const vec = vec_of(stage);
            __nv_bfloat16 *const out = p.out + static_cast<long long>(tok) * p.out_b +
                                       h * p.out_h + row0;
            mbar_pass(look + 8 * stage, turn, dead);
            __syncwarp();
            if (__builtin_expect(__any_sync(0xffffffffu, flag()), 0)) {
                if (waits) read_out(c - 1);
                float *const swap = reinterpret_cast<float *>(smem + Smem::kSwap);
                // the rows' sums over the quad's lanes and both warpgroups' columns (twice a token: the
                // first one's barrier has the parity 0)
                auto whole_rows = [&](float (&sum)[2][2], float *room, unsigned parity) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            sum[hh][e] += __shfl_xor_sync(0xffffffffu, sum[hh][e], 1);
                            sum[hh][e] += __shfl_xor_sync(0xffffffffu, sum[hh][e], 2);
                            if (t == 0) room[half * kDeltaRows + row_at(hh, e)] = sum[hh][e];
                        }
                    // (not a barrier of the CTA's: where a wait has given up, warps may have
                    // parted, and every wait has to end)
                    warp_arrive(bar_x, lane);
                    mbar_pass(bar_x, parity, dead);
                    __syncwarp();
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            sum[hh][e] =
                                room[row_at(hh, e)] + room[kDeltaRows + row_at(hh, e)];
                };
                // the thread's two columns of block i of token k's key or query, at its length (before
                // any product: a length past fp32 leaves zeros)
                auto pair_of = [&](int tile, int k, int i, float factor) {
                    const int col = half * kCols + 8 * i;
                    unsigned w;
                    asm volatile("ld.shared.u32 %0, [%1];"
                                 : "=r"(w)
                                 : "r"(swizzled(at + tile + (col / 64) * Smem::kBlock, k,
                                                col % 64 / 8) + 4 * t)
                                 : "memory");
                    return make_float2(__uint_as_float(w << 16) * factor,
                                       __uint_as_float(w & 0xffff0000u) * factor);
                };
#pragma unroll 1
                for (int k = 0; k < valid; ++k) {
                    const float a = vec[R::kDecay + k], rk = vec[R::kKey + k], rq = vec[R::kRead + k];
                    float sum[2][2] = {};
#pragma unroll
                    for (int i = 0; i < kCol8; ++i) {
                        const float2 key = pair_of(Smem::kK, k, i, rk);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float2 s = S[i][x / 2][x % 2];
                            sum[x / 2][x % 2] += s.x * key.x + s.y * key.y;
                        }
                    }
                    whole_rows(sum, swap, 0);
                    float e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int row = row_at(x / 2, x % 2);
                        unsigned short v;
                        asm volatile("ld.shared.u16 %0, [%1];"
                                     : "=h"(v)
                                     : "r"(swizzled(at + Smem::kV + row / 64 * kDeltaTile, k,
                                                    row % 64 / 8) + 2 * (row % 8))
                                     : "memory");
                        e[x] = vec[R::kBeta + k] * (__uint_as_float(static_cast<unsigned>(v) << 16) -
                                                    a * sum[x / 2][x % 2]);
                        sum[x / 2][x % 2] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < kCol8; ++i) {
                        const float2 key = pair_of(Smem::kK, k, i, rk),
                                     q = pair_of(Smem::kQ, k, i, rq);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float2 &s = S[i][x / 2][x % 2];
                            s.x = fmaf(s.x, a, e[x] * key.x);
                            s.y = fmaf(s.y, a, e[x] * key.y);
                            sum[x / 2][x % 2] += s.x * q.x + s.y * q.y;
                        }
                    }
                    whole_rows(sum, swap + kDeltaCompute, 1);
                    if (half == 0 && t == 0)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int row = row_at(x / 2, x % 2);
                            if (row0 + row < p.headdim)
                                out[k * p.out_b + row] = __float2bfloat16(sum[x / 2][x % 2]);
                        }
                }
                mbar_pass(bar_p, c & 1, dead);  // the issuer has come this far
                __syncwarp();
                if (c + 1 < chunks)
#pragma unroll
                    for (int x = 0; x < kPieces; ++x) publish(x);
                warp_arrive(bar_t + 8 * stage, lane);
                warp_arrive(empty + 8 * stage, lane);
                continue;
            }
            // R = beta v - (beta e^s / |k|) S k
            unsigned v[2][2][4];  // [piece][hh][block, e]
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) load_trans4(v[x][hh], v_at(at, x, hh));
            mbar_pass(bar_p, c & 1, dead);
            __syncwarp();
            tc_fence_after();
            {
                unsigned sk[2][2][8];
                auto fetch = [&](int x) {  // the next piece on its way under this one's work
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
                        tc_load_frag(tP + lanes + hh * kLanes16 + 32 * half + 16 * x, sk[x][hh]);
                };
                fetch(0);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float2 r[2][2][2];
                    tc_wait_ld();
                    if (x == 0) fetch(1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 beta = factors(vec, R::kBeta, 2 * x + i);
                        const float2 past = factors(vec, R::kPast, 2 * x + i);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const unsigned u = v[x][hh][2 * i + e];
                                const int k = 4 * i + 2 * e;
                                r[i][hh][e] = __ffma2_rn(
                                    make_float2(-past.x, -past.y),
                                    make_float2(__uint_as_float(sk[x][hh][k]),
                                                __uint_as_float(sk[x][hh][k + 1])),
                                    __fmul2_rn(beta, make_float2(__uint_as_float(u << 16),
                                                                 __uint_as_float(u & 0xffff0000u))));
                            }
                    }
                    put_parts(std::integral_constant<int, kParts>(), r, [&](int part) { return tD + part * 32 + 16 * half + 8 * x; });
                    // (R T^T goes over S K^T from its first piece on: no load of what the next product
                    // overwrites is in flight where its operand is handed over)
                    if (x == 0) tc_wait_ld();
                    hand_over(bar_r + 8 * x);
                }
            }
            if (waits) read_out(c - 1);  // under R T^T
            // U with its weights for the next state; then (under U K) S Q^T with its decays to where U M^T
            // will add to it, and U for the readout
            mbar_pass(bar_u, fast, dead);
            __syncwarp();
            tc_fence_after();
            {
                unsigned u[2][2][8];
                auto fetch = [&](int x) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
                        tc_load_frag(tP + lanes + hh * kLanes16 + 32 * half + 16 * x, u[x][hh]);
                };
                auto of_u = [&](int x, int i, int hh, int e) {
                    const int k = 4 * i + 2 * e;
                    return make_float2(__uint_as_float(u[x][hh][k]),
                                       __uint_as_float(u[x][hh][k + 1]));
                };
                fetch(0);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float2 w[2][2][2];
                    tc_wait_ld();
                    if (x == 0) fetch(1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 left = factors(vec, R::kLeft, 2 * x + i);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                w[i][hh][e] = __fmul2_rn(of_u(x, i, hh, e), left);
                    }
                    if (x == 0) tc_wait_ld();  // (the third part goes over what has been read)
                    put_parts(std::integral_constant<int, kParts>(), w, [&](int part) { return weighted(part, 2 * half + x); });
                    hand_over(bar_w + 8 * x);
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    unsigned sq[16];
                    tc_load_frag(tQ + lanes + hh * kLanes16 + 32 * half, sq);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 past = factors(vec, R::kReadS, i);
#pragma unroll
                        for (int k = 4 * i; k < 4 * i + 4; k += 2) {
                            const float2 f =
                                __fmul2_rn(past, make_float2(__uint_as_float(sq[k]),
                                                             __uint_as_float(sq[k + 1])));
                            sq[k] = __float_as_uint(f.x);
                            sq[k + 1] = __float_as_uint(f.y);
                        }
                    }
                    tc_store_frag(tM + lanes + hh * kLanes16 + 32 * half, sq);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float2 f[2][2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int e = 0; e < 2; ++e) f[i][hh][e] = of_u(x, i, hh, e);
                    put_parts(std::integral_constant<int, 2>(), f, [&](int part) { return tQ + 32 * half + 16 * part + 8 * x; });
                }
                hand_over(bar_q);
            }
            const float whole = vec[R::kWhole];
            mbar_pass(bar_d, fast, dead);
            __syncwarp();
            tc_fence_after();
            {
                unsigned d[2][2][8];
                auto fetch = [&](int x) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
                        tc_load_frag(tD + lanes + hh * kLanes16 + half * kCols + 16 * x,
                                     d[x % 2][hh]);
                };
                fetch(0);
#pragma unroll
                for (int x = 0; x < kPieces; ++x) {
                    tc_wait_ld();
                    if (x + 1 < kPieces) fetch(x + 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int k = 4 * i + 2 * e;
                                float2 &s = S[2 * x + i][hh][e];
                                s = __ffma2_rn(s, make_float2(whole, whole),
                                               make_float2(__uint_as_float(d[x % 2][hh][k]),
                                                           __uint_as_float(d[x % 2][hh][k + 1])));
                            }
                    if (c + 1 < chunks) publish(x);
                }
            }
            waits = true;
            fast ^= 1;
        }
        if (waits) read_out(chunks - 1);
        if (good && (chunks || fresh))
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = row0 + row_at(hh, e);
                    if (row >= p.headdim) continue;
                    ST *const to = state + row * p.st_row;
#pragma unroll
                    for (int i = 0; i < kCol8; ++i) {
                        if constexpr (sizeof(ST) == 4)
                            __stcs(reinterpret_cast<float2 *>(to + 8 * i), S[i][hh][e]);
                        else
                            __stcs(reinterpret_cast<unsigned *>(to + 8 * i),
                                   f2_to_bf2(S[i][hh][e].x, S[i][hh][e].y));
                    }
                }
    }
    tc_fence_before();
    if (__syncthreads_or(dead)) {  // what is in flight lands long before this is over
        if (tid == 0) atomicOr(&p.err[2], 1u);
        __nanosleep(1000000);
    }
    __syncthreads();
    if (warp == kDeltaIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

}  // namespace
