// One token's attention over a paged cache (sm_103a), instantiated by ssu_attend.cu.
//
// Mathematics.  For a key head and the query heads that share it, out = softmax(scale q K^T) V
// over the visible keys.  Any split of the keys can be computed apart: a part keeps, per query
// head, its largest score m, l = sum exp(s - m) and o = sum exp(s - m) v, and parts join by
// m* = max m, l* = sum l exp(m - m*), o* = sum o exp(m - m*).  Scores, m, l and o are fp32; the
// weights exp(s - m) are rounded to bf16 as operands of the product with v (2^-9 of a weight in
// the mean square, as much as v itself carries).
//
// What bounds it: HBM, reading K and V once (4 D bytes per key and key head).  Up to 16 query
// heads of a key head are the 16 rows of an m16n8k16 MMA, so every byte of K and V that reaches
// a warp is used for all of them, and 32 MMAs per 16 keys are far below the tensor pipe's rate
// whatever the rows' number.
//
// Split.  The work of all requests is one line of tiles of kTile keys (request by request, key
// head by key head), cut into equal stretches, one per CTA, one CTA per SM: the longest and the
// shortest requests of a batch are balanced to one tile whatever their lengths, without the
// host knowing any.  A CTA that has the whole of a unit (a request's key head) writes its
// output; units cut by a stretch's end leave their part in the workspace and the last CTA to
// arrive joins the parts, in their order, so results do not depend on timing.
//
// Inside a CTA every warp takes its 16 or 32 of a tile's keys into its own ring of stages with
// cp.async (rows 16 bytes apart in banks, so ldmatrix has no conflicts), ahead of their use across
// unit borders, and keeps its own m, l, o: no barrier until a unit ends.  (A bulk copy per row and
// lane instead was 20 % slower: its operands are a warp's, so 32 rows are 32 turns.)

#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ssu_device.cuh"

namespace {

struct AttendParams {
    const __nv_bfloat16 *q, *k, *v;
    const void *table, *lengths;
    __nv_bfloat16 *out;
    long long q_b, q_h, o_b, o_h;
    long long k_p, k_r, k_h, v_p, v_r, v_h;
    long long t_b, t_p, len_s;
    long long requests, num_pages, max_keys;
    long long window, sinks;
    int page_size, q_heads, kv_heads;
    int wide;        // the cache's extent in 16-byte vectors passes 32 bits
    int share;       // query heads per key head
    int head_tiles;  // ceil(share / 16)
    float scale_log2;  // scale * log2 e: weights are exp2 of differences
    unsigned *err;
    unsigned *arrived;  // one counter per CTA; zero between calls
    float *parts;       // two parts per CTA
};

constexpr int kAttendRows = 16;     // query heads per unit: the MMA's M

// Keys per warp and step: the second product's K, twice for the shortest rows, whose steps would
// otherwise be as long as those of twice the bytes (40 requests through a window of 1000, 8 heads
// of 64: 28.0 us, 0.92 of the time with 16).
template <int D>
struct AttendGeo {
    static constexpr int kKeys = D == 64 ? 32 : 16;
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kTile = kWarps * kKeys;
    static constexpr int kPitch = D * 2 + 16;  // bytes per row: 8 rows of an ldmatrix on 32 banks
    static constexpr int kStageBytes = 2 * kKeys * kPitch;  // K and V of a warp's keys
    static constexpr int kStages = 3;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = (kWarps / 2) * (kAttendRows / 2) * D * 4;  // half the rows
    static constexpr int kStatBytes = kWarps * kAttendRows * 2 * 4;
    static constexpr int kSmem = kRingBytes + kMergeBytes + kStatBytes;
    static constexpr int kPartFloats = kAttendRows * D + 2 * kAttendRows;
};

template <bool kIdx64>
__device__ __forceinline__ long long load_index(const void *ids, long long at) {
    if (kIdx64) return __ldg(static_cast<const long long *>(ids) + at);
    return static_cast<long long>(__ldg(static_cast<const int *>(ids) + at));
}

// A request's visible keys as one contiguous index: index i is position i for i < head, else
// i - head + from.
struct Visible {
    int count, head, from;
};

// The visible keys of request b; count = 0 for an invalid length (`good` = false).
template <bool kIdx64>
__device__ __forceinline__ Visible visible_of(const AttendParams &p, long long b, bool &good) {
    const long long n = load_index<kIdx64>(p.lengths, b * p.len_s);
    good = n >= 0 && n <= p.max_keys;
    Visible v{0, 0, 0};
    if (!good) return v;
    if (p.window > 0 && n > p.window) {
        v.from = static_cast<int>(n - p.window);
        v.head = static_cast<int>(p.sinks < v.from ? p.sinks : v.from);
    }
    v.count = static_cast<int>(n) - v.from + v.head;
    return v;
}

// A place in the line: tiles of a unit, then kUnitCost empty places that stand for the time that
// joining its warps takes, so that a stretch of many short units is as long as one of few long
// ones (128 ragged requests: 28.5 us, 0.89 of the time without).
constexpr int kUnitCost = 1;

// Whether request b has no places and is for CTA `cta` of `ctas` to see to in the end; threads also
// ask past the last request.
__host__ __device__ inline bool sees_to(long long b, long long requests, unsigned places,
                                        unsigned cta, unsigned ctas) {
    return b < requests && places == 0 && static_cast<unsigned>(b) % ctas == cta;
}

struct Cursor {
    long long at;   // place of the tile in the line
    long long b;    // request
    int unit;       // key head * head_tiles + head tile
    int tile, tiles;
    Visible vis;
};

template <int D, bool kIdx64>
__device__ __forceinline__ void enter_request(const AttendParams &p, Cursor &c) {
    bool good;
    c.vis = visible_of<kIdx64>(p, c.b, good);
    c.tiles = (c.vis.count + AttendGeo<D>::kTile - 1) / AttendGeo<D>::kTile;
}

// Moves to the next tile; past the line's last tile `at` is its end, and nothing else is right.
template <int D, bool kIdx64>
__device__ __forceinline__ void advance(const AttendParams &p, Cursor &c) {
    ++c.at;
    if (++c.tile < c.tiles) return;
    c.at += kUnitCost;
    c.tile = 0;
    if (++c.unit < p.kv_heads * p.head_tiles) return;
    c.unit = 0;
    do {
        if (++c.b >= p.requests) return;
        enter_request<D, kIdx64>(p, c);
    } while (c.tiles == 0);
}

__device__ __forceinline__ unsigned smem_addr(const void *p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where the lane's key of a step lies (where a step has 16 keys, lanes 16 .. 31 repeat lanes 0 ..
// 15).  The page id is kept as it was loaded, a step ahead of its use: a look at it right behind
// the load would wait for it.
template <bool kIdx64>
struct KeyPlace {
    using Id = typename std::conditional<kIdx64, long long, int>::type;
    Id page;
    int row;      // of the page; -1: no such key
    bool counts;  // whether a bad page is this key's to count
};

template <int D, bool kIdx64>
__device__ __forceinline__ KeyPlace<kIdx64> place_of(const AttendParams &p, const Cursor &c,
                                                     int warp, int lane) {
    using Id = typename KeyPlace<kIdx64>::Id;
    constexpr int kKeys = AttendGeo<D>::kKeys;
    const int i = c.tile * AttendGeo<D>::kTile + warp * kKeys + lane % kKeys;
    KeyPlace<kIdx64> at{0, -1, false};
    if (i >= c.vis.count) return at;
    const int j = i < c.vis.head ? i : i - c.vis.head + c.vis.from;
    const int col = j / p.page_size;
    at.row = j - col * p.page_size;
    at.page = __ldg(static_cast<const Id *>(p.table) + c.b * p.t_b + col * p.t_p);
    // a bad page counts once: for the request's first unit, at the page's first visible position
    // (its start, or the window's start where the sinks leave its earlier positions out)
    at.counts = c.unit == 0 && lane < kKeys &&
                (at.row == 0 || (j == c.vis.from && c.vis.head <= j - at.row));
    return at;
}

// Starts the copies of the warp's keys and values of one step into `stage` and returns which keys
// exist; rows without a key are zero-filled (a weight of zero meets what lies there).  Lane l
// works out where key l and its value lie, in 16-byte vectors from the cache's start, and hands
// that to the lanes that copy the rows.
template <int D, bool kIdx64>
__device__ __forceinline__ unsigned start_step(const AttendParams &p, const Cursor &c,
                                               const KeyPlace<kIdx64> &at, unsigned stage,
                                               int lane) {
    using Geo = AttendGeo<D>;
    constexpr int kPieces = D / 8;  // 16-byte pieces per row
    constexpr int kRowsPer = 32 / kPieces;
    const bool live = at.row >= 0 && at.page >= 0 && at.page < p.num_pages;
    if (at.row >= 0 && !live && at.counts) {
        atomicAdd(&p.err[0], 1u);
        atomicMin(&p.err[1], static_cast<unsigned>(c.b));
    }
    const unsigned keys =
        __ballot_sync(0xffffffffu, live) & (Geo::kKeys == 32 ? ~0u : (1u << (Geo::kKeys & 31)) - 1);
    const int kh = c.unit / p.head_tiles;
    unsigned long long k_off = 0, v_off = 0;
    if (live) {
        k_off = static_cast<unsigned long long>(at.page * p.k_p + at.row * p.k_r + kh * p.k_h) >> 3;
        v_off = static_cast<unsigned long long>(at.page * p.v_p + at.row * p.v_r + kh * p.v_h) >> 3;
    }
    const int piece = lane % kPieces, first = lane / kPieces;
    const uint4 *const k0 = reinterpret_cast<const uint4 *>(p.k) + piece;
    const uint4 *const v0 = reinterpret_cast<const uint4 *>(p.v) + piece;
    const unsigned dst = stage + first * Geo::kPitch + piece * 16;
#pragma unroll
    for (int i = 0; i < Geo::kKeys / kRowsPer; ++i) {
        const int key = i * kRowsPer + first;
        unsigned long long ko = __shfl_sync(0xffffffffu, static_cast<unsigned>(k_off), key);
        unsigned long long vo = __shfl_sync(0xffffffffu, static_cast<unsigned>(v_off), key);
        if (p.wide) {
            ko |= static_cast<unsigned long long>(
                      __shfl_sync(0xffffffffu, static_cast<unsigned>(k_off >> 32), key)) << 32;
            vo |= static_cast<unsigned long long>(
                      __shfl_sync(0xffffffffu, static_cast<unsigned>(v_off >> 32), key)) << 32;
        }
        const int bytes = (keys >> key) & 1u ? 16 : 0;  // of no key: vector 0 of the cache, unread
        const unsigned to = dst + i * kRowsPer * Geo::kPitch;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(k0 + ko),
                     "r"(bytes)
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         to + Geo::kKeys * Geo::kPitch),
                     "l"(v0 + vo), "r"(bytes)
                     : "memory");
    }
    return keys;
}

// A warp's sums over the keys it has seen of one unit, in the MMA's accumulator layout: lane
// (g = lane / 4, t = lane % 4) holds rows g and g + 8, columns 8 n + 2 t, + 1 of every n.
template <int D>
struct Sums {
    float o[D / 8][4];
    float m[2], l[2];
};

template <int D>
__device__ __forceinline__ void clear(Sums<D> &s) {
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s.o[n][i] = 0.0f;
    s.m[0] = s.m[1] = -INFINITY;
    s.l[0] = s.l[1] = 0.0f;
}

// 2^x by the hardware's approximation (2 ulp), results below 2^-126 as 0.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// One step: the keys of `stage` (of which those with a bit in `live` exist) into the sums.
template <int D>
__device__ __forceinline__ void step(const AttendParams &p, Sums<D> &s,
                                     const unsigned (&q)[D / 16][4], unsigned stage,
                                     unsigned live, int lane) {
    constexpr int kPitch = AttendGeo<D>::kPitch, kKeys = AttendGeo<D>::kKeys, kBlocks = kKeys / 8;
    const int mi = lane >> 3, r = lane & 7;
    // two chains per block of 8 keys, so that a product does not wait for the one before
    float sc[kBlocks][4] = {}, sd[kBlocks][4] = {};
    {
        const unsigned base = stage + ((mi >> 1) * 8 + r) * kPitch + (mi & 1) * 16;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2)
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) {
                unsigned b[4], c[4];
                ldmatrix4(b, base + k * 16 * kPitch + ks * 32);
                ldmatrix4(c, base + k * 16 * kPitch + ks * 32 + 32);
                mma_bf16(sc[2 * k], q[ks], b[0], b[1]);
                mma_bf16(sc[2 * k + 1], q[ks], b[2], b[3]);
                mma_bf16(sd[2 * k], q[ks + 1], c[0], c[1]);
                mma_bf16(sd[2 * k + 1], q[ks + 1], c[2], c[3]);
            }
    }
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = (sc[n][i] + sd[n][i]) * p.scale_log2;
    if (live != (kKeys == 32 ? ~0u : (1u << (kKeys & 31)) - 1)) {
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!((live >> (8 * n + 2 * t + (i & 1))) & 1u)) sc[n][i] = -INFINITY;
    }
    float keep[2], base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
            top = fmaxf(top, fmaxf(sc[n][2 * h], sc[n][2 * h + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float m = fmaxf(s.m[h], top);
        base[h] = finite_or_zero(m);
        keep[h] = exp2_ftz(s.m[h] - base[h]);
        s.m[h] = m;
    }
    unsigned w[kKeys / 16][4];
    float add[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = exp2_ftz(sc[n][2 * h] - base[h]);
            const float b = exp2_ftz(sc[n][2 * h + 1] - base[h]);
            add[h] += a + b;
            w[n / 2][2 * (n & 1) + h] = f2_to_bf2(a, b);
        }
    s.l[0] = s.l[0] * keep[0] + add[0];
    s.l[1] = s.l[1] * keep[1] + add[1];
    if (__any_sync(0xffffffffu, keep[0] != 1.0f || keep[1] != 1.0f)) {  // a new largest score
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            s.o[n][0] *= keep[0], s.o[n][1] *= keep[0];
            s.o[n][2] *= keep[1], s.o[n][3] *= keep[1];
        }
    }
    const unsigned vbase = stage + (kKeys + (mi & 1) * 8 + r) * kPitch + (mi >> 1) * 16;
#pragma unroll
    for (int k = 0; k < kKeys / 16; ++k)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            unsigned b[4];
            ldmatrix4_trans(b, vbase + k * 16 * kPitch + j * 32);
            mma_bf16(s.o[2 * j], w[k], b[0], b[1]);
            mma_bf16(s.o[2 * j + 1], w[k], b[2], b[3]);
        }
}

// The 16 query heads of the cursor's unit as A operands (rows past the last are zero).
template <int D>
__device__ __forceinline__ void load_queries(const AttendParams &p, const Cursor &c,
                                             unsigned (&q)[D / 16][4], int lane) {
    const int kh = c.unit / p.head_tiles, first = (c.unit - kh * p.head_tiles) * kAttendRows;
    const int g = lane >> 2, t = lane & 3;
    const __nv_bfloat16 *base = p.q + c.b * p.q_b + (kh * p.share + first) * p.q_h + 2 * t;
    const bool lo = first + g < p.share, hi = first + g + 8 < p.share;
    const unsigned *a = reinterpret_cast<const unsigned *>(base + (lo ? g : 0) * p.q_h);
    const unsigned *b = reinterpret_cast<const unsigned *>(base + (hi ? g + 8 : 0) * p.q_h);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        q[ks][0] = lo ? __ldg(a + ks * 8) : 0u;
        q[ks][1] = hi ? __ldg(b + ks * 8) : 0u;
        q[ks][2] = lo ? __ldg(a + ks * 8 + 4) : 0u;
        q[ks][3] = hi ? __ldg(b + ks * 8 + 4) : 0u;
    }
}

// Joins the warps' sums of a unit: every warp's o scaled to the unit's m, then added pairwise
// (upper half of the warps to the lower) and over the rest by all threads, always in the same
// order; half the rows at a time, to leave the ring its room, and the upper half only where there
// are query heads in it (`rows` of them in all).  m and l are the unit's for the lane's rows
// lane / 4 and lane / 4 + 8; `mine[h]` are the sums of the element pairs that the thread owns of
// row lane / 4 + 8 h: pair e is columns 8 n + 2 (lane % 4), + 1 with n = warp + e * kWarps.
template <int D>
using Owned = float2[2][D / 8 / AttendGeo<D>::kWarps];

template <int D>
__device__ __forceinline__ void merge_warps(Sums<D> &s, float *merge, float *stat, int rows,
                                            int warp, int lane, Owned<D> &mine, float (&m)[2],
                                            float (&l)[2]) {
    constexpr int W = AttendGeo<D>::kWarps;
    const int g = lane >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 1);
        s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 2);
        if ((lane & 3) == 0)
            reinterpret_cast<float2 *>(stat)[warp * kAttendRows + g + 8 * h] =
                make_float2(s.m[h], s.l[h]);
    }
    __syncthreads();
    float2 *buf = reinterpret_cast<float2 *>(merge);  // [W / 2][D / 8][32 lanes]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && rows <= 8) break;
        float2 ml[W];
        m[h] = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            ml[w] = reinterpret_cast<const float2 *>(stat)[w * kAttendRows + g + 8 * h];
            m[h] = fmaxf(m[h], ml[w].x);
        }
        const float base = finite_or_zero(m[h]);
        l[h] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) l[h] = fmaf(ml[w].y, exp2_ftz(ml[w].x - base), l[h]);
        const float own = exp2_ftz(s.m[h] - base);
        if (h) __syncthreads();
        if (warp >= W / 2) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                buf[((warp - W / 2) * (D / 8) + n) * 32 + lane] =
                    make_float2(s.o[n][2 * h] * own, s.o[n][2 * h + 1] * own);
        }
        __syncthreads();
        if (warp < W / 2) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                float2 &at = buf[(warp * (D / 8) + n) * 32 + lane];
                at = make_float2(fmaf(s.o[n][2 * h], own, at.x),
                                 fmaf(s.o[n][2 * h + 1], own, at.y));
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < D / 8 / W; ++e) {
            float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < W / 2; ++w) {
                const float2 a = buf[(w * (D / 8) + warp + e * W) * 32 + lane];
                t.x += a.x, t.y += a.y;
            }
            mine[h][e] = t;
        }
    }
}

// Query heads in the unit's 16 rows.
__device__ __forceinline__ int rows_of(const AttendParams &p, int unit) {
    const int left = p.share - unit % p.head_tiles * kAttendRows;
    return left < kAttendRows ? left : kAttendRows;
}

// The unit's output rows from the threads' sums.
template <int D>
__device__ __forceinline__ void write_rows(const AttendParams &p, long long b, int unit,
                                           const Owned<D> &mine, const float (&l)[2], int warp,
                                           int lane) {
    constexpr int W = AttendGeo<D>::kWarps;
    const int kh = unit / p.head_tiles, first = (unit - kh * p.head_tiles) * kAttendRows;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = first + (lane >> 2) + 8 * h;
        if (row >= p.share) return;
        const float f = l[h] == 0.0f ? 0.0f : 1.0f / l[h];  // no visible key (l = 0): zeros
        __nv_bfloat16 *dst = p.out + b * p.o_b + (kh * p.share + row) * p.o_h + 2 * (lane & 3);
#pragma unroll
        for (int e = 0; e < D / 8 / W; ++e)
            *reinterpret_cast<unsigned *>(dst + 8 * (warp + e * W)) =
                f2_to_bf2(mine[h][e].x * f, mine[h][e].y * f);
    }
}

// A unit that a CTA's stretch does not hold whole.
struct Partial {
    long long b, begin;  // request; place of the unit's first tile in the line
    int unit, tiles;     // tiles = 0: none
};

// A part is two slots per CTA: slot 1 for the unit that begins in the CTA's stretch, slot 0 for
// the one that began before it.  It holds (m, l) of the 16 rows, then the sums of the lower and the
// upper 8 rows: columns 8 n .. 8 n + 7 at float2 32 n + lane.
template <int D>
__device__ __forceinline__ float2 *part_of(const AttendParams &p, long long cta, int slot) {
    return reinterpret_cast<float2 *>(p.parts + (2 * cta + slot) * AttendGeo<D>::kPartFloats);
}

template <int D>
__device__ __forceinline__ void write_part(const AttendParams &p, int unit, int slot,
                                           const Owned<D> &mine, const float (&m)[2],
                                           const float (&l)[2], int warp, int lane) {
    constexpr int W = AttendGeo<D>::kWarps;
    float2 *to = part_of<D>(p, blockIdx.x, slot);
    const int rows = rows_of(p, unit);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && rows <= 8) break;
        if (warp == 0 && (lane & 3) == 0)
            __stcg(to + (lane >> 2) + 8 * h, make_float2(m[h], l[h]));
#pragma unroll
        for (int e = 0; e < D / 8 / W; ++e)
            __stcg(to + kAttendRows + (h * (D / 8) + warp + e * W) * 32 + lane, mine[h][e]);
    }
}

// Joins the parts of a unit and writes its rows: the parts come into shared memory (the ring is
// free by now), as many at a time as fit, all their copies together; (m, l) become each row's
// weights (a running maximum from part to part was a chain of 200 cycles for each), and every
// thread sums the pairs that it owns over the parts.  The order is fixed.  The loops stay rolled:
// this code runs once per CTA, after a stream that has pushed it out of every cache, and unrolled
// its fetch alone took longer than the join (14 us for 38 parts).
template <int D>
__device__ __forceinline__ void join_parts(const AttendParams &p, const Partial &u, int first,
                                           int last, float2 *room, float2 *stat, int warp,
                                           int lane) {
    using Geo = AttendGeo<D>;
    constexpr int W = Geo::kWarps, E = D / 8 / W;
    const int rows = rows_of(p, u.unit), tid = 32 * warp + lane;
    const int halves = rows > 8 ? 2 : 1;
    const int vecs = (kAttendRows + halves * (D / 8) * 32) / 2;  // 16-byte vectors of a part
    const int fit = Geo::kRingBytes / 16 / vecs;                 // parts at a time
    Owned<D> mine;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) mine[h][e] = make_float2(0.0f, 0.0f);
    for (int k0 = first; k0 <= last; k0 += fit) {
        const int count = min(fit, last + 1 - k0);
        __syncthreads();  // `room` is free
#pragma unroll 1
        for (int k = warp; k < count; k += W) {  // a part per warp
            const char *src =
                reinterpret_cast<const char *>(part_of<D>(p, k0 + k, k0 + k == first ? 1 : 0));
            const unsigned dst = smem_addr(room) + k * vecs * 16;
#pragma unroll 4
            for (int v = lane; v < vecs; v += 32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * v),
                             "l"(src + 16 * v)
                             : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        {
            // 2 W threads per row: its largest m, then weights exp2(m - m*) in m's place; m* and
            // the sum of l go to `stat`
            const int row = tid / (2 * W), j = tid % (2 * W);
            float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
            for (int k = j; k < count; k += 2 * W) top = fmaxf(top, room[k * vecs * 2 + row].x);
#pragma unroll
            for (int x = W; x >= 1; x >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float base = finite_or_zero(top);
#pragma unroll 1
            for (int k = j; k < count; k += 2 * W) {
                float2 &at = room[k * vecs * 2 + row];
                at.x = exp2_ftz(at.x - base);
                sum = fmaf(at.y, at.x, sum);
            }
#pragma unroll
            for (int x = W; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            if (j == 0) stat[row] = make_float2(top, sum);
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h >= halves) break;
            const int row = (lane >> 2) + 8 * h;
            // what the parts before these come to
            const float2 here = stat[row];
            const float top = fmaxf(m[h], here.x), base = finite_or_zero(top);
            const float a = exp2_ftz(m[h] - base), b = exp2_ftz(here.x - base);
            m[h] = top;
            l[h] = fmaf(here.y, b, l[h] * a);
            float2 sum[E];
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < count; ++k) {
                const float2 *part = room + k * vecs * 2;
                const float w = part[row].x;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 o = part[kAttendRows + (h * (D / 8) + warp + e * W) * 32 + lane];
                    sum[e].x = fmaf(o.x, w, sum[e].x);
                    sum[e].y = fmaf(o.y, w, sum[e].y);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                mine[h][e].x = fmaf(sum[e].x, b, mine[h][e].x * a);
                mine[h][e].y = fmaf(sum[e].y, b, mine[h][e].y * a);
            }
        }
    }
    write_rows<D>(p, u.b, u.unit, mine, l, warp, lane);
}

template <int D, bool kIdx64>
__global__ void __launch_bounds__(32 * AttendGeo<D>::kWarps, 1)
    ssu_attend_kernel(AttendParams p) {
    using Geo = AttendGeo<D>;
    constexpr int W = Geo::kWarps, kThreads = 32 * W, S = Geo::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ longlong2 scan[W];
    __shared__ long long found[2];
    __shared__ unsigned joins[2];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *merge = reinterpret_cast<float *>(smem + Geo::kRingBytes);
    float *stat = reinterpret_cast<float *>(smem + Geo::kRingBytes + Geo::kMergeBytes);
    const unsigned ring = smem_addr(smem) + warp * (S * Geo::kStageBytes);

    // The line's length for one unit of each request, then this CTA's stretch and the request that
    // holds its first place.  A scan of the first kThreads requests gives both at once; the sums
    // of 32 threads' places fit 32 bits (a request has at most 2^31 / kTile).
    const int units = p.kv_heads * p.head_tiles;
    auto places_of = [&](long long b) -> unsigned {
        if (b >= p.requests) return 0;
        bool good;
        const int count = visible_of<kIdx64>(p, b, good).count;
        return count ? (count + Geo::kTile - 1) / Geo::kTile + kUnitCost : 0;
    };
    auto warp_scan = [&](unsigned n) {  // inclusive
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, n, x);
            if (lane >= x) n += o;
        }
        return n;
    };
    const unsigned n0 = places_of(tid), incl0 = warp_scan(n0);
    bool empty = sees_to(tid, p.requests, n0, blockIdx.x, gridDim.x);
    long long rest = 0;
#pragma unroll 1
    for (long long b0 = kThreads; b0 < p.requests; b0 += kThreads) {
        const unsigned n = places_of(b0 + tid);
        rest += n;
        empty |= sees_to(b0 + tid, p.requests, n, blockIdx.x, gridDim.x);
    }
    if (p.requests > kThreads) {
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, x);
    }
    if (lane == 31) scan[warp] = longlong2{incl0, rest};
    const bool any_empty = __syncthreads_or(empty);
    // places up to and with request tid; of the first kThreads; of all
    long long to = incl0, before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const longlong2 v = scan[w];
        if (w < warp) to += v.x;
        before += v.x;
        total += v.x + v.y;
    }
    const long long all = total * units;
    const long long each = (all + gridDim.x - 1) / gridDim.x;
    const long long begin = blockIdx.x * each;
    const long long end = begin + each < all ? begin + each : all;
    if (begin < end) {
        auto look = [&](long long b, unsigned n, long long to) {
            if (n > 0 && begin >= (to - n) * units && begin < to * units) {
                found[0] = b;
                found[1] = (to - n) * units;
            }
        };
        look(tid, n0, to);
#pragma unroll 1
        for (long long b0 = kThreads; begin >= before * units; b0 += kThreads) {
            const unsigned n = places_of(b0 + tid), incl = warp_scan(n);
            __syncthreads();
            if (lane == 31) scan[warp].x = incl;
            __syncthreads();
            to = before + incl;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w < warp) to += scan[w].x;
                before += scan[w].x;
            }
            look(b0 + tid, n, to);
        }
        __syncthreads();

        Cursor at;
        at.b = found[0];
        enter_request<D, kIdx64>(p, at);
        at.unit = static_cast<int>((begin - found[1]) / (at.tiles + kUnitCost));
        at.tile = static_cast<int>((begin - found[1]) -
                                   static_cast<long long>(at.unit) * (at.tiles + kUnitCost));
        at.at = begin;
        if (at.tile >= at.tiles) {  // on a unit's empty places: to the next unit
            at.at += at.tiles + kUnitCost - 1 - at.tile - kUnitCost;
            at.tile = at.tiles - 1;
            advance<D, kIdx64>(p, at);
        }

        // `ahead` is the place of the next step to start, `next` the lane's key of it, and `live`
        // says of each of the `flying` steps in flight which of its keys exist.  The first S - 1
        // turns only fill the ring.
        Cursor ahead = at;
        int fill = 0, use = 0;  // stages: of the next step to start, of the next to compute
        int flying = 0, turn = 1 - S;
        unsigned live[S - 1] = {};
        KeyPlace<kIdx64> next{0, -1, false};
        Sums<D> sums;
        unsigned q[D / 16][4];
        clear<D>(sums);
        if (at.at < end) {
            next = place_of<D, kIdx64>(p, ahead, warp, lane);
            load_queries<D>(p, at, q, lane);
        }
        long long unit_begin = at.at - at.tile;  // place of the unit's first tile in the line
        Partial partial[2] = {};  // by slot
#pragma unroll 1
        while (at.at < end) {
            unsigned keys = 0;
            if (turn >= 0) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
                __syncwarp();
                keys = live[0];
#pragma unroll
                for (int k = 0; k + 1 < S - 1; ++k) live[k] = live[k + 1];
                --flying;
            }
            if (ahead.at < end) {  // into the stage that the step before this one has left
                const unsigned bits =
                    start_step<D, kIdx64>(p, ahead, next, ring + fill * Geo::kStageBytes, lane);
#pragma unroll
                for (int k = 0; k < S - 1; ++k)
                    if (k == flying) live[k] = bits;
                ++flying;
                fill = fill + 1 == S ? 0 : fill + 1;
                advance<D, kIdx64>(p, ahead);
                if (ahead.at < end) next = place_of<D, kIdx64>(p, ahead, warp, lane);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++turn <= 0) continue;
            if (keys) step<D>(p, sums, q, ring + use * Geo::kStageBytes, keys, lane);
            __syncwarp();
            use = use + 1 == S ? 0 : use + 1;
            const Partial u{at.b, unit_begin, at.unit, at.tiles};
            const bool unit_done = at.tile + 1 == at.tiles;
            advance<D, kIdx64>(p, at);
            if (unit_done || at.at >= end) {
                if (at.at < end) {  // the next unit's queries arrive while this one's sums join
                    unit_begin = at.at;
                    load_queries<D>(p, at, q, lane);
                }
                Owned<D> mine;
                float m[2], l[2];
                merge_warps<D>(sums, merge, stat, rows_of(p, u.unit), warp, lane, mine, m, l);
                const bool from_start = u.begin >= begin;
                if (unit_done && from_start) {
                    write_rows<D>(p, u.b, u.unit, mine, l, warp, lane);
                } else {
                    write_part<D>(p, u.unit, from_start, mine, m, l, warp, lane);
                    partial[from_start] = u;
                }
                clear<D>(sums);
                __syncthreads();  // merge and stat are free again
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");

        // Parts are announced once, when the CTA's stretch is done (an announcement waits for the
        // part to be visible; as one atomic that releases and acquires it takes 0.3 to 1.4 us less
        // of a call than between two fences); a unit's counter is that of the CTA where it begins,
        // as only one unit runs on past a stretch's end.  The last to announce joins.
        if (partial[0].tiles || partial[1].tiles) {
            __syncthreads();
            if (tid < 2) {
                unsigned join = 0;
                if (partial[tid].tiles) {
                    const long long first = partial[tid].begin / each;
                    const long long last = (partial[tid].begin + partial[tid].tiles - 1) / each;
                    // after the CTA's part (which the barrier orders before this), before the
                    // others' parts are read
                    unsigned before;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(p.arrived + first)
                                 : "memory");
                    join = before == static_cast<unsigned>(last - first);
                    if (join) p.arrived[first] = 0;  // as the next call wants it
                }
                joins[tid] = join;
            }
            __syncthreads();
#pragma unroll
            for (int slot = 0; slot < 2; ++slot)
                if (joins[slot])
                    join_parts<D>(p, partial[slot],
                                  static_cast<int>(partial[slot].begin / each),
                                  static_cast<int>((partial[slot].begin + partial[slot].tiles - 1) /
                                                   each),
                                  reinterpret_cast<float2 *>(smem),
                                  reinterpret_cast<float2 *>(stat), warp, lane);
        }
    }

    // Requests without visible keys: zeros; invalid lengths: counted.
    for (long long b = blockIdx.x; any_empty && b < p.requests; b += gridDim.x) {
        bool good;
        if (visible_of<kIdx64>(p, b, good).count) continue;
        if (!good) {
            if (tid == 0) {
                atomicAdd(&p.err[0], 1u);
                atomicMin(&p.err[1], static_cast<unsigned>(b));
            }
            continue;
        }
        for (int i = tid; i < p.q_heads * (D / 8); i += kThreads)
            reinterpret_cast<uint4 *>(p.out + b * p.o_b + (i / (D / 8)) * p.o_h)[i % (D / 8)] =
                make_uint4(0, 0, 0, 0);
    }
}

}  // namespace
