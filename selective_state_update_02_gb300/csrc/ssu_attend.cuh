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
// Inside a CTA every warp takes 16 of a tile's keys into its own ring of stages with cp.async
// (16-byte pieces, swizzled for ldmatrix), ahead of its use across unit borders, and keeps its
// own m, l, o: no barrier until a unit ends.

#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

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
    int share;       // query heads per key head
    int head_tiles;  // ceil(share / 16)
    float scale_log2;  // scale * log2 e: weights are exp2 of differences
    unsigned *err;
    unsigned *arrived;  // one counter per CTA; zero between calls
    float *parts;       // two parts per CTA
};

constexpr int kAttendRows = 16;     // query heads per unit: the MMA's M
constexpr int kAttendKeys = 16;     // keys per warp and step: the second product's K

template <int D>
struct AttendGeo {
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kTile = kWarps * kAttendKeys;
    static constexpr int kStageBytes = 2 * kAttendKeys * D * 2;  // K and V of a warp's 16 keys
    static constexpr int kStages = D == 64 ? 5 : 3;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = (kWarps / 2) * kAttendRows * D * 4;
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

// A place in the line of tiles.
struct Cursor {
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

// Moves to the next tile; callers do not move past the last tile of the line.
template <int D, bool kIdx64>
__device__ __forceinline__ void advance(const AttendParams &p, Cursor &c) {
    if (++c.tile < c.tiles) return;
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

// Where the lane's key of a step lies (lanes 16 .. 31 repeat lanes 0 .. 15): its page (-1: no
// such key) and row.
struct KeyPlace {
    int page, row;
};

// The lane's key of the warp's step at cursor `c`; a bad page id counts once, at the page's
// first visible position, for the request's first unit.
template <int D, bool kIdx64>
__device__ __forceinline__ KeyPlace place_of(const AttendParams &p, const Cursor &c, int warp,
                                             int lane) {
    const int i = c.tile * AttendGeo<D>::kTile + warp * kAttendKeys + (lane & 15);
    KeyPlace at{-1, 0};
    if (i >= c.vis.count) return at;
    const int j = i < c.vis.head ? i : i - c.vis.head + c.vis.from;
    const int col = j / p.page_size;
    at.row = j - col * p.page_size;
    const long long page = load_index<kIdx64>(p.table, c.b * p.t_b + col * p.t_p);
    if (page >= 0 && page < p.num_pages) {
        at.page = static_cast<int>(page);
    } else if (c.unit == 0 && lane < 16) {
        // first visible position of its page: the page's start, or the window's start where
        // the sinks leave the page's earlier positions out
        const bool first = at.row == 0 || (j == c.vis.from && c.vis.head <= j - at.row);
        if (first) {
            atomicAdd(&p.err[0], 1u);
            atomicMin(&p.err[1], static_cast<unsigned>(c.b));
        }
    }
    return at;
}

// Starts the copies of the warp's 16 keys and values of one step into `stage`; places without a
// key are zero-filled.
template <int D>
__device__ __forceinline__ void start_step(const AttendParams &p, const Cursor &c,
                                           const KeyPlace &at, unsigned stage, int lane) {
    constexpr int kPieces = D / 8;               // 16-byte pieces per key
    constexpr int kRowsPer = 32 / kPieces > 0 ? 32 / kPieces : 1;  // keys per warp instruction
    const int kh = c.unit / p.head_tiles;
    const __nv_bfloat16 *k0 = p.k + kh * p.k_h, *v0 = p.v + kh * p.v_h;
#pragma unroll
    for (int i = 0; i < kAttendKeys / kRowsPer; ++i) {
        const int key = i * kRowsPer + lane / kPieces, piece = lane % kPieces;
        const int page = __shfl_sync(0xffffffffu, at.page, key);
        const int row = __shfl_sync(0xffffffffu, at.row, key);
        const bool live = page >= 0;
        const long long pg = live ? page : 0;
        const __nv_bfloat16 *ks = k0 + pg * p.k_p + row * p.k_r + piece * 8;
        const __nv_bfloat16 *vs = v0 + pg * p.v_p + row * p.v_r + piece * 8;
        const unsigned dst = stage + key * (D * 2) + ((piece ^ (key & 7)) << 4);
        const int bytes = live ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                     "l"(live ? ks : p.q), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + kAttendKeys * D * 2),
                     "l"(live ? vs : p.q), "r"(bytes)
                     : "memory");
    }
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

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// One step: 16 keys of `stage` (of which those with a bit in `live` exist) into the sums.
template <int D>
__device__ __forceinline__ void step(const AttendParams &p, Sums<D> &s,
                                     const unsigned (&q)[D / 16][4], unsigned stage,
                                     unsigned live, int lane) {
    float sc[2][4] = {};
    const int mi = lane >> 3, r = lane & 7;
    {
        const int key = (mi >> 1) * 8 + r;
        const unsigned base = stage + key * (D * 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            unsigned b[4];
            ldmatrix4(b, base + (((2 * ks + (mi & 1)) ^ (key & 7)) << 4));
            mma_bf16(sc[0], q[ks], b[0], b[1]);
            mma_bf16(sc[1], q[ks], b[2], b[3]);
        }
    }
    const int t = lane & 3;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool seen = (live >> (8 * n + 2 * t + (i & 1))) & 1u;
            sc[n][i] = seen ? sc[n][i] * p.scale_log2 : -INFINITY;
            top[i >> 1] = fmaxf(top[i >> 1], sc[n][i]);
        }
    float keep[2], base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const float m = fmaxf(s.m[h], top[h]);
        base[h] = finite_or_zero(m);
        keep[h] = exp2f(s.m[h] - base[h]);
        s.m[h] = m;
    }
    unsigned w[4];
    float add[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = exp2f(sc[n][2 * h] - base[h]), b = exp2f(sc[n][2 * h + 1] - base[h]);
            add[h] += a + b;
            w[2 * n + h] = f2_to_bf2(a, b);
        }
    s.l[0] = s.l[0] * keep[0] + add[0];
    s.l[1] = s.l[1] * keep[1] + add[1];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        s.o[n][0] *= keep[0], s.o[n][1] *= keep[0];
        s.o[n][2] *= keep[1], s.o[n][3] *= keep[1];
    }
    const int key = (mi & 1) * 8 + r;
    const unsigned vbase = stage + kAttendKeys * D * 2 + key * (D * 2);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        unsigned b[4];
        ldmatrix4_trans(b, vbase + (((2 * j + (mi >> 1)) ^ (key & 7)) << 4));
        mma_bf16(s.o[2 * j], w, b[0], b[1]);
        mma_bf16(s.o[2 * j + 1], w, b[2], b[3]);
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

// Column of element i of a lane's accumulators; its row is lane / 4 + 8 (i / 2 % 2).
__device__ __forceinline__ int col_of(int i, int lane) {
    return (i >> 2) * 8 + 2 * (lane & 3) + (i & 1);
}

// After merge_warps: the one row of all pairs of a thread (pair k has row half k % 2, and k is
// the warp's number modulo an even number of warps).
__device__ __forceinline__ int thread_row(int warp, int lane) {
    return (lane >> 2) + 8 * (warp & 1);
}

// Joins the warps' sums of a unit: every warp's o scaled to the unit's m, then added pairwise
// (upper half of the warps to the lower) and over the rest by all threads, always in the same
// order.  m and l are the unit's for the lane's rows lane / 4 and lane / 4 + 8; `mine` are the
// sums of the element pairs that the thread owns: pair e is accumulator elements 2 k, 2 k + 1
// of its lane with k = warp + e * kWarps.
template <int D>
__device__ __forceinline__ void merge_warps(Sums<D> &s, float *merge, float *stat, int warp,
                                            int lane, float2 (&mine)[D / 4 / AttendGeo<D>::kWarps],
                                            float (&m)[2], float (&l)[2]) {
    constexpr int W = AttendGeo<D>::kWarps;
    const int g = lane >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 1);
        s.l[h] += __shfl_xor_sync(0xffffffffu, s.l[h], 2);
        if ((lane & 3) == 0) {
            stat[(warp * kAttendRows + g + 8 * h) * 2] = s.m[h];
            stat[(warp * kAttendRows + g + 8 * h) * 2 + 1] = s.l[h];
        }
    }
    __syncthreads();
    float own[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        m[h] = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w)
            m[h] = fmaxf(m[h], stat[(w * kAttendRows + g + 8 * h) * 2]);
        const float base = finite_or_zero(m[h]);
        l[h] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            l[h] = fmaf(stat[(w * kAttendRows + g + 8 * h) * 2 + 1],
                        exp2f(stat[(w * kAttendRows + g + 8 * h) * 2] - base), l[h]);
        own[h] = exp2f(s.m[h] - base);
    }
    float2 *buf = reinterpret_cast<float2 *>(merge);  // [W / 2][D / 4 pairs][32 lanes]
    constexpr int kPairs = D / 4;
    if (warp >= W / 2) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            float2 *at = buf + ((warp - W / 2) * kPairs + 2 * n) * 32 + lane;
            at[0] = make_float2(s.o[n][0] * own[0], s.o[n][1] * own[0]);
            at[32] = make_float2(s.o[n][2] * own[1], s.o[n][3] * own[1]);
        }
    }
    __syncthreads();
    if (warp < W / 2) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            float2 *at = buf + (warp * kPairs + 2 * n) * 32 + lane;
            const float2 a = at[0], b = at[32];
            at[0] = make_float2(fmaf(s.o[n][0], own[0], a.x), fmaf(s.o[n][1], own[0], a.y));
            at[32] = make_float2(fmaf(s.o[n][2], own[1], b.x), fmaf(s.o[n][3], own[1], b.y));
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kPairs / W; ++e) {
        const int k = warp + e * W;
        float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W / 2; ++w) {
            const float2 a = buf[(w * kPairs + k) * 32 + lane];
            t.x += a.x, t.y += a.y;
        }
        mine[e] = t;
    }
}

// The unit's output rows from the threads' sums.
template <int D>
__device__ __forceinline__ void write_rows(const AttendParams &p, long long b, int unit,
                                           const float2 (&mine)[D / 4 / AttendGeo<D>::kWarps],
                                           float l, int warp, int lane) {
    constexpr int W = AttendGeo<D>::kWarps;
    const int kh = unit / p.head_tiles, first = (unit - kh * p.head_tiles) * kAttendRows;
    const int row = thread_row(warp, lane);
    if (first + row >= p.share) return;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;  // no visible key (l = 0): zeros
    __nv_bfloat16 *dst = p.out + b * p.o_b + (kh * p.share + first + row) * p.o_h;
#pragma unroll
    for (int e = 0; e < D / 4 / W; ++e)
        *reinterpret_cast<unsigned *>(dst + col_of(2 * (warp + e * W), lane)) =
            f2_to_bf2(mine[e].x * f, mine[e].y * f);
}

// Writes this CTA's part of a unit that its stretch does not hold whole, and, in the CTA that
// arrives last, joins all parts in their order and writes the unit's rows.  A part is two slots
// per CTA: slot 1 for the unit that begins in the CTA's stretch, slot 0 for the one that began
// before it; the unit's counter is that of the CTA where it begins (only one such unit runs on
// past a stretch's end).
template <int D>
__device__ __forceinline__ void join_parts(const AttendParams &p, const Cursor &at,
                                           long long unit_begin, long long each, bool from_start,
                                           float2 (&mine)[D / 4 / AttendGeo<D>::kWarps],
                                           const float (&m)[2], const float (&l)[2],
                                           unsigned *last_flag, int warp, int lane) {
    using Geo = AttendGeo<D>;
    constexpr int W = Geo::kWarps, E = D / 4 / W, F = Geo::kPartFloats;
    const int first = static_cast<int>(unit_begin / each);
    const int last = static_cast<int>((unit_begin + at.tiles - 1) / each);
    const int row = thread_row(warp, lane), h = warp & 1;
    const int kh = at.unit / p.head_tiles;
    const bool used = (at.unit - kh * p.head_tiles) * kAttendRows + row < p.share;
    float *slot = p.parts + (2ll * blockIdx.x + (from_start ? 1 : 0)) * F;
    if (used) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            __stcg(reinterpret_cast<float2 *>(slot) + (warp + e * W) * 32 + lane, mine[e]);
        if (warp < 2 && (lane & 3) == 0)
            __stcg(reinterpret_cast<float2 *>(slot + kAttendRows * D) + row,
                   make_float2(m[h], l[h]));
    }
    __threadfence();
    __syncthreads();
    if (warp == 0 && lane == 0) {
        const unsigned parts = static_cast<unsigned>(last - first + 1);
        const bool all = atomicAdd(&p.arrived[first], 1u) == parts - 1;
        if (all) p.arrived[first] = 0;  // as the next call wants it
        *last_flag = all;
    }
    __syncthreads();
    if (!*last_flag) return;
    __threadfence();
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) mine[e] = make_float2(0.0f, 0.0f);
    constexpr int kBatch = E >= 8 ? 2 : 4;  // parts whose loads are in flight together
    if (used) {
        for (int c0 = first; c0 <= last; c0 += kBatch) {
            float2 ml[kBatch], o[kBatch][E];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int c = c0 + k <= last ? c0 + k : last;
                const float *src = p.parts + (2ll * c + (c == first ? 1 : 0)) * F;
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(src + kAttendRows * D) + row);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[k][e] = __ldcg(reinterpret_cast<const float2 *>(src) +
                                     (warp + e * W) * 32 + lane);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (c0 + k > last) break;
                const float t = fmaxf(top, ml[k].x), base = finite_or_zero(t);
                const float a = exp2f(top - base), b = exp2f(ml[k].x - base);
                top = t;
                sum = sum * a + ml[k].y * b;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    mine[e].x = mine[e].x * a + o[k][e].x * b;
                    mine[e].y = mine[e].y * a + o[k][e].y * b;
                }
            }
        }
    }
    write_rows<D>(p, at.b, at.unit, mine, sum, warp, lane);
}

template <int D, bool kIdx64>
__global__ void __launch_bounds__(32 * AttendGeo<D>::kWarps, 1)
    ssu_attend_kernel(AttendParams p) {
    using Geo = AttendGeo<D>;
    constexpr int W = Geo::kWarps, kThreads = 32 * W, S = Geo::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long scan[W + 1];
    __shared__ long long found[2];
    __shared__ unsigned last_flag;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *merge = reinterpret_cast<float *>(smem + Geo::kRingBytes);
    float *stat = reinterpret_cast<float *>(smem + Geo::kRingBytes + Geo::kMergeBytes);
    const unsigned ring = smem_addr(smem) + warp * (S * Geo::kStageBytes);

    // Requests without visible keys: zeros; invalid lengths: counted.
    for (long long b = blockIdx.x; b < p.requests; b += gridDim.x) {
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

    // The line's length in tiles of one unit, then this CTA's stretch.
    const int units = p.kv_heads * p.head_tiles;
    long long sum = 0;
    for (long long b = tid; b < p.requests; b += kThreads) {
        bool good;
        sum += (visible_of<kIdx64>(p, b, good).count + Geo::kTile - 1) / Geo::kTile;
    }
    long long total = sum;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) total += scan[w];
    const long long all = total * units;
    const long long each = (all + gridDim.x - 1) / gridDim.x;
    const long long begin = blockIdx.x * each;
    const long long end = begin + each < all ? begin + each : all;
    if (begin >= end) return;

    // The request that holds tile `begin`: its tiles start at units * (tiles before it).
    long long before = 0;
    for (long long b0 = 0; b0 < p.requests; b0 += kThreads) {
        const long long b = b0 + tid;
        long long n = 0;
        if (b < p.requests) {
            bool good;
            n = (visible_of<kIdx64>(p, b, good).count + Geo::kTile - 1) / Geo::kTile;
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
        long long base = before, whole = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) base += scan[w];
            whole += scan[w];
        }
        incl += base;
        if (n > 0 && begin >= (incl - n) * units && begin < incl * units) {
            found[0] = b;
            found[1] = (incl - n) * units;
        }
        before += whole;
        if (begin < before * units) break;
    }
    __syncthreads();

    Cursor at;
    at.b = found[0];
    enter_request<D, kIdx64>(p, at);
    at.unit = static_cast<int>((begin - found[1]) / at.tiles);
    at.tile = static_cast<int>((begin - found[1]) - static_cast<long long>(at.unit) * at.tiles);

    // Fill the ring: steps begin .. begin + S - 2; `ahead` is the place of the next step to
    // start, `next` the lane's key of it, and `live` holds 16 bits for each step in flight: which
    // of its keys exist.
    Cursor ahead = at;
    long long started = begin;
    unsigned long long live = 0;
    KeyPlace next = place_of<D, kIdx64>(p, ahead, warp, lane);
    auto start = [&](long long done) {
        if (started < end) {
            const unsigned long long mask = __ballot_sync(0xffffffffu, next.page >= 0) & 0xffffu;
            live |= mask << (16 * static_cast<int>(started - done));
            start_step<D>(p, ahead, next,
                          ring + static_cast<int>((started - begin) % S) * Geo::kStageBytes,
                          lane);
            if (++started < end) {
                advance<D, kIdx64>(p, ahead);
                next = place_of<D, kIdx64>(p, ahead, warp, lane);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) start(begin);

    Sums<D> sums;
    unsigned q[D / 16][4];
    clear<D>(sums);
    load_queries<D>(p, at, q, lane);
    long long unit_begin = begin - at.tile;  // place of the unit's first tile in the line
    for (long long i = begin; i < end; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        const unsigned keys = static_cast<unsigned>(live) & 0xffffu;
        live >>= 16;
        start(i + 1);  // into the stage that the step before this one has left
        if (keys)
            step<D>(p, sums, q, ring + static_cast<int>((i - begin) % S) * Geo::kStageBytes, keys,
                    lane);
        __syncwarp();
        const bool unit_done = at.tile + 1 == at.tiles;
        if (unit_done || i + 1 == end) {
            float2 mine[D / 4 / W];
            float m[2], l[2];
            merge_warps<D>(sums, merge, stat, warp, lane, mine, m, l);
            const bool from_start = unit_begin >= begin;
            if (unit_done && from_start) {
                write_rows<D>(p, at.b, at.unit, mine, l[warp & 1], warp, lane);
            } else {
                join_parts<D>(p, at, unit_begin, each, from_start, mine, m, l, &last_flag, warp,
                              lane);
            }
            clear<D>(sums);
            __syncthreads();  // merge and stat are free again
        }
        if (i + 1 < end) {
            advance<D, kIdx64>(p, at);
            if (unit_done) {
                unit_begin = i + 1;
                load_queries<D>(p, at, q, lane);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace
