// Norm and rotation of queries and keys and their way into the paged cache (ssu_rotate_qk): one
// pass over q, k and v.
//
// Mathematics.  A head a of D elements becomes u = a / sqrt(mean a^2 + eps) * w, and pairs
// (u_i, u_j) of its first R elements turn by their position's angle.  Everything is fp32 and is
// rounded once, when the head is stored.
//
// What bounds it: HBM, then the issue of instructions.  Every element of q, k and v is read once and
// written once (2 + 2 bytes), at 8192 tokens of 48 heads of 128 in 39.7 us: 5.2 TB/s, 0.78 of the
// measured copy rate, with 0.64 of the issue slots taken (81 us with a head per warp and the norm,
// the weight and the turn one after the other; 47 with four loads in flight; 43 with the
// coefficients below).  Short calls are bound by their launch: 8 tokens take as long as 777.
//
// Layout.  A head is D / 8 lanes with one 16-byte vector each (8, 16 or 32 lanes), so a warp
// instruction moves 512 contiguous bytes of neighbouring heads; the sum of squares is a
// butterfly over the head's lanes, and pairs whose halves lie in different lanes (R a multiple of
// 16, so R / 2 is a whole number of vectors) are four shuffles of two bf16 each.  A warp takes four
// vectors per lane of one token (8 heads of 128), so that a token's table row is read once for
// all of them and four loads per lane are in flight.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ssu.h"
#include "ssu_device.cuh"
#include "ssu_host.h"

using ssu_host::aligned;
using ssu_host::DeviceGuard;
using ssu_host::fail;
using ssu_host::ok;

namespace {

struct RotateParams {
    const __nv_bfloat16 *q, *k, *v;
    const float *q_weight, *k_weight, *table;
    const void *positions, *slots;
    __nv_bfloat16 *q_out, *k_pages, *v_pages;
    long long q_t, k_t, v_t, o_t, kp_p, kp_r, vp_p, vp_r;
    int q_h, k_h, v_h, o_h, kp_h, vp_h;  // head strides
    long long table_r, positions_s, slots_s;
    long long num_positions, num_slots, page_size;
    long long tokens;
    int q_heads, kv_heads, rotary;
    int batches;  // of a warp: kRotateUnroll vector rows each
    int groups;   // warps per token
    float eps;
    unsigned *err;
};

template <bool kIdx64>
__device__ __forceinline__ long long load_index(const void *ids, long long at) {
    if (kIdx64) return __ldg(static_cast<const long long *>(ids) + at);
    return static_cast<long long>(__ldg(static_cast<const int *>(ids) + at));
}

// A turned element is a_i (w_i cos) + a_j (-+ w_j sin), all times the head's 1 / rms: the
// coefficients depend on the token and on whether the head is a query or a key, not on the head,
// so a lane works its 8 pairs out once for all heads of a kind that its warp takes.
struct Turn {
    float2 own[4], other[4];  // of the lane's elements 2 i, 2 i + 1
};

template <bool kInterleaved>
__device__ __forceinline__ void load_turn(Turn &a, const float *weight, const float *row, int l,
                                          int partner, int rotary) {
    const float4 *w4 = reinterpret_cast<const float4 *>(weight);
    const float4 wa = __ldg(w4 + 2 * l), wb = __ldg(w4 + 2 * l + 1);
    const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
    if (8 * l >= rotary) {  // past the rotated elements
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.own[i] = make_float2(w[2 * i], w[2 * i + 1]);
            a.other[i] = make_float2(0.0f, 0.0f);
        }
    } else if (kInterleaved) {  // elements 2 i and 2 i + 1 turn by angle 4 l + i
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row) + l);
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + rotary / 2) + l);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.own[i] = make_float2(w[2 * i] * c[i], w[2 * i + 1] * c[i]);
            a.other[i] = make_float2(-w[2 * i + 1] * s[i], w[2 * i] * s[i]);
        }
    } else {  // the lane's vector turns with its partner's, element by element
        const bool first = l < partner;
        const int at = 2 * (first ? l : partner);
        const float4 *cr = reinterpret_cast<const float4 *>(row) + at;
        const float4 *sr = reinterpret_cast<const float4 *>(row + rotary / 2) + at;
        const float4 pa = __ldg(w4 + 2 * partner), pb = __ldg(w4 + 2 * partner + 1);
        const float4 ca = __ldg(cr), cb = __ldg(cr + 1), sa = __ldg(sr), sb = __ldg(sr + 1);
        const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
        const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
        const float sign = first ? -1.0f : 1.0f;  // a cos - b sin; b cos + a sin
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.own[i] = make_float2(w[2 * i] * c[2 * i], w[2 * i + 1] * c[2 * i + 1]);
            a.other[i] =
                make_float2(sign * p[2 * i] * s[2 * i], sign * p[2 * i + 1] * s[2 * i + 1]);
        }
    }
}

// Norm and rotation of one head spread over LPH lanes, 8 elements each.
template <int LPH, bool kInterleaved>
__device__ __forceinline__ uint4 norm_rotate(const uint4 &raw, const Turn &a, int partner,
                                             float eps) {
    const unsigned u[4] = {raw.x, raw.y, raw.z, raw.w};
    float2 v[4], sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        sq = __ffma2_rn(v[i], v[i], sq);
    }
    float s = sq.x + sq.y;
#pragma unroll
    for (int m = LPH / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    const float r = rsqrtf(s * (1.0f / (8 * LPH)) + eps);
    unsigned o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 t;  // what the elements turn with
        if (kInterleaved) {
            t = make_float2(v[i].y, v[i].x);
        } else {
            const unsigned w = __shfl_sync(0xffffffffu, u[i], partner, LPH);
            t = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
        const float2 y = __fmul2_rn(
            make_float2(r, r), __ffma2_rn(t, a.other[i], __fmul2_rn(v[i], a.own[i])));
        o[i] = f2_to_bf2(y.x, y.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kRotateWarps = 4, kRotateUnroll = 4;

// A warp takes kRotateUnroll * 32 / LPH neighbouring heads of one token (queries, then keys, then
// values): all their loads go out together, and the table row is read once for them.
template <int LPH, bool kInterleaved, bool kIdx64>
__global__ void __launch_bounds__(32 * kRotateWarps, 32 / kRotateWarps)
    ssu_rotate_kernel(RotateParams p) {
    pdl_wait();
    pdl_trigger();
    constexpr int HPW = 32 / LPH, U = kRotateUnroll;  // heads per warp instruction
    const int lane = threadIdx.x & 31, l = lane & (LPH - 1);
    const int heads = p.q_heads + 2 * p.kv_heads;
    const unsigned block = blockIdx.x / p.groups;
    const int group = static_cast<int>(blockIdx.x - block * p.groups);
    const long long t = static_cast<long long>(block) * kRotateWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const long long pos = load_index<kIdx64>(p.positions, t * p.positions_s);
    const long long slot = load_index<kIdx64>(p.slots, t * p.slots_s);
    // The heads' loads do not wait for the position and the slot: they are inside q, k and v
    // whatever those say.
    const __nv_bfloat16 *const q = p.q + t * p.q_t + 8 * l, *const k = p.k + t * p.k_t + 8 * l;
    const __nv_bfloat16 *const v = p.v + t * p.v_t + 8 * l;
    const int end = min(heads, (group + 1) * p.batches * (U * HPW));
    uint4 raw[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * HPW, hk = h - p.q_heads, hv = hk - p.kv_heads;
            const __nv_bfloat16 *const base = hk < 0 ? q : hv < 0 ? k : v;
            const int at = hk < 0 ? h : hv < 0 ? hk : hv;
            const int stride = hk < 0 ? p.q_h : hv < 0 ? p.k_h : p.v_h;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (h < end)
                raw[u] = __ldcs(reinterpret_cast<const uint4 *>(
                    base + static_cast<long long>(at) * stride));
        }
    };
    int h0 = group * p.batches * (U * HPW) + lane / LPH;
    load(h0);
    if (pos < 0 || pos >= p.num_positions || slot < -1 || slot >= p.num_slots) {
        if (group == 0 && lane == 0) {
            atomicAdd(&p.err[0], 1u);
            atomicMin(&p.err[1], static_cast<unsigned>(t));
        }
        return;
    }
    long long page = 0, r = 0;
    if (slot >= 0) {
        // 32 bits where they hold (a 64-bit division is some hundred instructions)
        page = p.num_slots <= INT_MAX ? static_cast<unsigned>(slot) /
                                            static_cast<unsigned>(p.page_size)
                                      : slot / p.page_size;
        r = slot - page * p.page_size;
    }
    const int half = p.rotary / 16;  // vectors per half
    const int partner = kInterleaved || 8 * l >= p.rotary ? l : l < half ? l + half : l - half;
    __nv_bfloat16 *const q_out = p.q_out + t * p.o_t + 8 * l;
    __nv_bfloat16 *const k_out = p.k_pages + page * p.kp_p + r * p.kp_r + 8 * l;
    __nv_bfloat16 *const v_out = p.v_pages + page * p.vp_p + r * p.vp_r + 8 * l;
    const float *row = p.table + pos * p.table_r, *weight = nullptr;
    Turn turn;
#pragma unroll 1
    while (true) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * HPW;
            const bool turns = h < p.q_heads + p.kv_heads;
            if (__any_sync(0xffffffffu, turns)) {
                const float *w = h < p.q_heads ? p.q_weight : p.k_weight;
                if (__any_sync(0xffffffffu, w != weight)) {
                    load_turn<kInterleaved>(turn, w, row, l, partner, p.rotary);
                    weight = w;
                }
                const uint4 v = norm_rotate<LPH, kInterleaved>(raw[u], turn, partner, p.eps);
                if (turns) raw[u] = v;
            }
            const int hk = h - p.q_heads, hv = hk - p.kv_heads;
            __nv_bfloat16 *const base = hk < 0 ? q_out : hv < 0 ? k_out : v_out;
            const int at = hk < 0 ? h : hv < 0 ? hk : hv;
            const int stride = hk < 0 ? p.o_h : hv < 0 ? p.kp_h : p.vp_h;
            if (h < end && (hk < 0 || slot >= 0))
                *reinterpret_cast<uint4 *>(base + static_cast<long long>(at) * stride) = raw[u];
        }
        h0 += U * HPW;
        if (h0 - lane / LPH >= end) return;
        load(h0);
    }
}

template <int LPH>
cudaError_t launch_rotate(RotateParams p, bool interleaved, bool i64, int sm_count, bool pdl,
                          cudaStream_t st) {
    // A warp's fixed work (its token's place, addresses and coefficients) is that of one to two
    // batches, so warps take as many as leave some 32 warps per SM: 8192 tokens of 48 heads of 128
    // 43.2 us with one batch, 39.7 with all six; at few tokens one.
    constexpr int kHeads = kRotateUnroll * (32 / LPH);  // per batch
    const long long most = (p.q_heads + 2 * p.kv_heads + kHeads - 1) / kHeads;
    const long long fair = p.tokens * most / (32ll * sm_count);
    p.batches = static_cast<int>(fair < 1 ? 1 : fair < most ? fair : most);
    p.groups = static_cast<int>((most + p.batches - 1) / p.batches);
    p.batches = static_cast<int>((most + p.groups - 1) / p.groups);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.tokens + kRotateWarps - 1) / kRotateWarps *
                                             p.groups));
    cfg.blockDim = dim3(32 * kRotateWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (interleaved)
        return i64 ? cudaLaunchKernelEx(&cfg, ssu_rotate_kernel<LPH, true, true>, p)
                   : cudaLaunchKernelEx(&cfg, ssu_rotate_kernel<LPH, true, false>, p);
    return i64 ? cudaLaunchKernelEx(&cfg, ssu_rotate_kernel<LPH, false, true>, p)
               : cudaLaunchKernelEx(&cfg, ssu_rotate_kernel<LPH, false, false>, p);
}

}  // namespace

extern "C" ssu_status_t ssu_rotate_qk(ssu_handle_t handle, const uint16_t *q, const uint16_t *k,
                                      const uint16_t *v, const float *q_weight,
                                      const float *k_weight, const float *table,
                                      const void *positions, uint16_t *q_out, uint16_t *k_pages,
                                      uint16_t *v_pages, const void *slots,
                                      const ssu_rotate_shape_t *shape,
                                      const ssu_rotate_strides_t *strides, float eps,
                                      ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    if (!shape || !strides)
        return fail(SSU_ERR_INVALID_ARG, "shape and strides must not be NULL");
    const ssu_rotate_shape_t &s = *shape;
    const ssu_rotate_strides_t &u = *strides;
    if (s.tokens < 0 || s.num_positions < 0 || s.num_pages < 0)
        return fail(SSU_ERR_INVALID_ARG, "tokens, num_positions and num_pages must be >= 0");
    if (s.q_heads < 1 || s.kv_heads < 1 || s.page_size < 1)
        return fail(SSU_ERR_INVALID_ARG, "q_heads, kv_heads and page_size must be >= 1");
    if (s.index_dtype != SSU_INDEX_I32 && s.index_dtype != SSU_INDEX_I64)
        return fail(SSU_ERR_INVALID_ARG, "index_dtype %d is neither I32 nor I64", s.index_dtype);
    if (s.headdim != 64 && s.headdim != 128 && s.headdim != 256)
        return fail(SSU_ERR_UNSUPPORTED, "headdim %lld: this build implements 64, 128 and 256",
                    (long long)s.headdim);
    if (s.rotary < 0 || s.rotary > s.headdim || s.rotary % 16 != 0)
        return fail(SSU_ERR_UNSUPPORTED, "rotary %lld is not a multiple of 16 in 0..headdim",
                    (long long)s.rotary);
    if (s.q_heads > 65535 || s.kv_heads > 65535)
        return fail(SSU_ERR_UNSUPPORTED, "q_heads and kv_heads are limited to 65535");
    if (s.num_pages > 0 && s.page_size > LLONG_MAX / s.num_pages)
        return fail(SSU_ERR_UNSUPPORTED, "num_pages * page_size exceeds 2^63");
    if (!(eps >= 0.0f)) return fail(SSU_ERR_INVALID_ARG, "eps must be >= 0");
    if (s.tokens == 0) return ok();
    const int64_t vec[] = {u.q[0], u.q[1], u.k[0], u.k[1], u.v[0], u.v[1], u.q_out[0], u.q_out[1],
                           u.k_pages[0], u.k_pages[1], u.k_pages[2], u.v_pages[0], u.v_pages[1],
                           u.v_pages[2]};
    for (int64_t x : vec) {
        if (x < 0) return fail(SSU_ERR_INVALID_ARG, "negative stride");
        if (x % 8) return fail(SSU_ERR_MISALIGNED, "a stride of %lld elements is not a multiple "
                               "of 16 bytes", (long long)x);
    }
    if (u.table < 0 || u.positions < 0 || u.slots < 0)
        return fail(SSU_ERR_INVALID_ARG, "negative stride");
    if (s.rotary && u.table % 4)
        return fail(SSU_ERR_MISALIGNED, "the table stride is not a multiple of 4");
    if (!q || !k || !v || !q_weight || !k_weight || !positions || !q_out || !slots ||
        (s.rotary && s.num_positions && !table) || (s.num_pages && (!k_pages || !v_pages)))
        return fail(SSU_ERR_INVALID_ARG, "a data pointer is NULL");
    const void *a16[] = {q, k, v, q_weight, k_weight, s.rotary ? table : nullptr, q_out,
                         k_pages, v_pages};
    for (const void *ptr : a16)
        if (!aligned(ptr, 16)) return fail(SSU_ERR_MISALIGNED, "an operand is not 16-byte aligned");
    const unsigned isz = s.index_dtype == SSU_INDEX_I64 ? 8 : 4;
    if (!aligned(positions, isz) || !aligned(slots, isz))
        return fail(SSU_ERR_MISALIGNED, "positions or slots are not aligned to their type");
    if (s.tokens > INT_MAX / (s.q_heads + 2 * s.kv_heads))
        return fail(SSU_ERR_UNSUPPORTED, "tokens * heads exceeds 2^31");

    RotateParams p;
    auto bf = [](const uint16_t *t) { return reinterpret_cast<const __nv_bfloat16 *>(t); };
    auto bfw = [](uint16_t *t) { return reinterpret_cast<__nv_bfloat16 *>(t); };
    p.q = bf(q), p.k = bf(k), p.v = bf(v);
    p.q_weight = q_weight, p.k_weight = k_weight, p.table = table;
    p.positions = positions, p.slots = slots;
    p.q_out = bfw(q_out), p.k_pages = bfw(k_pages), p.v_pages = bfw(v_pages);
    p.q_t = u.q[0], p.k_t = u.k[0], p.v_t = u.v[0], p.o_t = u.q_out[0];
    p.kp_p = u.k_pages[0], p.kp_r = u.k_pages[1], p.vp_p = u.v_pages[0], p.vp_r = u.v_pages[1];
    const int64_t head[] = {u.q[1], u.k[1], u.v[1], u.q_out[1], u.k_pages[2], u.v_pages[2]};
    int *const to[] = {&p.q_h, &p.k_h, &p.v_h, &p.o_h, &p.kp_h, &p.vp_h};
    for (int i = 0; i < 6; ++i) {
        if (head[i] > INT_MAX)
            return fail(SSU_ERR_UNSUPPORTED, "head strides are limited to 2^31 - 1 elements");
        *to[i] = static_cast<int>(head[i]);
    }
    p.table_r = u.table, p.positions_s = u.positions, p.slots_s = u.slots;
    p.num_positions = s.num_positions, p.num_slots = s.num_pages * s.page_size;
    p.page_size = s.page_size;
    p.tokens = s.tokens;
    p.q_heads = static_cast<int>(s.q_heads), p.kv_heads = static_cast<int>(s.kv_heads);
    p.rotary = static_cast<int>(s.rotary);
    p.eps = eps;
    p.err = handle->err;

    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool i64 = s.index_dtype == SSU_INDEX_I64, inter = s.interleaved != 0;
    const int sms = handle->sm_count;
    const cudaError_t e = s.headdim == 64    ? launch_rotate<8>(p, inter, i64, sms, handle->pdl, cs)
                          : s.headdim == 128 ? launch_rotate<16>(p, inter, i64, sms, handle->pdl, cs)
                                             : launch_rotate<32>(p, inter, i64, sms, handle->pdl, cs);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}
