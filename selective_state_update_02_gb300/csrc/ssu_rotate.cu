// Norm and rotation of queries and keys and their way into the paged cache (ssu_rotate_qk): one
// pass over q, k and v.
//
// Mathematics.  A head a of D elements becomes u = a / sqrt(mean a^2 + eps) * w, and pairs
// (u_i, u_j) of its first R elements turn by their position's angle.  Everything is fp32 and is
// rounded once, when the head is stored.
//
// What bounds it: HBM.  Every element of q, k and v is read once and written once (2 + 2 bytes);
// the arithmetic is a handful of instructions per element, and the table rows (R fp32 per token)
// are shared by all heads of a token through L1 and L2.
//
// Layout.  A head is D / 8 lanes with one 16-byte vector each (8, 16 or 32 lanes), so a warp
// instruction moves 512 contiguous bytes of neighbouring heads; the sum of squares is a
// butterfly over the head's lanes, and a pair whose halves lie in different lanes (R a multiple
// of 16, so R / 2 is a whole number of vectors) is one shuffle per element.

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
    long long q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    long long kp_p, kp_r, kp_h, vp_p, vp_r, vp_h;
    long long table_r, positions_s, slots_s;
    long long num_positions, num_slots, page_size;
    long long tokens;
    int q_heads, kv_heads, rotary;
    float eps;
    unsigned *err;
};

template <bool kIdx64>
__device__ __forceinline__ long long load_index(const void *ids, long long at) {
    if (kIdx64) return __ldg(static_cast<const long long *>(ids) + at);
    return static_cast<long long>(__ldg(static_cast<const int *>(ids) + at));
}

__device__ __forceinline__ void widen8(const uint4 &w, float (&v)[8]) {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
    return make_uint4(f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3]), f2_to_bf2(v[4], v[5]),
                      f2_to_bf2(v[6], v[7]));
}

// Norm and rotation of one head spread over LPH lanes, 8 elements each (lane `l` of the head
// holds elements 8 l ..).  `row` is the token's table row.
template <int LPH, bool kInterleaved>
__device__ __forceinline__ void norm_rotate(float (&v)[8], const float *weight, const float *row,
                                            int l, int rotary, float eps) {
    constexpr int D = 8 * LPH;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
#pragma unroll
    for (int m = LPH / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    const float r = rsqrtf(s * (1.0f / D) + eps);
    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(weight) + 2 * l);
    const float4 w1 = __ldg(reinterpret_cast<const float4 *>(weight) + 2 * l + 1);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
    if (kInterleaved) {
        if (8 * l < rotary) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row) + l);
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + rotary / 2) + l);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * c[i] - b * sn[i];
                v[2 * i + 1] = b * c[i] + a * sn[i];
            }
        }
    } else {
        // Element 8 l + i pairs with the same element of the vector `half` lanes up or down.
        const int half = rotary / 16;
        const bool first = l < half, turns = l < 2 * half;
        const int partner = first ? l + half : turns ? l - half : l;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, v[i], partner, LPH);
        if (turns) {
            const int m = first ? l : l - half;
            const float4 *cr = reinterpret_cast<const float4 *>(row) + 2 * m;
            const float4 *sr = reinterpret_cast<const float4 *>(row + rotary / 2) + 2 * m;
            const float4 ca = __ldg(cr), cb = __ldg(cr + 1), sa = __ldg(sr), sb = __ldg(sr + 1);
            const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
            const float sn[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // first half: a cos - b sin; second half: b cos + a sin
                const float t = first ? -o[i] : o[i];
                v[i] = fmaf(t, sn[i], v[i] * c[i]);
            }
        }
    }
}

// One head of one token per LPH lanes: heads 0 .. q_heads - 1 are queries, then keys, then
// values.
template <int LPH, bool kInterleaved, bool kIdx64>
__global__ void __launch_bounds__(256) ssu_rotate_kernel(RotateParams p) {
    pdl_wait();
    constexpr int HPW = 32 / LPH;  // heads per warp
    const int lane = threadIdx.x & 31, l = lane & (LPH - 1);
    const int heads = p.q_heads + 2 * p.kv_heads;
    const long long items = p.tokens * heads;
    const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) +
                           (threadIdx.x >> 5);
    const long long item = warp * HPW + lane / LPH;
    const bool live = item < items;
    const long long t = live ? item / heads : 0;
    const int h = live ? static_cast<int>(item - t * heads) : 0;
    const long long pos = load_index<kIdx64>(p.positions, t * p.positions_s);
    const long long slot = load_index<kIdx64>(p.slots, t * p.slots_s);
    const bool good = pos >= 0 && pos < p.num_positions && slot >= -1 && slot < p.num_slots;
    if (live && !good && h == 0 && l == 0) {
        atomicAdd(&p.err[0], 1u);
        atomicMin(&p.err[1], static_cast<unsigned>(t));
    }
    const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
    const int kh = h - p.q_heads - (is_k ? 0 : p.kv_heads);
    const __nv_bfloat16 *src = is_q   ? p.q + t * p.q_t + h * p.q_h
                               : is_k ? p.k + t * p.k_t + kh * p.k_h
                                      : p.v + t * p.v_t + kh * p.v_h;
    const bool stores = live && good && (is_q || slot >= 0);
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (stores) raw = __ldcs(reinterpret_cast<const uint4 *>(src) + l);
    if (is_q || is_k || LPH < 32) {  // uniform over the warp where a head is a whole warp
        float v[8];
        widen8(raw, v);
        norm_rotate<LPH, kInterleaved>(v, is_q ? p.q_weight : p.k_weight,
                                       p.table + (stores ? pos : 0) * p.table_r, l, p.rotary,
                                       p.eps);
        if (is_q || is_k) raw = narrow8(v);
    }
    if (!stores) return;
    __nv_bfloat16 *dst;
    if (is_q) {
        dst = p.q_out + t * p.o_t + h * p.o_h;
    } else {
        const long long page = slot / p.page_size, r = slot - page * p.page_size;
        dst = is_k ? p.k_pages + page * p.kp_p + r * p.kp_r + kh * p.kp_h
                   : p.v_pages + page * p.vp_p + r * p.vp_r + kh * p.vp_h;
    }
    reinterpret_cast<uint4 *>(dst)[l] = raw;
}

template <int LPH>
cudaError_t launch_rotate(const RotateParams &p, bool interleaved, bool i64, bool pdl,
                          cudaStream_t st) {
    constexpr int kWarps = 8, HPW = 32 / LPH;
    const long long items = p.tokens * (p.q_heads + 2 * p.kv_heads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((items + kWarps * HPW - 1) / (kWarps * HPW)));
    cfg.blockDim = dim3(32 * kWarps);
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
    if (s.rotary && u.table % 4) return fail(SSU_ERR_MISALIGNED, "the table stride is not a multiple of 4");
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
    p.q_t = u.q[0], p.q_h = u.q[1], p.k_t = u.k[0], p.k_h = u.k[1];
    p.v_t = u.v[0], p.v_h = u.v[1], p.o_t = u.q_out[0], p.o_h = u.q_out[1];
    p.kp_p = u.k_pages[0], p.kp_r = u.k_pages[1], p.kp_h = u.k_pages[2];
    p.vp_p = u.v_pages[0], p.vp_r = u.v_pages[1], p.vp_h = u.v_pages[2];
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
    const cudaError_t e = s.headdim == 64    ? launch_rotate<8>(p, inter, i64, handle->pdl, cs)
                          : s.headdim == 128 ? launch_rotate<16>(p, inter, i64, handle->pdl, cs)
                                             : launch_rotate<32>(p, inter, i64, handle->pdl, cs);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}
