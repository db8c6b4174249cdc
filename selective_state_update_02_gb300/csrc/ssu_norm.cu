// The residual's addition and RMS norm (ssu_add_norm): one pass over a token's row.
//
// Mathematics.  r = x + residual, y = r / sqrt(mean r^2 + eps) * weight, in fp32; r goes back to the
// residual and y out as bf16, or as e4m3 with one scale, max |y| / 448, per group of columns.
//
// What bounds it: HBM.  Every element of x and the residual is read once and of the residual and
// out written once: a row's sum stays in registers between the sum of squares and the output.
// 16384 x 8192 into bf16 154 us (1.03 of the measured copy rate); 8192 x 4096 into e4m3 with scales of
// 128 columns 42 us (0.83; 45 with half of the warps at 78 registers), where the groups' maxima,
// scales and conversions add issue; 8 x 4096 2.7 to 3.2 (a launch: it differs as much between boxes).
// Rows past 16384 columns take eight vectors a thread and one CTA per SM: 4096 x 32768 into bf16 192 us
// (0.82), into e4m3 233 (0.60, with 52 spilled bytes); 4096 x 20000 111 and 179 (0.87 and 0.48).
//
// Layout.  A row belongs to a number of whole warps with up to kMostVectors vectors of 8 columns
// per thread, neighbours in neighbouring threads, so that a warp instruction moves 512 contiguous
// bytes and a group of 32 .. 256 columns is 4 .. 32 neighbouring lanes.  All loads of a thread go
// out before the first is used.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
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

constexpr int kMostVectors = 8, kMostThreads = 512;
constexpr float kE4m3Most = 448.0f;

struct NormParams {
    const __nv_bfloat16 *x;
    void *residual;  // NULL: none
    const float *weight;
    void *out;
    float *scales;
    long long x_t, r_t, o_t, s_t, s_c;
    long long tokens;
    int vectors;  // of 8 columns per row
    int lanes;    // per group; 0: the whole row
    float eps, width;
};

enum class Residual { kNone, kBf16, kF32 };

// The larger, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

__device__ __forceinline__ float largest(const float2 (&v)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max_nan(m, max_nan(fabsf(v[j].x), fabsf(v[j].y)));
    return m;
}

__device__ __forceinline__ uint4 packed(const float2 (&v)[4]) {
    return make_uint4(f2_to_bf2(v[0].x, v[0].y), f2_to_bf2(v[1].x, v[1].y),
                      f2_to_bf2(v[2].x, v[2].y), f2_to_bf2(v[3].x, v[3].y));
}

// The combined value of a row's threads (every thread of the CTA calls it: rows share the barrier).
template <typename F>
__device__ __forceinline__ float over_row(float v, F join, float *room) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, m));
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float *const mine = room + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
    __syncthreads();
    float all = mine[0];
    for (int w = 1; w < warps; ++w) all = join(all, mine[w]);
    return all;
}

// blockDim = (threads per row, rows).
template <int V, Residual kResidual, bool kE4m3>
__global__ void __launch_bounds__(kMostThreads, V <= 4 ? 2 : 1) ssu_add_norm_kernel(
    const __grid_constant__ NormParams p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float room[2][32];
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = t < p.tokens;
    uint4 raw[V], res[V][kResidual == Residual::kF32 ? 2 : 1];
    auto holds = [&](int i) { return live && threadIdx.x + i * blockDim.x < p.vectors; };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        raw[i] = res[i][0] = make_uint4(0, 0, 0, 0);
        if constexpr (kResidual == Residual::kF32) res[i][1] = make_uint4(0, 0, 0, 0);
        if (!holds(i)) continue;
        const long long at = 8ll * (threadIdx.x + i * blockDim.x);
        raw[i] = __ldcs(reinterpret_cast<const uint4 *>(p.x + t * p.x_t + at));
        if constexpr (kResidual == Residual::kBf16)
            res[i][0] = __ldcs(reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(p.residual) + t * p.r_t + at));
        if constexpr (kResidual == Residual::kF32) {
            const uint4 *r = reinterpret_cast<const uint4 *>(
                static_cast<const float *>(p.residual) + t * p.r_t + at);
            res[i][0] = __ldcs(r);
            res[i][1] = __ldcs(r + 1);
        }
    }
    // With few vectors per thread the weights come under the sum of squares; more would cost resident
    // warps, of which a call of many rows has enough to hide them (8192 x 4096 into e4m3: 45 us, 54
    // with them, before the arithmetic was packed).
    constexpr bool kEarly = V <= 2;
    float4 weight[kEarly ? V : 1][2];
    auto weigh = [&](int i, float4 (&to)[2]) {
        const float4 *const w =
            reinterpret_cast<const float4 *>(p.weight) + 2 * (threadIdx.x + i * blockDim.x);
        to[0] = __ldg(w);
        to[1] = __ldg(w + 1);
    };
    if constexpr (kEarly)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (holds(i)) weigh(i, weight[i]);
    float2 v[V][4], squares = make_float2(0.0f, 0.0f);  // packed fp32x2 arithmetic: issue counts
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const unsigned u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        const unsigned r[4] = {res[i][0].x, res[i][0].y, res[i][0].z, res[i][0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i][j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
            if constexpr (kResidual == Residual::kBf16)
                v[i][j] = __fadd2_rn(v[i][j], make_float2(__uint_as_float(r[j] << 16),
                                                          __uint_as_float(r[j] & 0xffff0000u)));
        }
        if constexpr (kResidual == Residual::kF32) {
            const uint4 &a = res[i][0], &b = res[i][1];
            const unsigned f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[i][j] = __fadd2_rn(v[i][j], make_float2(__uint_as_float(f[2 * j]),
                                                          __uint_as_float(f[2 * j + 1])));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) squares = __ffma2_rn(v[i][j], v[i][j], squares);
        if (kResidual == Residual::kNone || !holds(i)) continue;
        const long long at = 8ll * (threadIdx.x + i * blockDim.x);
        if constexpr (kResidual == Residual::kBf16) {
            __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.residual) + t * p.r_t +
                                             at),
                   packed(v[i]));
        } else {
            float4 *r = reinterpret_cast<float4 *>(static_cast<float *>(p.residual) + t * p.r_t +
                                                   at);
            __stcs(r, make_float4(v[i][0].x, v[i][0].y, v[i][1].x, v[i][1].y));
            __stcs(r + 1, make_float4(v[i][2].x, v[i][2].y, v[i][3].x, v[i][3].y));
        }
    }
    const float sum = over_row(squares.x + squares.y, [](float a, float b) { return a + b; },
                               room[0]);
    const float rms = 1.0f / sqrtf(sum / p.width + p.eps);
    float most = 0.0f;  // of the thread's columns, where the row has one scale
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (!holds(i)) continue;
        if constexpr (!kEarly) weigh(i, weight[0]);
        const float4 a = weight[kEarly ? i : 0][0], b = weight[kEarly ? i : 0][1];
        const float2 f[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y),
                             make_float2(b.z, b.w)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[i][j] = __fmul2_rn(__fmul2_rn(v[i][j], make_float2(rms, rms)), f[j]);
        if constexpr (kE4m3) {
            if (p.lanes == 0) most = max_nan(most, largest(v[i]));
        } else {
            __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + t * p.o_t +
                                             8ll * (threadIdx.x + i * blockDim.x)),
                   packed(v[i]));
        }
    }
    if constexpr (kE4m3) {
        auto scale_of = [](float m) {
            const float s = m * (1.0f / kE4m3Most);
            return s < 0x1p-126f ? 0x1p-126f : s;  // NaN stays
        };
        float scale = 0.0f;
        if (p.lanes == 0) {
            scale = scale_of(over_row(most, max_nan, room[1]));
            if (live && threadIdx.x == 0) p.scales[t * p.s_t] = scale;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (p.lanes) {
                float m = largest(v[i]);
                for (int x = p.lanes >> 1; x >= 1; x >>= 1)
                    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
                scale = scale_of(m);
                if (holds(i) && (at & (p.lanes - 1)) == 0)
                    p.scales[t * p.s_t + at / p.lanes * p.s_c] = scale;
            }
            if (!holds(i)) continue;
            // 2 ulp; scales lie in 2^-126 .. 2^120.  (Eight divisions per vector instead: 48.4 us for
            // 42.3 of 8192 x 4096, 6.5 for 4.9 of 777 x 2560.  The rounding to 4 bits moves a value by
            // 2^-4 at most, and 2^-21 of it shows only next to the middle of two neighbours.)
            const float inverse = __fdividef(1.0f, scale);
            unsigned o[2] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j / 2] |= static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(
                                __fmul2_rn(v[i][j], make_float2(inverse, inverse)), __NV_SATFINITE,
                                __NV_E4M3))
                            << (16 * (j % 2));
            __stcs(reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.out) + t * p.o_t +
                                             8ll * at),
                   make_uint2(o[0], o[1]));
        }
    }
}

template <int V, Residual kResidual>
cudaError_t launch_norm(const cudaLaunchConfig_t &cfg, const NormParams &p, bool e4m3) {
    return e4m3 ? cudaLaunchKernelEx(&cfg, ssu_add_norm_kernel<V, kResidual, true>, p)
                : cudaLaunchKernelEx(&cfg, ssu_add_norm_kernel<V, kResidual, false>, p);
}

template <int V>
cudaError_t launch_norm(const cudaLaunchConfig_t &cfg, const NormParams &p, Residual residual,
                        bool e4m3) {
    return residual == Residual::kNone   ? launch_norm<V, Residual::kNone>(cfg, p, e4m3)
           : residual == Residual::kBf16 ? launch_norm<V, Residual::kBf16>(cfg, p, e4m3)
                                         : launch_norm<V, Residual::kF32>(cfg, p, e4m3);
}

cudaError_t launch_norm(const NormParams &p, Residual residual, bool e4m3, int sm_count, bool pdl,
                        cudaStream_t st) {
    // Threads per row for `v` vectors each, in whole warps.
    auto threads = [&](int v) { return (p.vectors + 32 * v - 1) / (32 * v) * 32; };
    // Many rows: up to four vectors per thread (16384 x 8192: 154 us, 170 with two).  Rows that are all
    // resident at once: fewer, for more loads of weights under the sums (777 x 2560 into e4m3 with a
    // scale per row 5.8 us, 8.3 with four, before the arithmetic was packed; 4.9 now).
    const int most = p.tokens <= 8ll * sm_count ? 256 : 128;
    int v = 1;
    while (v < 4 && threads(v) > most) v *= 2;
    if (threads(v) > kMostThreads) v = kMostVectors;
    const int per_row = threads(v);
    const int rows = per_row >= 128 ? 1 : 128 / per_row;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.tokens + rows - 1) / rows));
    cfg.blockDim = dim3(static_cast<unsigned>(per_row), static_cast<unsigned>(rows));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return v == 1   ? launch_norm<1>(cfg, p, residual, e4m3)
           : v == 2 ? launch_norm<2>(cfg, p, residual, e4m3)
           : v == 4 ? launch_norm<4>(cfg, p, residual, e4m3)
                    : launch_norm<kMostVectors>(cfg, p, residual, e4m3);
}

}  // namespace

extern "C" ssu_status_t ssu_add_norm(ssu_handle_t handle, const uint16_t *x, void *residual,
                                     const float *weight, void *out, float *scales,
                                     const ssu_norm_args_t *args, float eps,
                                     ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    if (!args) return fail(SSU_ERR_INVALID_ARG, "args must not be NULL");
    const ssu_norm_args_t &s = *args;
    if (s.tokens < 0 || s.tokens > INT_MAX)
        return fail(SSU_ERR_INVALID_ARG, "tokens %lld outside 0..2^31 - 1", (long long)s.tokens);
    if (s.out_dtype != SSU_NORM_BF16 && s.out_dtype != SSU_NORM_E4M3)
        return fail(SSU_ERR_INVALID_ARG, "out_dtype %d is neither BF16 nor E4M3", s.out_dtype);
    if (residual && s.residual_dtype != SSU_RESIDUAL_BF16 && s.residual_dtype != SSU_RESIDUAL_F32)
        return fail(SSU_ERR_INVALID_ARG, "residual_dtype %d is neither BF16 nor F32",
                    s.residual_dtype);
    if (s.width < 8 || s.width > 8 * kMostVectors * kMostThreads || s.width % 8)
        return fail(SSU_ERR_UNSUPPORTED, "width %lld is not a multiple of 8 in 8..%d",
                    (long long)s.width, 8 * kMostVectors * kMostThreads);
    const bool e4m3 = s.out_dtype == SSU_NORM_E4M3;
    if (e4m3 && s.group != s.width &&
        ((s.group != 32 && s.group != 64 && s.group != 128 && s.group != 256) ||
         s.width % s.group))
        return fail(SSU_ERR_UNSUPPORTED, "group %lld: 32, 64, 128, 256 that divide the width %lld, "
                    "or the width", (long long)s.group, (long long)s.width);
    if (!(eps >= 0.0f)) return fail(SSU_ERR_INVALID_ARG, "eps must be >= 0");
    if (s.tokens == 0) return ok();
    const int64_t rows[] = {s.x, residual ? s.residual : 0, s.out};
    for (int64_t u : rows) {
        if (u < 0) return fail(SSU_ERR_INVALID_ARG, "negative stride");
        if (u % 8) return fail(SSU_ERR_MISALIGNED, "a stride of %lld elements is not a multiple "
                               "of 8", (long long)u);
    }
    if (s.tokens > 1 && (s.out < s.width || (residual && s.residual < s.width)))
        return fail(SSU_ERR_INVALID_ARG, "rows of out or of the residual overlap");
    if (!x || !weight || !out || (e4m3 && !scales))
        return fail(SSU_ERR_INVALID_ARG, "a data pointer is NULL");
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
        !aligned(out, e4m3 ? 8 : 16))
        return fail(SSU_ERR_MISALIGNED, "an operand is not 16-byte aligned");
    if (e4m3) {
        if (s.scales[0] < 0 || s.scales[1] < 0)
            return fail(SSU_ERR_INVALID_ARG, "negative stride");
        if ((s.tokens > 1 && s.scales[0] == 0) || (s.group < s.width && s.scales[1] == 0))
            return fail(SSU_ERR_INVALID_ARG, "scales overlap");
        if (!aligned(scales, 4)) return fail(SSU_ERR_MISALIGNED, "scales are not 4-byte aligned");
    }
    NormParams p{};
    p.x = reinterpret_cast<const __nv_bfloat16 *>(x);
    p.residual = residual, p.weight = weight, p.out = out, p.scales = scales;
    p.x_t = s.x, p.r_t = s.residual, p.o_t = s.out, p.s_t = s.scales[0], p.s_c = s.scales[1];
    p.tokens = s.tokens;
    p.vectors = static_cast<int>(s.width / 8);
    p.lanes = e4m3 && s.group != s.width ? static_cast<int>(s.group / 8) : 0;
    p.eps = eps, p.width = static_cast<float>(s.width);
    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    const cudaError_t e = launch_norm(
        p, !residual                               ? Residual::kNone
           : s.residual_dtype == SSU_RESIDUAL_BF16 ? Residual::kBf16
                                                   : Residual::kF32,
        e4m3, handle->sm_count, handle->pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}
