// Attention of one new token per request over a paged cache: the C entry points
// ssu_attend_workspace_bytes and ssu_attend; the kernel is in ssu_attend.cuh.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ssu.h"
#include "ssu_attend.cuh"
#include "ssu_host.h"

using ssu_host::aligned;
using ssu_host::DeviceGuard;
using ssu_host::fail;
using ssu_host::ok;

namespace {

// Workspace: the counters, then two parts per CTA.
struct AttendLayout {
    long long parts, total;
};

AttendLayout attend_layout(int ctas, int64_t headdim) {
    AttendLayout w;
    w.parts = (ctas * 4ll + 255) / 256 * 256;
    w.total = w.parts + 2ll * ctas * (kAttendRows * headdim + 2 * kAttendRows) * 4;
    return w;
}

template <int D>
cudaError_t launch_attend(const AttendParams &p, ssu_handle_s &handle, bool i64,
                          cudaStream_t st) {
    using Geo = AttendGeo<D>;
    auto *kernel = i64 ? ssu_attend_kernel<D, true> : ssu_attend_kernel<D, false>;
    cudaError_t e = ssu_host::allow_smem(handle, reinterpret_cast<const void *>(kernel),
                                         Geo::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(handle.sm_count));
    cfg.blockDim = dim3(32 * Geo::kWarps);
    cfg.dynamicSmemBytes = Geo::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = handle.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

ssu_status_t validate_shape(const ssu_attend_shape_t &s) {
    if (s.requests < 0 || s.num_pages < 0 || s.max_pages < 0)
        return fail(SSU_ERR_INVALID_ARG, "requests, num_pages and max_pages must be >= 0");
    if (s.q_heads < 1 || s.kv_heads < 1 || s.page_size < 1)
        return fail(SSU_ERR_INVALID_ARG, "q_heads, kv_heads and page_size must be >= 1");
    if (s.q_heads % s.kv_heads)
        return fail(SSU_ERR_INVALID_ARG, "q_heads %lld is not a multiple of kv_heads %lld",
                    (long long)s.q_heads, (long long)s.kv_heads);
    if (s.index_dtype != SSU_INDEX_I32 && s.index_dtype != SSU_INDEX_I64)
        return fail(SSU_ERR_INVALID_ARG, "index_dtype %d is neither I32 nor I64", s.index_dtype);
    if (s.headdim != 64 && s.headdim != 128 && s.headdim != 256)
        return fail(SSU_ERR_UNSUPPORTED, "headdim %lld: this build implements 64, 128 and 256",
                    (long long)s.headdim);
    if (s.q_heads > 65535)
        return fail(SSU_ERR_UNSUPPORTED, "q_heads is limited to 65535");
    if (s.requests > INT_MAX / s.q_heads)
        return fail(SSU_ERR_UNSUPPORTED, "requests * q_heads exceeds 2^31");
    if (s.num_pages > INT_MAX) return fail(SSU_ERR_UNSUPPORTED, "num_pages exceeds 2^31");
    if (s.max_pages > 0 && s.page_size > (INT_MAX - 4096) / s.max_pages)
        return fail(SSU_ERR_UNSUPPORTED, "max_pages * page_size exceeds 2^31");
    return SSU_OK;
}

}  // namespace

extern "C" {

ssu_status_t ssu_attend_workspace_bytes(ssu_handle_t handle, const ssu_attend_shape_t *shape,
                                        int64_t *bytes) {
    if (!handle || !shape || !bytes) return fail(SSU_ERR_INVALID_ARG, "NULL argument");
    const ssu_status_t st = validate_shape(*shape);
    if (st != SSU_OK) return st;
    *bytes = attend_layout(handle->sm_count, shape->headdim).total;
    return ok();
}

ssu_status_t ssu_attend(ssu_handle_t handle, const uint16_t *q, const uint16_t *k_pages,
                        const uint16_t *v_pages, const void *page_table, const void *lengths,
                        uint16_t *out, const ssu_attend_shape_t *shape,
                        const ssu_attend_strides_t *strides, float scale, int64_t window,
                        int64_t sinks, void *workspace, int64_t workspace_bytes,
                        ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    if (!shape || !strides)
        return fail(SSU_ERR_INVALID_ARG, "shape and strides must not be NULL");
    const ssu_attend_shape_t &s = *shape;
    const ssu_attend_strides_t &u = *strides;
    ssu_status_t st = validate_shape(s);
    if (st != SSU_OK) return st;
    if (window < 0 || sinks < 0)
        return fail(SSU_ERR_INVALID_ARG, "window and sinks must be >= 0");
    if (!(scale == scale) || scale - scale != 0.0f)
        return fail(SSU_ERR_INVALID_ARG, "scale must be finite");
    if (s.requests == 0) return ok();
    const int64_t vec[] = {u.q[0], u.q[1], u.out[0], u.out[1], u.k_pages[0], u.k_pages[1],
                           u.k_pages[2], u.v_pages[0], u.v_pages[1], u.v_pages[2]};
    for (int64_t x : vec) {
        if (x < 0) return fail(SSU_ERR_INVALID_ARG, "negative stride");
        if (x % 8) return fail(SSU_ERR_MISALIGNED, "a stride of %lld elements is not a multiple "
                               "of 16 bytes", (long long)x);
    }
    if (u.page_table[0] < 0 || u.page_table[1] < 0 || u.lengths < 0)
        return fail(SSU_ERR_INVALID_ARG, "negative stride");
    if (!q || !lengths || !out || (s.num_pages && (!k_pages || !v_pages)) ||
        (s.max_pages && !page_table))
        return fail(SSU_ERR_INVALID_ARG, "a data pointer is NULL");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16))
        return fail(SSU_ERR_MISALIGNED, "an operand is not 16-byte aligned");
    const unsigned isz = s.index_dtype == SSU_INDEX_I64 ? 8 : 4;
    if (!aligned(page_table, isz) || !aligned(lengths, isz))
        return fail(SSU_ERR_MISALIGNED, "page_table or lengths are not aligned to their type");
    int64_t need = 0;
    st = ssu_attend_workspace_bytes(handle, shape, &need);
    if (st != SSU_OK) return st;
    if (workspace_bytes < need || (need && !workspace))
        return fail(SSU_ERR_INVALID_ARG, "workspace holds %lld bytes; this shape needs %lld",
                    (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (need && !aligned(workspace, 256))
        return fail(SSU_ERR_MISALIGNED, "workspace is not 256-byte aligned");

    AttendParams p;
    auto bf = [](const uint16_t *t) { return reinterpret_cast<const __nv_bfloat16 *>(t); };
    p.q = bf(q), p.k = bf(k_pages), p.v = bf(v_pages);
    p.table = page_table, p.lengths = lengths;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.q_b = u.q[0], p.q_h = u.q[1], p.o_b = u.out[0], p.o_h = u.out[1];
    p.k_p = u.k_pages[0], p.k_r = u.k_pages[1], p.k_h = u.k_pages[2];
    p.v_p = u.v_pages[0], p.v_r = u.v_pages[1], p.v_h = u.v_pages[2];
    p.t_b = u.page_table[0], p.t_p = u.page_table[1], p.len_s = u.lengths;
    p.requests = s.requests, p.num_pages = s.num_pages;
    p.page_size = static_cast<int>(s.page_size < INT_MAX ? s.page_size : INT_MAX);
    p.max_keys = s.max_pages * s.page_size;
    p.window = window, p.sinks = sinks;
    p.q_heads = static_cast<int>(s.q_heads), p.kv_heads = static_cast<int>(s.kv_heads);
    p.share = static_cast<int>(s.q_heads / s.kv_heads);
    p.head_tiles = (p.share + kAttendRows - 1) / kAttendRows;
    // The last vector of the caches, in 16-byte vectors from their start (in double: a stride may
    // be any number of an array with one page).
    const double last_k = static_cast<double>(s.num_pages) * u.k_pages[0] +
                          static_cast<double>(s.page_size) * u.k_pages[1] +
                          static_cast<double>(s.kv_heads) * u.k_pages[2];
    const double last_v = static_cast<double>(s.num_pages) * u.v_pages[0] +
                          static_cast<double>(s.page_size) * u.v_pages[1] +
                          static_cast<double>(s.kv_heads) * u.v_pages[2];
    p.wide = last_k / 8 > 4e9 || last_v / 8 > 4e9;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = handle->err;
    p.arrived = static_cast<unsigned *>(workspace);
    p.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                        attend_layout(handle->sm_count, s.headdim).parts);

    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool i64 = s.index_dtype == SSU_INDEX_I64;
    const cudaError_t e = s.headdim == 64    ? launch_attend<64>(p, *handle, i64, cs)
                          : s.headdim == 128 ? launch_attend<128>(p, *handle, i64, cs)
                                             : launch_attend<256>(p, *handle, i64, cs);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
