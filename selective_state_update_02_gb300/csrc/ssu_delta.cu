// The gated delta rule: the C entry points ssu_delta_update, ssu_delta_workspace_bytes and
// ssu_delta_prompts (validation, choice of form) and the kernels' instantiations.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ssu.h"
#include "ssu_delta.cuh"
#include "ssu_delta_mma.cuh"
#include "ssu_host.h"
#include "ssu_tma.h"

using ssu_host::aligned;
using ssu_host::DeviceGuard;
using ssu_host::fail;
using ssu_host::ok;
using ssu_host::validate_batch;
using ssu_host::validate_shape;

namespace {

struct DeltaOperands {
    void *state_pool;
    const void *idx;
    const uint16_t *q, *k, *v, *dt, *b;
    const float *dt_bias, *A;
    uint16_t *out;
};

ssu_status_t validate_delta(const DeltaOperands &o, const ssu_shape_t *shape,
                            const ssu_delta_strides_t *strides, float scale, float eps) {
    if (!shape || !strides)
        return fail(SSU_ERR_INVALID_ARG, "shape and strides must not be NULL");
    const ssu_shape_t &s = *shape;
    const ssu_delta_strides_t &u = *strides;
    const ssu_status_t sizes = validate_shape(s);
    if (sizes != SSU_OK) return sizes;
    if (!(scale == scale) || scale - scale != 0.0f)
        return fail(SSU_ERR_INVALID_ARG, "scale must be finite");
    if (!(eps == eps)) return fail(SSU_ERR_INVALID_ARG, "qk_eps must not be NaN");
    if (s.batch == 0) return ok();
    const int64_t all[] = {u.state[0], u.state[1], u.state[2], u.q[0], u.q[1], u.k[0], u.k[1],
                           u.v[0], u.v[1], u.out[0], u.out[1], u.dt[0], u.dt[1], u.b[0], u.b[1],
                           u.dt_bias, u.A, u.idx};
    for (int64_t x : all)
        if (x < 0) return fail(SSU_ERR_INVALID_ARG, "negative stride");
    const int per16 = s.state_dtype == SSU_STATE_BF16 ? 8 : 4;
    for (int j = 0; j < 3; ++j)
        if (u.state[j] % per16)
            return fail(SSU_ERR_MISALIGNED,
                        "state stride %d (%lld elements) is not a multiple of 16 bytes", j,
                        (long long)u.state[j]);
    if (!o.state_pool || !o.idx || !o.q || !o.k || !o.v || !o.dt || !o.b || !o.dt_bias || !o.A ||
        !o.out)
        return fail(SSU_ERR_INVALID_ARG, "a data pointer is NULL");
    if (!aligned(o.state_pool, 16))
        return fail(SSU_ERR_MISALIGNED, "state_pool is not 16-byte aligned");
    if (!aligned(o.idx, s.index_dtype == SSU_INDEX_I64 ? 8 : 4))
        return fail(SSU_ERR_MISALIGNED, "state_batch_indices is not aligned to its type");
    for (const void *ptr : {o.q, o.k, o.v, o.dt, o.b, static_cast<const uint16_t *>(o.out)})
        if (!aligned(ptr, 2))
            return fail(SSU_ERR_MISALIGNED, "a bf16 operand is not 2-byte aligned");
    if (!aligned(o.dt_bias, 4) || !aligned(o.A, 4))
        return fail(SSU_ERR_MISALIGNED, "an fp32 operand is not 4-byte aligned");
    return validate_batch(s);
}

DeltaParams delta_params(const ssu_handle_s &handle, const DeltaOperands &o, const ssu_shape_t &s,
                         const ssu_delta_strides_t &u, float scale, float eps) {
    DeltaParams d{};
    SsuParams &p = d.m.p;
    auto bf = [](const uint16_t *t) { return reinterpret_cast<const __nv_bfloat16 *>(t); };
    p.state = o.state_pool, p.idx = o.idx;
    p.x = bf(o.v), p.B = bf(o.k), p.C = bf(o.q), p.dt = bf(o.dt), d.beta = bf(o.b);
    p.dt_bias = o.dt_bias, p.A = o.A;
    p.out = reinterpret_cast<__nv_bfloat16 *>(o.out);
    p.st_pool = u.state[0], p.st_head = u.state[1], p.st_row = u.state[2];
    p.x_b = u.v[0], p.x_h = u.v[1], p.out_b = u.out[0], p.out_h = u.out[1];
    p.dt_b = u.dt[0], p.dt_h = u.dt[1], d.beta_t = u.b[0], d.beta_h = u.b[1];
    p.B_b = u.k[0], p.B_g = u.k[1], p.C_b = u.q[0], p.C_g = u.q[1];
    p.bias_h = u.dt_bias, p.A_h = u.A, p.idx_s = u.idx;
    p.pool_size = s.pool_size, p.batch = s.batch;
    p.nheads = static_cast<int>(s.nheads), p.headdim = static_cast<int>(s.headdim);
    p.heads_per_group = static_cast<int>(s.nheads / s.ngroups);
    p.group_magic = group_magic(static_cast<unsigned>(p.heads_per_group));
    p.err = handle.err;
    const int epv = s.state_dtype == SSU_STATE_BF16 ? 8 : 4;
    d.m.bc_vec = aligned(o.k, 2 * epv) && p.B_b % epv == 0 && p.B_g % epv == 0 &&
                 aligned(o.q, 2 * epv) && p.C_b % epv == 0 && p.C_g % epv == 0;
    d.scale = scale, d.eps = eps;
    return d;
}

// Launches `kernel` with a warp per kRows rows of a head, up to four warps to a CTA.
template <int kRows, typename Kernel>
cudaError_t launch_rows(Kernel *kernel, DeltaParams d, bool pdl, cudaStream_t st) {
    SsuParams &p = d.m.p;
    int warps = 4;
    while (warps > 1 && kRows * (warps / 2) >= p.headdim) warps >>= 1;
    p.rows_per_cta = kRows * warps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.headdim + p.rows_per_cta - 1) / p.rows_per_cta),
                       static_cast<unsigned>(p.nheads),
                       static_cast<unsigned>(p.batch < 65535 ? p.batch : 65535));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, d);
}

template <int N, typename ST, bool kIdx64>
cudaError_t launch_step(const DeltaParams &d, bool pdl, cudaStream_t st) {
    constexpr int kSlots = RowGeo<N, ST>::L == 8 ? 4 : RowGeo<N, ST>::L / 4;
    return launch_rows<kSlots * RowGeo<N, ST>::RPI>(ssu_delta_step_kernel<kSlots, N, ST, kIdx64>, d,
                                                    pdl, st);
}

constexpr int kSeqSlots = 4;

template <int N, typename ST, bool kIdx64>
cudaError_t launch_seq(const DeltaParams &d, bool pdl, cudaStream_t st) {
    return launch_rows<kSeqSlots * RowGeo<N, ST>::RPI>(
        ssu_delta_seq_kernel<kSeqSlots, N, ST, kIdx64>, d, pdl, st);
}

// `launch` (a generic functor of dstate, state and index type) at the call's types.
template <typename F>
cudaError_t dispatch(const ssu_shape_t &s, F launch) {
    const bool bf16 = s.state_dtype == SSU_STATE_BF16, i64 = s.index_dtype == SSU_INDEX_I64;
    auto typed = [&](auto n) {
        if (bf16)
            return i64 ? launch(n, __nv_bfloat16(), std::true_type())
                       : launch(n, __nv_bfloat16(), std::false_type());
        return i64 ? launch(n, float(), std::true_type()) : launch(n, float(), std::false_type());
    };
    if (s.dstate == 64) return typed(std::integral_constant<int, 64>());
    if (s.dstate == 128) return typed(std::integral_constant<int, 128>());
    return typed(std::integral_constant<int, 256>());
}

ssu_status_t validate_tokens(int64_t tokens) {
    if (tokens < 0 || tokens > INT_MAX)
        return fail(SSU_ERR_INVALID_ARG, "tokens %lld outside 0..2^31 - 1", (long long)tokens);
    return ok();
}

// ---- the chunked form ----------------------------------------------------------------

// Where its arrays lie in the workspace.
struct DeltaPlan {
    long long chunks;  // the most that good prompts can have
    long long prompts, list, records, total;
};

// Records past this (2.4 million tokens of 32 heads) leave a call to the token-by-token form.
constexpr double kMostRecords = 3.2e10;

// Few tokens go token by token.  Both forms in us, fitted to 1 to 128 prompts of 1 to 2048 tokens, with
// w the elements of a request's state by those of 32 heads of 128 x 128:
//   chunks          5 and 11 (dstate 64: 8) for every round of SMs that prompts times heads' slabs come
//                   to (32 heads, 1 prompt 15.8, 8 prompts 27, 32 83, 128 302; 16 of 64 x 64, 1 prompt
//                   13, 128 118)
//   token by token  3 and 0.32 + 0.16 w for each token of the longest prompt (1 prompt of 24: 12.8, of
//                   36: 17.8; 64 heads 18.8 and 27.2), or what all of them take: w (0.8 a prompt, 0.26
//                   a token) (128 prompts of 6 tokens: 278)
// Of the longest prompt the host knows no more than that the others may have a token each, and takes
// that.  Where tokens are spread evenly, token by token would pay for more than the rule leaves to it,
// most where heads are few and small: 8 prompts of 8 tokens through 32 heads take 27.0 in chunks and
// 24.4 token by token (33.5 where one has 57 of them), 16 of 8 through 16 of 64 x 64 21.8 and 8.0
// (40.8).
// Below kFewest every call goes token by token, whose workspace is none.
constexpr int kFewest = 20;

bool few_tokens(const ssu_shape_t &s, int64_t tokens, int sm_count) {
    if (tokens <= kFewest) return true;
    const double prompts = static_cast<double>(s.batch), all = static_cast<double>(tokens);
    const double w = static_cast<double>(s.nheads) * s.headdim * s.dstate / (32 * 128 * 128);
    const double rounds =
        std::ceil(prompts * s.nheads * ((s.headdim + kDeltaRows - 1) / kDeltaRows) / sm_count);
    const double chain = 3 + (0.32 + 0.16 * w) * (all - prompts + 1);
    const double work = 1.5 + w * (0.8 * prompts + 0.26 * all);
    return (chain > work ? chain : work) <= 5 + (s.dstate == 64 ? 8 : 11) * rounds;
}

// Whether a call of these sizes, or one of fewer prompts with the same sizes otherwise, may go in
// chunks: what the workspace query answers by.  Unlike a call's own choice it only grows with
// prompts, tokens and heads up to kMostRecords, so that a buffer for the largest call serves all.
bool chunk_sizes(const ssu_shape_t &s, int64_t tokens) {
    return (s.dstate == 64 || s.dstate == 128) && s.batch > 0 && tokens > kFewest &&
           (tokens / kDeltaChunk + static_cast<double>(s.batch)) * s.nheads *
                   DeltaRecord::kBytes <= kMostRecords;
}

// Whether a call goes in chunks, as far as its sizes say.
bool mma_sizes(const ssu_shape_t &s, int64_t tokens, int sm_count) {
    return chunk_sizes(s, tokens) && !few_tokens(s, tokens, sm_count) &&
           s.batch * static_cast<double>(s.nheads) * ((s.headdim + kDeltaRows - 1) / kDeltaRows) <=
               INT_MAX;
}

DeltaPlan delta_plan(const ssu_shape_t &s, int64_t tokens) {
    auto up = [](long long bytes) { return (bytes + 255) / 256 * 256; };
    DeltaPlan w;
    w.chunks = tokens / kDeltaChunk + s.batch;
    w.prompts = 256;
    w.list = w.prompts + up(s.batch * static_cast<long long>(sizeof(DeltaPrompt)));
    w.records = w.list + up(8ll * w.chunks);
    w.total = w.records + w.chunks * s.nheads * DeltaRecord::kBytes;
    return w;
}

// Operands that the chunked form can read: 16-byte rows for the tensor maps.
bool mma_operands(const DeltaParams &d) {
    const SsuParams &p = d.m.p;
    if (!aligned(p.x, 16) || !aligned(p.B, 16) || !aligned(p.C, 16) || !aligned(p.out, 16))
        return false;
    const long long strides[] = {p.x_b, p.x_h, p.B_b, p.B_g, p.C_b, p.C_g, p.out_b, p.out_h};
    for (long long v : strides)
        if (v % 8 != 0 || v >= (1ll << 38)) return false;
    return true;
}

template <int N, typename ST, bool kIdx64>
cudaError_t launch_mma(const DeltaMmaParams &m, const DeltaPlan &w, const CUtensorMap (&maps)[6],
                       ssu_handle_s &handle, cudaStream_t st) {
    auto *prep = ssu_delta_prep_kernel<N>;
    auto *main = ssu_delta_mma_kernel<N, ST>;
    constexpr int kPrepBytes = PrepSmem<N>::kTotal + 1024, kBytes = DeltaSmem<N>::kTotal + 1024;
    cudaError_t e =
        ssu_host::allow_smem(handle, reinterpret_cast<const void *>(prep), kPrepBytes);
    if (e == cudaSuccess)
        e = ssu_host::allow_smem(handle, reinterpret_cast<const void *>(main), kBytes);
    if (e != cudaSuccess) return e;
    const SsuParams &p = m.d.m.p;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = handle.pdl ? 1 : 0;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    if (!m.few) {
        e = cudaLaunchKernelEx(&cfg, ssu_delta_plan_kernel<kIdx64>, m);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(w.chunks),
                       static_cast<unsigned>(p.nheads / m.per_cta));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = kPrepBytes;
    e = cudaLaunchKernelEx(&cfg, prep, m, maps[4], maps[5]);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.nheads * m.slabs));
    cfg.blockDim = dim3(kDeltaThreads);
    cfg.dynamicSmemBytes = kBytes;
    return cudaLaunchKernelEx(&cfg, main, m, maps[0], maps[1], maps[2], maps[3]);
}

cudaError_t launch_mma(const DeltaMmaParams &m, const DeltaPlan &w, const CUtensorMap (&maps)[6],
                       const ssu_shape_t &s, ssu_handle_s &handle, cudaStream_t st) {
    const bool bf16 = s.state_dtype == SSU_STATE_BF16, i64 = s.index_dtype == SSU_INDEX_I64;
#define SSU_MMA(N_, ST_)                                              \
    return i64 ? launch_mma<N_, ST_, true>(m, w, maps, handle, st)    \
               : launch_mma<N_, ST_, false>(m, w, maps, handle, st)
    if (s.dstate == 64) {
        if (bf16) SSU_MMA(64, __nv_bfloat16);
        SSU_MMA(64, float);
    }
    if (bf16) SSU_MMA(128, __nv_bfloat16);
    SSU_MMA(128, float);
#undef SSU_MMA
}

}  // namespace

extern "C" {

ssu_status_t ssu_delta_update(ssu_handle_t handle, void *state_pool,
                              const void *state_batch_indices, const uint16_t *q,
                              const uint16_t *k, const uint16_t *v, const uint16_t *dt,
                              const float *dt_bias, const float *A, const uint16_t *b,
                              uint16_t *out, const ssu_shape_t *shape,
                              const ssu_delta_strides_t *strides, float scale, float qk_eps,
                              ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    const DeltaOperands o = {state_pool, state_batch_indices, q, k, v, dt, b, dt_bias, A, out};
    const ssu_status_t st = validate_delta(o, shape, strides, scale, qk_eps);
    if (st != SSU_OK || shape->batch == 0) return st;
    const DeltaParams d = delta_params(*handle, o, *shape, *strides, scale, qk_eps);
    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dispatch(*shape, [&](auto n, auto st, auto i64) {
        return launch_step<decltype(n)::value, decltype(st), decltype(i64)::value>(d, handle->pdl,
                                                                                 cs);
    });
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

ssu_status_t ssu_delta_workspace_bytes(ssu_handle_t handle, const ssu_shape_t *shape,
                                       int64_t tokens, int64_t *bytes) {
    if (!handle || !shape || !bytes) return fail(SSU_ERR_INVALID_ARG, "NULL argument");
    ssu_status_t st = validate_shape(*shape);
    if (st == SSU_OK) st = validate_batch(*shape);
    if (st == SSU_OK) st = validate_tokens(tokens);
    if (st != SSU_OK) return st;
    *bytes = chunk_sizes(*shape, tokens) ? delta_plan(*shape, tokens).total : 0;
    return ok();
}

ssu_status_t ssu_delta_prompts(ssu_handle_t handle, void *state_pool,
                               const void *state_batch_indices, const void *cu_tokens,
                               const uint8_t *fresh, const uint16_t *q, const uint16_t *k,
                               const uint16_t *v, const uint16_t *dt, const float *dt_bias,
                               const float *A, const uint16_t *b, uint16_t *out,
                               const ssu_shape_t *shape, const ssu_delta_strides_t *strides,
                               int64_t tokens, float scale, float qk_eps, void *workspace,
                               int64_t workspace_bytes, ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    ssu_status_t st = validate_tokens(tokens);
    if (st != SSU_OK) return st;
    if (tokens == 0) {  // no token row is read: the operands may be empty arrays
        static const uint16_t none[2] = {};
        q = k = v = dt = b = none;
        out = const_cast<uint16_t *>(none);
    }
    const DeltaOperands o = {state_pool, state_batch_indices, q, k, v, dt, b, dt_bias, A, out};
    st = validate_delta(o, shape, strides, scale, qk_eps);
    if (st != SSU_OK || shape->batch == 0) return st;
    const ssu_shape_t &s = *shape;
    if (!cu_tokens) return fail(SSU_ERR_INVALID_ARG, "cu_tokens is NULL");
    if (!aligned(cu_tokens, s.index_dtype == SSU_INDEX_I64 ? 8 : 4))
        return fail(SSU_ERR_MISALIGNED, "cu_tokens is not aligned to its type");
    const bool chunks = mma_sizes(s, tokens, handle->sm_count);
    const int64_t need = chunks ? delta_plan(s, tokens).total : 0;
    if (workspace_bytes < need || (need && !workspace))
        return fail(SSU_ERR_INVALID_ARG, "workspace holds %lld bytes; this shape needs %lld",
                    (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (need && !aligned(workspace, 256))
        return fail(SSU_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    DeltaParams d = delta_params(*handle, o, s, *strides, scale, qk_eps);
    d.m.cu = cu_tokens, d.m.fresh = fresh, d.m.tokens = tokens;
    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorNotSupported;
    if (chunks && mma_operands(d)) {
        const SsuParams &p = d.m.p;
        const DeltaPlan w = delta_plan(s, tokens);
        DeltaMmaParams m{};
        m.d = d;
        m.idx64 = s.index_dtype == SSU_INDEX_I64;
        m.few = s.batch <= 32;
        m.slabs = static_cast<int>((s.headdim + kDeltaRows - 1) / kDeltaRows);
        // Heads of one key head share its products in the first pass where that leaves two CTAs
        // per SM and more.
        m.per_cta = 1;
        while (m.per_cta < kPrepHeads && p.heads_per_group % (2 * m.per_cta) == 0 &&
               w.chunks * (s.nheads / (2 * m.per_cta)) >= 2 * handle->sm_count)
            m.per_cta *= 2;
        char *const room = static_cast<char *>(workspace);
        m.total = reinterpret_cast<int *>(room);
        m.prompts = reinterpret_cast<DeltaPrompt *>(room + w.prompts);
        m.chunks = reinterpret_cast<int2 *>(room + w.list);
        m.records = reinterpret_cast<unsigned char *>(room + w.records);
        CUtensorMap maps[6];
        if (encode_map(&maps[0], k, s.dstate, s.ngroups, tokens, p.B_g, p.B_b, kDeltaChunk) &&
            encode_map(&maps[1], q, s.dstate, s.ngroups, tokens, p.C_g, p.C_b, kDeltaChunk) &&
            encode_map(&maps[2], v, s.headdim, s.nheads, tokens, p.x_h, p.x_b, kDeltaChunk) &&
            encode_map(&maps[3], out, s.headdim, s.nheads, tokens, p.out_h, p.out_b, kDeltaChunk) &&
            encode_map(&maps[4], k, s.dstate, s.ngroups, tokens, p.B_g, p.B_b, kDeltaChunk / 4) &&
            encode_map(&maps[5], q, s.dstate, s.ngroups, tokens, p.C_g, p.C_b, kDeltaChunk / 4))
            e = launch_mma(m, w, maps, s, *handle, cs);
    }
    if (e == cudaErrorNotSupported) e = dispatch(s, [&](auto n, auto st, auto i64) {
        return launch_seq<decltype(n)::value, decltype(st), decltype(i64)::value>(d, handle->pdl,
                                                                                cs);
    });
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
