// Prompts: the C entry points ssu_prompts_workspace_bytes and ssu_update_prompts (validation,
// choice of form) and the kernels' instantiations.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ssu.h"
#include "ssu_host.h"
#include "ssu_prompt.cuh"
#include "ssu_prompt_mma.cuh"
#include "ssu_tma.h"

using ssu_host::aligned;
using ssu_host::DeviceGuard;
using ssu_host::fail;
using ssu_host::ok;
using ssu_host::validate_batch;
using ssu_host::validate_impl;
using ssu_host::validate_shape;

namespace {

constexpr int kSeqSlots = 4, kSeqWarps = 4;

template <int N, typename ST>
cudaError_t launch_seq(PromptParams q, bool i64, bool pdl, cudaStream_t st) {
    constexpr int kRows = kSeqSlots * RowGeo<N, ST>::RPI;
    int warps = kSeqWarps;
    while (warps > 1 && kRows * (warps / 2) >= q.p.headdim) warps >>= 1;
    q.p.rows_per_cta = kRows * warps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((q.p.headdim + kRows * warps - 1) / (kRows * warps)),
                       static_cast<unsigned>(q.p.nheads),
                       static_cast<unsigned>(q.p.batch < 65535 ? q.p.batch : 65535));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return i64 ? cudaLaunchKernelEx(&cfg, ssu_prompt_seq_kernel<kSeqSlots, N, ST, true>, q)
               : cudaLaunchKernelEx(&cfg, ssu_prompt_seq_kernel<kSeqSlots, N, ST, false>, q);
}

cudaError_t launch_seq(const PromptParams &q, int dstate, bool bf16, bool i64, bool pdl,
                       cudaStream_t st) {
    if (dstate == 64)
        return bf16 ? launch_seq<64, __nv_bfloat16>(q, i64, pdl, st)
                    : launch_seq<64, float>(q, i64, pdl, st);
    if (dstate == 128)
        return bf16 ? launch_seq<128, __nv_bfloat16>(q, i64, pdl, st)
                    : launch_seq<128, float>(q, i64, pdl, st);
    return bf16 ? launch_seq<256, __nv_bfloat16>(q, i64, pdl, st)
                : launch_seq<256, float>(q, i64, pdl, st);
}

ssu_status_t validate_tokens(int64_t tokens) {
    if (tokens < 0 || tokens > INT_MAX)
        return fail(SSU_ERR_INVALID_ARG, "tokens %lld outside 0..2^31 - 1", (long long)tokens);
    return ok();
}

// ---- the chunked form ----------------------------------------------------------------

// How a call is cut: chunks per stretch, the most stretches that gives, the most of them that are
// not their prompt's last (those have a first pass), and the workspace.
struct PromptPlan {
    long long seg, stretches, earlier, columns, ctas;  // ctas: per stretch
    long long decay, hand, turn, total;  // offsets of PromptMmaParams' arrays; bytes
    bool line;               // the second pass runs along the line
};

// The kernels' token numbers are 32 bits wide and run up to two chunks past a prompt's end.
bool mma_sizes(const ssu_shape_t &s, int64_t tokens) {
    return (s.dstate == 64 || s.dstate == 128) && s.headdim % kSlab == 0 &&
           tokens <= INT_MAX - 4 * kChunk;
}

// Grids that the device can launch (the line's is one CTA per SM).
bool mma_grids(const PromptPlan &w) {
    return w.earlier * w.ctas <= INT_MAX && (w.line || w.stretches * w.ctas <= INT_MAX);
}

PromptPlan prompt_plan(const ssu_shape_t &s, int64_t tokens, int sm_count) {
    PromptPlan w{};
    w.columns = s.nheads * (s.headdim / kSlab);
    w.ctas = s.ngroups * ((w.columns / s.ngroups + 1) / 2);
    // One CTA per SM: as many chunks per stretch as spread the call's over them.  Where the prompts
    // alone come to more than half the SMs, a prompt of up to twice the mean length stays whole, as
    // what a cut would gain it costs in the first pass (6 prompts of 5 to 10 chunks, 16 CTAs each:
    // 45 us whole, 1.28 of that cut in two; 24 of 1 to 25, 8 CTAs each: 50 us in stretches of 5,
    // 1.09 of that in 3, 1.25 in 8; one of 16 chunks, 8 CTAs: 29 us in stretches of 1, 1.31 in 5).
    const long long chunks = tokens / kChunk + s.batch;
    w.seg = (chunks * w.ctas + sm_count - 1) / sm_count;
    // Where the prompts alone are more than the SMs, whole ones take the time of `rounds` of them
    // and the line (ssu_prompt_mma.cuh) that of their share, and some 4 chunks more for the parts
    // that it adds.  The line's time over that of whole ones, 16 heads: 24 prompts of 4 chunks 1.03
    // (it saves 3.3 chunks), 60 of 4 1.02 (3.8), 24 of 8 0.86 (6.3), 20 of 8 0.76 (8), 24 of 16
    // 0.77 (12); lengths that differ by factors move these by 10 % either way.
    const long long units = s.batch * w.ctas, rounds = (units + sm_count - 1) / sm_count;
    const double mean = 0.5 + static_cast<double>(tokens) / kChunk / s.batch;
    w.line = rounds > 1 && mean * (rounds - static_cast<double>(units) / sm_count) > 4.5;
    if (!w.line && 2 * units > sm_count) {
        const long long whole = 2 * (tokens / kChunk) / s.batch;
        if (w.seg < whole) w.seg = whole;
    }
    if (s.batch == 1) w.seg = (tokens / kChunk * w.ctas + sm_count - 1) / sm_count;
    if (w.seg < 1) w.seg = 1;
    if (w.seg > 1 << 23) w.seg = 1 << 23;  // token offsets stay below 2^31
    w.stretches = tokens / (w.seg * kChunk) + s.batch;
    w.earlier = tokens / (w.seg * kChunk);
    if (tokens <= w.seg * kChunk) w.earlier = 0;
    if (w.earlier) {
        w.decay = w.stretches * w.columns * kSlab * s.dstate * 4;
        w.total = w.decay + (w.stretches * w.columns * 4 + 255) / 256 * 256;
    }
    if (w.line) {
        w.hand = w.total;
        w.turn = w.hand + static_cast<long long>(sm_count) * kPair * kSlab * s.dstate * 4;
        w.total = w.turn + (4ll * (sm_count + 1) + 255) / 256 * 256;
    }
    return w;
}

// Operands that the chunked form can read: 16-byte rows for the tensor maps (x, B, C) and for
// the stores of out.
bool mma_operands(const PromptParams &q) {
    const SsuParams &p = q.p;
    if (!aligned(p.x, 16) || !aligned(p.B, 16) || !aligned(p.C, 16) || !aligned(p.out, 16))
        return false;
    const long long strides[] = {p.x_b, p.x_h, p.B_b, p.B_g, p.C_b, p.C_g, p.out_b, p.out_h};
    for (long long v : strides)
        if (v % 8 != 0 || v >= (1ll << 38)) return false;
    return true;
}

template <int N, typename ST, bool kIdx64>
cudaError_t launch_mma(const PromptMmaParams &m, const PromptPlan &w, const CUtensorMap (&maps)[4],
                       ssu_handle_s &handle, cudaStream_t st) {
    constexpr int kBytes = PromptSmem<N>::kTotal + 1024;
    auto *first = ssu_prompt_mma_kernel<N, ST, kIdx64, Pass::kFirst>;
    auto *second = w.line ? ssu_prompt_mma_kernel<N, ST, kIdx64, Pass::kLine>
                          : ssu_prompt_mma_kernel<N, ST, kIdx64, Pass::kSecond>;
    cudaError_t e =
        ssu_host::allow_smem(handle, reinterpret_cast<const void *>(first), kBytes);
    if (e == cudaSuccess)
        e = ssu_host::allow_smem(handle, reinterpret_cast<const void *>(second), kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = handle.pdl ? 1 : 0;
    if (w.line) {
        e = cudaMemsetAsync(m.turn, 0, 4 * (handle.sm_count + 1), st);
        if (e != cudaSuccess) return e;
    }
    if (w.earlier) {
        cfg.gridDim = dim3(static_cast<unsigned>(w.earlier * w.ctas));
        e = cudaLaunchKernelEx(&cfg, first, m, maps[0], maps[1], maps[2], maps[3]);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(w.line ? static_cast<unsigned>(handle.sm_count)
                              : static_cast<unsigned>(w.stretches * w.ctas));
    return cudaLaunchKernelEx(&cfg, second, m, maps[0], maps[1], maps[2], maps[3]);
}

cudaError_t launch_mma(const PromptMmaParams &m, const PromptPlan &w, const CUtensorMap (&maps)[4],
                       int dstate, bool bf16, bool i64, ssu_handle_s &handle, cudaStream_t st) {
#define SSU_MMA(N_, ST_)                                              \
    return i64 ? launch_mma<N_, ST_, true>(m, w, maps, handle, st)    \
               : launch_mma<N_, ST_, false>(m, w, maps, handle, st)
    if (dstate == 64) {
        if (bf16) SSU_MMA(64, __nv_bfloat16);
        SSU_MMA(64, float);
    }
    if (bf16) SSU_MMA(128, __nv_bfloat16);
    SSU_MMA(128, float);
#undef SSU_MMA
}

}  // namespace

extern "C" {

ssu_status_t ssu_prompts_workspace_bytes(ssu_handle_t handle, const ssu_shape_t *shape,
                                         int64_t tokens, int64_t *bytes) {
    if (!handle || !shape || !bytes) return fail(SSU_ERR_INVALID_ARG, "NULL argument");
    ssu_status_t st = validate_shape(*shape);
    if (st == SSU_OK) st = validate_batch(*shape);
    if (st == SSU_OK) st = validate_tokens(tokens);
    if (st != SSU_OK) return st;
    *bytes = 0;
    if (mma_sizes(*shape, tokens)) {
        const PromptPlan w = prompt_plan(*shape, tokens, handle->sm_count);
        if (mma_grids(w)) *bytes = w.total;
    }
    return ok();
}

ssu_status_t ssu_update_prompts(ssu_handle_t handle, void *state_pool,
                                const void *state_batch_indices, const void *cu_tokens,
                                const uint8_t *fresh, const uint16_t *x, const uint16_t *dt,
                                const float *dt_bias, const float *A, const uint16_t *B,
                                const uint16_t *C, const float *D, uint16_t *out,
                                const ssu_shape_t *shape, const ssu_strides_t *strides,
                                int64_t tokens, void *workspace, int64_t workspace_bytes,
                                ssu_stream_t stream) {
    if (!handle) return fail(SSU_ERR_INVALID_ARG, "NULL handle");
    ssu_status_t st = validate_tokens(tokens);
    if (st != SSU_OK) return st;
    if (tokens == 0) {  // no token row is read: the operands may be empty arrays
        static const uint16_t none[2] = {};
        x = dt = B = C = none;
        out = const_cast<uint16_t *>(none);
    }
    st = validate_impl(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D,
                       out, shape, strides);
    if (st != SSU_OK || shape->batch == 0) return st;
    const ssu_shape_t &s = *shape;
    if (!cu_tokens) return fail(SSU_ERR_INVALID_ARG, "cu_tokens is NULL");
    if (!aligned(cu_tokens, s.index_dtype == SSU_INDEX_I64 ? 8 : 4))
        return fail(SSU_ERR_MISALIGNED, "cu_tokens is not aligned to its type");
    int64_t need = 0;
    st = ssu_prompts_workspace_bytes(handle, shape, tokens, &need);
    if (st != SSU_OK) return st;
    if (workspace_bytes < need || (need && !workspace))
        return fail(SSU_ERR_INVALID_ARG, "workspace holds %lld bytes; this shape needs %lld",
                    (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (need && !aligned(workspace, 256))
        return fail(SSU_ERR_MISALIGNED, "workspace is not 256-byte aligned");

    PromptParams q{};
    SsuParams &p = q.p;
    p.state = state_pool;
    p.idx = state_batch_indices;
    p.x = reinterpret_cast<const __nv_bfloat16 *>(x);
    p.dt = reinterpret_cast<const __nv_bfloat16 *>(dt);
    p.dt_bias = dt_bias;
    p.A = A;
    p.B = reinterpret_cast<const __nv_bfloat16 *>(B);
    p.C = reinterpret_cast<const __nv_bfloat16 *>(C);
    p.D = D;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.st_pool = strides->state[0];
    p.st_head = strides->state[1];
    p.st_row = strides->state[2];
    p.x_b = strides->x[0];
    p.x_h = strides->x[1];
    p.out_b = strides->out[0];
    p.out_h = strides->out[1];
    p.dt_b = strides->dt[0];
    p.dt_h = strides->dt[1];
    p.B_b = strides->B[0];
    p.B_g = strides->B[1];
    p.C_b = strides->C[0];
    p.C_g = strides->C[1];
    p.bias_h = strides->dt_bias[0];
    p.D_h = strides->D[0];
    p.A_h = strides->A[0];
    p.idx_s = strides->idx;
    p.pool_size = s.pool_size;
    p.batch = s.batch;
    p.nheads = static_cast<int>(s.nheads);
    p.headdim = static_cast<int>(s.headdim);
    p.heads_per_group = static_cast<int>(s.nheads / s.ngroups);
    p.group_magic = group_magic(static_cast<unsigned>(p.heads_per_group));
    p.err = handle->err;
    q.cu = cu_tokens;
    q.fresh = fresh;
    q.tokens = tokens;
    const int epv = s.state_dtype == SSU_STATE_BF16 ? 8 : 4;
    q.bc_vec = aligned(B, 2 * epv) && p.B_b % epv == 0 && p.B_g % epv == 0 &&
               aligned(C, 2 * epv) && p.C_b % epv == 0 && p.C_g % epv == 0;

    DeviceGuard guard(handle->device);
    if (guard.err != cudaSuccess)
        return fail(SSU_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(guard.err));
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = s.state_dtype == SSU_STATE_BF16, i64 = s.index_dtype == SSU_INDEX_I64;
    cudaError_t e = cudaErrorNotSupported;
    if (tokens > 0 && mma_sizes(s, tokens) && mma_operands(q)) {
        const PromptPlan w = prompt_plan(s, tokens, handle->sm_count);
        PromptMmaParams m{};
        m.q = q;
        m.seg = static_cast<int>(w.seg);
        m.after_first = w.earlier > 0 && handle->pdl;
        m.slabs = static_cast<int>(s.headdim / kSlab);
        m.local = static_cast<float *>(workspace);
        char *const room = static_cast<char *>(workspace);
        m.decay = reinterpret_cast<float *>(room + w.decay);
        m.hand = reinterpret_cast<float *>(room + w.hand);
        m.turn = reinterpret_cast<unsigned *>(room + w.turn);
        CUtensorMap maps[4];
        if (mma_grids(w) &&
            encode_map(&maps[0], x, s.headdim, s.nheads, tokens, p.x_h, p.x_b,
                       kChunk) &&
            encode_map(&maps[1], B, s.dstate, s.ngroups, tokens, p.B_g, p.B_b,
                       kChunk) &&
            encode_map(&maps[2], C, s.dstate, s.ngroups, tokens, p.C_g, p.C_b,
                       kChunk) &&
            encode_map(&maps[3], out, s.headdim, s.nheads, tokens, p.out_h, p.out_b,
                       kChunk))
            e = launch_mma(m, w, maps, static_cast<int>(s.dstate), bf16, i64, *handle, cs);
    }
    if (e == cudaErrorNotSupported)
        e = launch_seq(q, static_cast<int>(s.dstate), bf16, i64, handle->pdl, cs);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
