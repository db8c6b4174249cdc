// Prompts, token by token (sm_103a), instantiated by ssu_prompt.cu: the form that is right for
// every shape.
//
// Each warp keeps SLOTS * RPI rows of one head's state in registers (the row geometry of
// ssu_device.cuh) and applies the decode step to them for every token of the prompt in turn, so
// the state is read and written once per prompt.  What bounds it: the chain of one token after
// the other in a warp (update, readout tree), not bytes.

#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssu_device.cuh"

namespace {

struct PromptParams {
    SsuParams p;  // x_b, out_b, dt_b, B_b and C_b are the token strides; batch = prompts
    const void *cu;
    const unsigned char *fresh;
    long long tokens;
    int bc_vec;  // B and C rows can be read as whole column groups (aligned vectors)
};

// Prompt b's slot and tokens; false (and counted, once per call of this by `counts`) where they
// are out of range.
template <bool kIdx64>
__device__ __forceinline__ bool load_prompt(const PromptParams &q, long long b, bool counts,
                                            long long &slot, long long &begin, long long &end) {
    slot = load_slot<kIdx64>(q.p, b);
    if (kIdx64) {
        begin = __ldg(static_cast<const long long *>(q.cu) + b);
        end = __ldg(static_cast<const long long *>(q.cu) + b + 1);
    } else {
        begin = __ldg(static_cast<const int *>(q.cu) + b);
        end = __ldg(static_cast<const int *>(q.cu) + b + 1);
    }
    const bool good = slot >= 0 && slot < q.p.pool_size && begin >= 0 && begin <= end &&
                      end <= q.tokens;
    if (!good && counts) record_skip(q.p, b);
    return good;
}

template <int SLOTS, int N, typename ST, bool kIdx64>
__global__ void __launch_bounds__(128) ssu_prompt_seq_kernel(PromptParams q) {
    pdl_wait();
    using G = RowGeo<N, ST>;
    const SsuParams &p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y;
    const int row0 = blockIdx.x * p.rows_per_cta + warp * SLOTS * G::RPI;
    if (row0 >= p.headdim) return;
    const int grp = group_of(h, p.group_magic);
    const float bias = __ldg(p.dt_bias + h * p.bias_h), A = __ldg(p.A + h * p.A_h);
    const float D = __ldg(p.D + h * p.D_h);
    const int col0 = col0_of<G>(lane), sub = sub_of<G>(lane);
    for (long long b = blockIdx.z; b < p.batch; b += gridDim.z) {
        long long slot, begin, end;
        const bool counts = h == 0 && row0 == 0 && lane == 0;
        if (!load_prompt<kIdx64>(q, b, counts, slot, begin, end)) continue;
        const bool fresh = q.fresh && q.fresh[b] != 0;
        if (begin == end && !fresh) continue;
        ST *state = static_cast<ST *>(p.state) + slot * p.st_pool + h * p.st_head + col0;
        float S[SLOTS][G::NC];
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            const int row = row0 + r * G::RPI + sub;
            RawRow<G> raw{};
            if (!fresh && row < p.headdim) load_raw<G>(state + row * p.st_row, raw);
            raw_to_f32<G, ST>(raw, S[r]);
        }
        for (long long t = begin; t < end; ++t) {
            float bb[G::NC], cc[G::NC], part[SLOTS];
            load_bc<G>(p.B + t * p.B_b + grp * p.B_g + col0, q.bc_vec, bb);
            load_bc<G>(p.C + t * p.C_b + grp * p.C_g + col0, q.bc_vec, cc);
            const float dtv =
                softplus_f32(__bfloat162float(p.dt[t * p.dt_b + h * p.dt_h]) + bias);
            const float dA = expf(dtv * A);
            const __nv_bfloat16 *xt = p.x + t * p.x_b + h * p.x_h;
#pragma unroll
            for (int r = 0; r < SLOTS; ++r) {
                const int row = row0 + r * G::RPI + sub;
                const float x = row < p.headdim ? __bfloat162float(xt[row]) : 0.0f;
                part[r] = update_lane<G::NC>(S[r], dA, dtv * x, bb, cc);
            }
            const float y = reduce_rows<SLOTS, G::L>(part, lane);
            const int row = row0 + slot_of_lane<SLOTS, G::L>(lane) * G::RPI + sub;
            if (writes_row<SLOTS, G::L>(lane) && row < p.headdim)
                p.out[t * p.out_b + h * p.out_h + row] =
                    __float2bfloat16(fmaf(D, __bfloat162float(xt[row]), y));
        }
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            const int row = row0 + r * G::RPI + sub;
            RawRow<G> raw;
            f32_to_raw<G, ST>(S[r], raw);
            if (row < p.headdim) store_raw<G>(state + row * p.st_row, raw);
        }
    }
}

}  // namespace
