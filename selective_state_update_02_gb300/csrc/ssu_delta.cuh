// The gated delta rule token by token (sm_103a), instantiated by ssu_delta.cu: one new token per
// request (ssu_delta_update), and prompts in the form that is right for every shape.
//
// Mathematics.  With kn, qn the token's key and query (at length one, the query scaled), a its
// decay and beta its gate, S' = a S + e kn^T with e = beta (v - a S kn), and the readout is
//
//   S' qn = a (S qn) + e (kn . qn)
//
// so both products with the state are with what was loaded: one reduction tree gives S kn and S qn
// of all the warp's rows, and the state is stored as soon as e is known.  All of it is fp32.
//
// What bounds the one-token form: HBM, reading and writing the state once.  Rows are spread over
// lanes as in the decode step (RowGeo, ssu_device.cuh); all of a warp's state loads are in flight
// before anything else (256 requests of 32 heads of 128 x 128 fp32: 156 us, 1.02 of the measured copy
// rate).  What bounds prompts in this form: the chain of one token after the other in a warp (two
// products, a tree of shuffles, e back to the lanes), 0.42 us per token.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ssu_device.cuh"
#include "ssu_prompt.cuh"

namespace {

// v, k and q take the places of the decode step's x, B and C.
struct DeltaParams {
    PromptParams m;  // of it cu, fresh and tokens for prompts alone; bc_vec speaks of k and q
    const __nv_bfloat16 *beta;
    long long beta_t, beta_h;
    float scale, eps;  // eps < 0: q and k as they are
};

// A lane's columns of a key or query as loaded.
template <class G>
struct RawKey {
    unsigned w[G::NC / 2];
};

// `p` points at the lane's first column; `vec`: rows can be read as whole column groups.
template <class G>
__device__ __forceinline__ void load_key(const __nv_bfloat16 *p, bool vec, RawKey<G> &r) {
    const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
    if (vec) {
#pragma unroll
        for (int v = 0; v < G::VPR; ++v) {
            if constexpr (G::kEPV == 8) {
                const uint4 u = *reinterpret_cast<const uint4 *>(q + v * G::kVecStride);
                r.w[4 * v] = u.x, r.w[4 * v + 1] = u.y, r.w[4 * v + 2] = u.z, r.w[4 * v + 3] = u.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(q + v * G::kVecStride);
                r.w[2 * v] = u.x, r.w[2 * v + 1] = u.y;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < G::NC; e += 2) {
            const unsigned short *c = q + (e / G::kEPV) * G::kVecStride + e % G::kEPV;
            r.w[e / 2] = c[0] | static_cast<unsigned>(c[1]) << 16;
        }
    }
}

template <class G>
__device__ __forceinline__ void widen_key(const RawKey<G> &r, float (&o)[G::NC]) {
#pragma unroll
    for (int i = 0; i < G::NC / 2; ++i) {
        o[2 * i] = __uint_as_float(r.w[i] << 16);
        o[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
}

// What a token brings to every row: its key (at length one) and query (raw: the readout takes rq)
// at the lane's columns.
template <class G>
struct Token {
    float k[G::NC], q[G::NC];
    float a, beta;  // decay and gate
    float rq, kq;   // the query's factor; key times query, with it
};

template <class G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = G::L / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// A head's decay and gate at a token.
__device__ __forceinline__ float2 rates_of(float dt, float bias, float A, float b) {
    return make_float2(expf(softplus_f32(dt + bias) * A), 1.0f / (1.0f + expf(-b)));
}

// (Without branches, so that it can run beside another token's work; rsqrtf is within 2 ulp.)
template <class G>
__device__ __forceinline__ void make_token(const DeltaParams &d, const RawKey<G> &k,
                                           const RawKey<G> &q, float2 rates, Token<G> &t) {
    widen_key<G>(k, t.k);
    widen_key<G>(q, t.q);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int i = 0; i < G::NC; ++i) {
        kk = fmaf(t.k[i], t.k[i], kk);
        qq = fmaf(t.q[i], t.q[i], qq);
        kq = fmaf(t.k[i], t.q[i], kq);
    }
    kk = row_sum<G>(kk), qq = row_sum<G>(qq), kq = row_sum<G>(kq);
    const float rk = d.eps >= 0.0f ? rsqrtf(kk + d.eps) : 1.0f;
    t.rq = d.scale * (d.eps >= 0.0f ? rsqrtf(qq + d.eps) : 1.0f);
    // (A length past fp32 leaves zeros, which an overflowed product must not undo: finite, it becomes
    // zero with them.  An infinity or NaN in the key or query comes through its products with the
    // state.  Choosing zero by the factors left the step's loads 16 registers fewer and cost 0.7 %.)
    constexpr float kMost = 3.402823466e38f;
    t.kq = fminf(fmaxf(kq, -kMost), kMost) * rk * t.rq;
#pragma unroll
    for (int i = 0; i < G::NC; ++i) t.k[i] *= rk;
    t.a = rates.x;
    t.beta = rates.y;
}

// The lane of its row's group that reduce_rows<R, L> leaves the total of `slot` in.
template <int R, int L>
__host__ __device__ constexpr int lane_of_slot(int slot) {
    int lane = 0;
    for (int n = R, m = L / 2; n > 1; n >>= 1, m >>= 1)
        if (slot >= n / 2) lane |= m, slot -= n / 2;
    return lane;
}

// The row (of the warp's SLOTS * RPI) that the lane works e out for, and whether it is the lane
// that writes that row's readout.
template <class G, int SLOTS>
__device__ __forceinline__ int row_of_lane(int lane) {
    return slot_of_lane<2 * SLOTS, G::L>(lane) % SLOTS * G::RPI + sub_of<G>(lane);
}

template <class G, int SLOTS>
__device__ __forceinline__ bool reads_out(int lane) {
    return writes_row<2 * SLOTS, G::L>(lane) && !(lane & (G::L / 2));
}

// One token through SLOTS vector rows S; v is the value of the lane's row (row_of_lane).  Returns
// that row's readout.
template <class G, int SLOTS>
__device__ __forceinline__ float delta_rows(float (&S)[SLOTS][G::NC], const Token<G> &t, float v,
                                            int lane) {
    static_assert(2 * SLOTS <= G::L, "both products' totals have a lane each");
    float part[2 * SLOTS];
#pragma unroll
    for (int r = 0; r < SLOTS; ++r) {
        float2 sk = make_float2(0.0f, 0.0f), sq = sk;
#pragma unroll
        for (int i = 0; i < G::NC; i += 2) {
            const float2 s = make_float2(S[r][i], S[r][i + 1]);
            sk = __ffma2_rn(s, make_float2(t.k[i], t.k[i + 1]), sk);
            sq = __ffma2_rn(s, make_float2(t.q[i], t.q[i + 1]), sq);
        }
        part[r] = sk.x + sk.y;
        part[SLOTS + r] = sq.x + sq.y;
    }
    // lanes of the upper half of a row's group hold the readouts, the lower ones the predictions
    const float mine = reduce_rows<2 * SLOTS, G::L>(part, lane);
    const float other = __shfl_xor_sync(0xffffffffu, mine, G::L / 2);
    const bool upper = (lane & (G::L / 2)) != 0;
    const float sk = upper ? other : mine, sq = upper ? mine : other;
    const float e = t.beta * fmaf(-t.a, sk, v);
#pragma unroll
    for (int r = 0; r < SLOTS; ++r) {
        const float er = __shfl_sync(0xffffffffu, e, lane_of_slot<2 * SLOTS, G::L>(r), G::L);
        const float2 a2 = make_float2(t.a, t.a), e2 = make_float2(er, er);
#pragma unroll
        for (int i = 0; i < G::NC; i += 2) {
            const float2 w =
                __ffma2_rn(make_float2(S[r][i], S[r][i + 1]), a2,
                           __fmul2_rn(e2, make_float2(t.k[i], t.k[i + 1])));
            S[r][i] = w.x;
            S[r][i + 1] = w.y;
        }
    }
    return fmaf(t.a * t.rq, sq, e * t.kq);
}

// Grid: x = slab of rows, y = head, z = request (requests past gridDim.z loop).
template <int SLOTS, int N, typename ST, bool kIdx64>
__global__ void __launch_bounds__(128) ssu_delta_step_kernel(const __grid_constant__ DeltaParams d) {
    pdl_wait();
    using G = RowGeo<N, ST>;
    const SsuParams &p = d.m.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int row0 = blockIdx.x * p.rows_per_cta + warp * SLOTS * G::RPI;
    if (row0 >= p.headdim) return;
    const int col0 = col0_of<G>(lane), sub = sub_of<G>(lane);
    const int grp = group_of(h, p.group_magic);
    for (long long b = blockIdx.z; b < p.batch; b += gridDim.z) {
        const long long slot = load_slot<kIdx64>(p, b);
        if (slot < 0 || slot >= p.pool_size) {
            if (h == 0 && row0 == 0 && lane == 0) record_skip(p, b);
            continue;
        }
        ST *const state = static_cast<ST *>(p.state) + slot * p.st_pool + h * p.st_head +
                          (row0 + sub) * p.st_row + col0;
        const long long slot_stride = G::RPI * p.st_row;
        RawRow<G> raw[SLOTS];
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            if (row0 + sub + r * G::RPI < p.headdim)
                load_raw<G>(state + r * slot_stride, raw[r]);
            else
                raw[r] = RawRow<G>{};
        }
        RawKey<G> rk, rq;
        load_key<G>(p.B + b * p.B_b + grp * p.B_g + col0, d.m.bc_vec, rk);
        load_key<G>(p.C + b * p.C_b + grp * p.C_g + col0, d.m.bc_vec, rq);
        const int row = row0 + row_of_lane<G, SLOTS>(lane);
        const float v = row < p.headdim
                            ? __bfloat162float(p.x[b * p.x_b + h * p.x_h + row]) : 0.0f;
        const float dt = __bfloat162float(p.dt[b * p.dt_b + h * p.dt_h]);
        const float gate = __bfloat162float(d.beta[b * d.beta_t + h * d.beta_h]);
        Token<G> t;
        make_token<G>(d, rk, rq, rates_of(dt, p.dt_bias[h * p.bias_h], p.A[h * p.A_h], gate), t);
        float S[SLOTS][G::NC];
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) raw_to_f32<G, ST>(raw[r], S[r]);
        const float y = delta_rows<G, SLOTS>(S, t, v, lane);
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            f32_to_raw<G, ST>(S[r], raw[r]);
            if (row0 + sub + r * G::RPI < p.headdim)
                store_raw<G>(state + r * slot_stride, raw[r]);
        }
        if (reads_out<G, SLOTS>(lane) && row < p.headdim)
            p.out[b * p.out_b + h * p.out_h + row] = __float2bfloat16(y);
    }
    pdl_trigger();
}

// Prompts: a warp takes its rows through every token of a prompt, the next token's operands in
// flight meanwhile.
template <int SLOTS, int N, typename ST, bool kIdx64>
__global__ void __launch_bounds__(128) ssu_delta_seq_kernel(const __grid_constant__ DeltaParams d) {
    pdl_wait();
    using G = RowGeo<N, ST>;
    const SsuParams &p = d.m.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int row0 = blockIdx.x * p.rows_per_cta + warp * SLOTS * G::RPI;
    if (row0 >= p.headdim) return;
    const int grp = group_of(h, p.group_magic);
    const float bias = __ldg(p.dt_bias + h * p.bias_h), A = __ldg(p.A + h * p.A_h);
    const int col0 = col0_of<G>(lane), sub = sub_of<G>(lane);
    const int row = row0 + row_of_lane<G, SLOTS>(lane);
    for (long long b = blockIdx.z; b < p.batch; b += gridDim.z) {
        long long slot, begin, end;
        const bool counts = h == 0 && row0 == 0 && lane == 0;
        if (!load_prompt<kIdx64>(d.m, b, counts, slot, begin, end)) continue;
        const bool fresh = d.m.fresh && d.m.fresh[b] != 0;
        if (begin == end && !fresh) continue;
        ST *const state =
            static_cast<ST *>(p.state) + slot * p.st_pool + h * p.st_head + col0;
        float S[SLOTS][G::NC];
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            RawRow<G> raw{};
            const int at = row0 + sub + r * G::RPI;
            if (!fresh && at < p.headdim) load_raw<G>(state + at * p.st_row, raw);
            raw_to_f32<G, ST>(raw, S[r]);
        }
        // A token's operands are fetched kAhead tokens ahead and made ready, its lengths, beside the
        // chain of the token before; decays and gates are worked out for 32 tokens at a time, one
        // per lane.
        constexpr int kAhead = G::NC <= 4 ? 4 : 2;
        struct {
            RawKey<G> k, q;
            unsigned short v;
        } raw[kAhead] = {};
        auto wide = [](unsigned short u) {
            return __uint_as_float(static_cast<unsigned>(u) << 16);
        };
        auto fetch = [&](int i, long long t) {
            if (t >= end) return;
            load_key<G>(p.B + t * p.B_b + grp * p.B_g + col0, d.m.bc_vec, raw[i].k);
            load_key<G>(p.C + t * p.C_b + grp * p.C_g + col0, d.m.bc_vec, raw[i].q);
            if (row < p.headdim)
                raw[i].v =
                    reinterpret_cast<const unsigned short *>(p.x)[t * p.x_b + h * p.x_h + row];
        };
        float2 rates = make_float2(0.0f, 0.0f);  // of the lane's token
        auto rate = [&](long long t0) {
            const long long t = t0 + lane;
            if (t >= end) return;
            const unsigned short *const dt = reinterpret_cast<const unsigned short *>(p.dt);
            const unsigned short *const gate = reinterpret_cast<const unsigned short *>(d.beta);
            rates = rates_of(wide(dt[t * p.dt_b + h * p.dt_h]), bias, A,
                             wide(gate[t * d.beta_t + h * d.beta_h]));
        };
        Token<G> now, next;
        float value = 0.0f, after = 0.0f;
        auto prepare = [&](int i, int n) {  // the n-th token of those whose rates the lanes have
            make_token<G>(d, raw[i].k, raw[i].q,
                          make_float2(__shfl_sync(0xffffffffu, rates.x, n),
                                      __shfl_sync(0xffffffffu, rates.y, n)),
                          next);
            after = wide(raw[i].v);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i, begin + i);
        rate(begin);
        prepare(0, 0);
        for (long long t0 = begin; t0 < end; t0 += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const long long t = t0 + i;
                if (t >= end) break;
                const int n = static_cast<int>(t - begin + 1) & 31;
                if (n == 0) rate(t + 1);
                now = next;
                value = after;
                fetch(i, t + kAhead);
                prepare((i + 1) % kAhead, n);
                const float y = delta_rows<G, SLOTS>(S, now, value, lane);
                if (reads_out<G, SLOTS>(lane) && row < p.headdim)
                    p.out[t * p.out_b + h * p.out_h + row] = __float2bfloat16(y);
            }
        }
#pragma unroll
        for (int r = 0; r < SLOTS; ++r) {
            RawRow<G> raw;
            f32_to_raw<G, ST>(S[r], raw);
            const int at = row0 + sub + r * G::RPI;
            if (at < p.headdim) store_raw<G>(state + at * p.st_row, raw);
        }
    }
}

}  // namespace
