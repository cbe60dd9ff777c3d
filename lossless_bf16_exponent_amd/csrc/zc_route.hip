// Routing of tokens to experts and its gradient, MI355X / gfx950.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias,  group score = sum of a group's
//   best one or two c,  top_k largest c inside the best groups,  w = scale * s
//   (/ sum of the chosen s).
//
// One wave holds a token's scores in registers (expert e in lane e mod 64).
// The choice is made on 64-bit scores: a 32-bit exponential would decide near
// ties by its rounding.
#include "zc_moe_device.h"

namespace zc {
namespace moe {

constexpr uint32_t kRouteWaves = 4;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    uint64_t stride;
    uint32_t tokens;
    zc_route_config cfg;
};

template <bool BF16>
__device__ __forceinline__ float logit(const void *p, uint64_t i) {
    return BF16 ? bf_one(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
    return v;
}
__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
    return v;
}

// A 64-bit score as an integer in the same order.  NaN and -inf share the
// lowest place (1; 0 is for experts that may not be chosen).
__device__ __forceinline__ uint64_t order_of(double c) {
    if (!(c > -__builtin_inf())) return 1u;
    const uint64_t u = __builtin_bit_cast(uint64_t, c + 0.0);  // -0 + 0 = +0: the zeros tie
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// Softmax or sigmoid scores of the token in this wave, 64 bits; experts past
// the end get 0.
template <uint32_t R, bool BF16>
__device__ __forceinline__ void scores(const RouteArgs &a, uint64_t row, uint32_t lane, double (&s)[R]) {
    const uint32_t E = a.cfg.experts;
    float l[R];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) {
        const uint32_t e = lane + 64u * i;
        l[i] = e < E ? logit<BF16>(a.logits, row * a.stride + e) : -__builtin_inff();
    }
    if (a.cfg.score == ZC_SCORE_SIGMOID) {
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
        float m = l[0];
#pragma unroll
        for (uint32_t i = 1; i < R; ++i) m = fmaxf(m, l[i]);
        m = wave_maxf(m);
        // a row of -inf only has no largest value to subtract: all scores 0
        const double shift = m > -__builtin_inff() ? (double)m : 0.0;
        double sum = 0.0;
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            s[i] = exp((double)l[i] - shift);
            sum += s[i];
        }
        sum = wave_sum(sum);
        const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) s[i] = s[i] * inv;
    }
}

template <uint32_t R, bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
    __shared__ uint64_t keys[kRouteWaves][R * 64];
    const uint32_t lane = lane_id(), wave = threadIdx.x / 64;
    const uint32_t E = a.cfg.experts, G = a.cfg.groups, K = a.cfg.top_k;
    for (uint64_t row = (uint64_t)blockIdx.x * kRouteWaves + wave; row < a.tokens;
         row += (uint64_t)gridDim.x * kRouteWaves) {
        double s[R];
        scores<R, BF16>(a, row, lane, s);
        uint64_t key[R];
        double c[R];
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            const uint32_t e = lane + 64u * i;
            c[i] = s[i] + (a.bias && e < E ? (double)a.bias[e] : 0.0);
            key[i] = e < E ? order_of(c[i]) : 0u;
        }
        if (G > 1) {
            // every group's best scores, one lane a group
            double *cs = reinterpret_cast<double *>(keys[wave]);
#pragma unroll
            for (uint32_t i = 0; i < R; ++i)
                if (lane + 64u * i < E) cs[lane + 64u * i] = c[i];
            __builtin_amdgcn_wave_barrier();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const uint32_t per = E / G;
            uint64_t gkey = 0;
            if (lane < G) {
                double b1 = -__builtin_inf(), b2 = -__builtin_inf();
                for (uint32_t j = 0; j < per; ++j) {
                    const double v = cs[lane * per + j];
                    if (v > b1) {
                        b2 = b1;
                        b1 = v;
                    } else if (v > b2) {
                        b2 = v;
                    }
                }
                gkey = order_of(a.cfg.group_score == 2 && per > 1 ? b1 + b2 : b1);
            }
            // a group stays when fewer than group_top groups come before it
            uint32_t before = 0;
            for (uint32_t g = 0; g < G; ++g) {
                const uint64_t other = __shfl(gkey, (int)g);
                before += other > gkey || (other == gkey && g < lane);
            }
            const uint64_t kept = __ballot(lane < G && before < a.cfg.group_top);
#pragma unroll
            for (uint32_t i = 0; i < R; ++i) {
                const uint32_t e = lane + 64u * i;
                if (e < E && !((kept >> (e / per)) & 1u)) key[i] = 0;
            }
        }
        float sum = 0.0f, mine = 0.0f;
        int32_t my_id = 0;
        for (uint32_t k = 0; k < K; ++k) {
            uint64_t best = key[0];
            uint32_t at = lane;
            double score = s[0];
#pragma unroll
            for (uint32_t i = 1; i < R; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = lane + 64u * i;
                    score = s[i];
                }
            float sc = (float)score;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t ob = __shfl_xor(best, d);
                const uint32_t oa = (uint32_t)__shfl_xor((int)at, d);
                const float os = __shfl_xor(sc, d);
                if (ob > best || (ob == best && oa < at)) {
                    best = ob;
                    at = oa;
                    sc = os;
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < R; ++i)
                if (at == lane + 64u * i) key[i] = 0;
            sum += sc;
            if (lane == k) {
                mine = sc;
                my_id = (int32_t)at;
            }
        }
        if (lane < K) {
            const float w = a.cfg.renormalise ? mine / (sum + 1e-20f) : mine;
            a.ids[row * K + lane] = my_id;
            a.weights[row * K + lane] = w * a.cfg.scale;
        }
    }
}

struct RouteBackArgs {
    RouteArgs f;  // ids holds the chosen experts; weights and bias unused
    const float *dweights;
    void *dlogits;
    uint64_t dstride;
};

// One wave a token: lane k holds chosen expert k, and the gradient of its score
//   renormalised: d = scale * (dw - sum(dw p) / S) / S,  else d = scale * dw;
// sigmoid: dl = d s (1 - s) at the chosen, 0 elsewhere;
// softmax: dl_i = s_i (d_i - sum d s), d_i = 0 for experts not chosen.
template <uint32_t R, bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void route_backward_kernel(RouteBackArgs a) {
    __shared__ float ds[kRouteWaves][R * 64];
    const uint32_t lane = lane_id(), wave = threadIdx.x / 64;
    const uint32_t E = a.f.cfg.experts, K = a.f.cfg.top_k;
    for (uint64_t row = (uint64_t)blockIdx.x * kRouteWaves + wave; row < a.f.tokens;
         row += (uint64_t)gridDim.x * kRouteWaves) {
        float l[R], s[R];
        float m = -__builtin_inff();
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            const uint32_t e = lane + 64u * i;
            l[i] = e < E ? logit<BF16>(a.f.logits, row * a.f.stride + e) : -__builtin_inff();
            m = fmaxf(m, l[i]);
        }
        const bool sigmoid = a.f.cfg.score == ZC_SCORE_SIGMOID;
        float inv = 1.0f;
        if (!sigmoid) {
            m = wave_maxf(m);
            const float shift = m > -__builtin_inff() ? m : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < R; ++i) {
                s[i] = expf(l[i] - shift);
                sum += s[i];
            }
            sum = group_sum<64>(sum);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        }
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            s[i] = sigmoid ? 1.0f / (1.0f + expf(-l[i])) : s[i] * inv;
            ds[wave][lane + 64u * i] = s[i];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const int32_t id = lane < K ? a.f.ids[row * K + lane] : -1;
        const bool on = id >= 0 && (uint32_t)id < E;
        const float p = on ? ds[wave][id] : 0.0f;
        float d = on ? a.dweights[row * K + lane] * a.f.cfg.scale : 0.0f;
        if (a.f.cfg.renormalise) {
            const float S = group_sum<64>(p) + 1e-20f;
            const float mean = group_sum<64>(d * p) / S;
            d = on ? (d - mean) / S : 0.0f;
        }
        const float dot = sigmoid ? 0.0f : group_sum<64>(d * p);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) ds[wave][lane + 64u * i] = 0.0f;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (on) ds[wave][id] = d;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            const uint32_t e = lane + 64u * i;
            const float di = ds[wave][e];
            float g = sigmoid ? di * s[i] * (1.0f / (1.0f + expf(l[i]))) : s[i] * (di - dot);
            if (s[i] == 0.0f) g = 0.0f;  // a masked row's d may have overflowed (its sum of scores is 0)
            if (e < E) {
                const uint64_t o = row * a.dstride + e;
                if (BF16)
                    static_cast<uint16_t *>(a.dlogits)[o] = bf_round(g);
                else
                    static_cast<float *>(a.dlogits)[o] = g;
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

static zc_status check_config(const zc_route_config *c) {
    if (!c || c->experts == 0 || c->experts > ZC_MAX_EXPERTS || c->groups == 0 || c->groups > ZC_MAX_EXPERT_GROUPS ||
        c->experts % c->groups || c->group_top == 0 || c->group_top > c->groups ||
        (c->group_score != 1 && c->group_score != 2) || c->renormalise > 1 || c->score > ZC_SCORE_SIGMOID ||
        c->top_k == 0 || c->top_k > ZC_MAX_TOP_K || c->top_k > c->group_top * (c->experts / c->groups) ||
        !(c->scale - c->scale == 0.0f))
        return ZC_ERR_INVALID_ARG;
    return ZC_OK;
}

static zc_status check_rows(const void *logits, uint32_t type, uint64_t tokens, uint64_t stride,
                            const zc_route_config *cfg) {
    const zc_status s = check_config(cfg);
    if (s != ZC_OK) return s;
    if ((type != ZC_F32 && type != ZC_BF16) || tokens > kMaxRows || tokens * cfg->top_k > kMaxRows ||
        (tokens && !logits) || stride < cfg->experts || stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    return aligned(logits, type == ZC_F32 ? 4 : 2) ? ZC_OK : ZC_ERR_MISALIGNED;
}

static uint32_t route_blocks(uint64_t tokens) {
    const uint64_t b = ceil_div(tokens, kRouteWaves);
    return (uint32_t)(b < 8192 ? b : 8192);
}

template <uint32_t R>
static void launch_route(const RouteArgs &a, bool bf16, hipStream_t st) {
    const dim3 grid(route_blocks(a.tokens)), block(kRouteWaves * 64);
    if (bf16)
        hipLaunchKernelGGL((route_kernel<R, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((route_kernel<R, false>), grid, block, 0, st, a);
}

template <uint32_t R>
static void launch_route_backward(const RouteBackArgs &a, bool bf16, hipStream_t st) {
    const dim3 grid(route_blocks(a.f.tokens)), block(kRouteWaves * 64);
    if (bf16)
        hipLaunchKernelGGL((route_backward_kernel<R, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((route_backward_kernel<R, false>), grid, block, 0, st, a);
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" zc_status zc_route(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                              const float *d_bias, const zc_route_config *cfg, int32_t *d_ids, float *d_weights,
                              void *stream) {
    const zc_status s = check_rows(d_logits, logits_type, tokens, logits_stride, cfg);
    if (s != ZC_OK) return s;
    if (tokens && (!d_ids || !d_weights)) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_bias, 4) || !aligned(d_ids, 4) || !aligned(d_weights, 4)) return ZC_ERR_MISALIGNED;
    if (!tokens) return ZC_OK;
    const RouteArgs a = {d_logits, d_bias, d_ids, d_weights, logits_stride, (uint32_t)tokens, *cfg};
    const bool bf16 = logits_type == ZC_BF16;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (cfg->experts <= 64)
        launch_route<1>(a, bf16, st);
    else if (cfg->experts <= 128)
        launch_route<2>(a, bf16, st);
    else if (cfg->experts <= 256)
        launch_route<4>(a, bf16, st);
    else if (cfg->experts <= 512)
        launch_route<8>(a, bf16, st);
    else
        launch_route<16>(a, bf16, st);
    return launched();
}

extern "C" zc_status zc_route_backward(const void *d_logits, uint32_t logits_type, uint64_t tokens,
                                       uint64_t logits_stride, const zc_route_config *cfg, const int32_t *d_ids,
                                       const float *d_dweights, void *d_dlogits, uint64_t dlogits_stride,
                                       void *stream) {
    const zc_status s = check_rows(d_logits, logits_type, tokens, logits_stride, cfg);
    if (s != ZC_OK) return s;
    if ((tokens && (!d_ids || !d_dweights || !d_dlogits)) || dlogits_stride < cfg->experts ||
        dlogits_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!aligned(d_ids, 4) || !aligned(d_dweights, 4) || !aligned(d_dlogits, logits_type == ZC_F32 ? 4 : 2))
        return ZC_ERR_MISALIGNED;
    if (!tokens) return ZC_OK;
    const RouteArgs f = {d_logits, nullptr, const_cast<int32_t *>(d_ids), nullptr, logits_stride, (uint32_t)tokens,
                         *cfg};
    const RouteBackArgs a = {f, d_dweights, d_dlogits, dlogits_stride};
    const bool bf16 = logits_type == ZC_BF16;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (cfg->experts <= 64)
        launch_route_backward<1>(a, bf16, st);
    else if (cfg->experts <= 128)
        launch_route_backward<2>(a, bf16, st);
    else if (cfg->experts <= 256)
        launch_route_backward<4>(a, bf16, st);
    else if (cfg->experts <= 512)
        launch_route_backward<8>(a, bf16, st);
    else
        launch_route_backward<16>(a, bf16, st);
    return launched();
}
