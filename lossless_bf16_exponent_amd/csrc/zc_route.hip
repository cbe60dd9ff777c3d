// Routing of tokens to experts and its gradient, MI355X / gfx950.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias,  group score = sum of a group's
//   best one or two c,  top_k largest c inside the best groups,  w = scale * s
//   (/ sum of the chosen s).
//
// The choice is that of 64-bit scores: a 32-bit exponential would decide near
// ties by its rounding.  Two kernels make it:
//   rank_kernel   one wave a token, every score in 64 bits;
//   route_kernel  16 lanes a token, scores in 32 bits with a bound on their
//                 error.  The bound leaves few candidates for the top_k places,
//                 and only those are scored and ranked in 64 bits.  A token whose
//                 groups the bound cannot tell apart, or with more than 16
//                 candidates, goes through the first one's code in place.
// Softmax weights that are not renormalised, and softmax with a bias, have no such
// bound and take the first: 8192 tokens of 256 experts in 8 groups 31.5 us there,
// 10 to 13 in the second.
#include <type_traits>

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
    uint32_t first = 0;  // first token of the launch
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

// LDS traffic between the lanes of a wave: accesses complete in order; the
// clobber keeps the compiler from moving them across.
__device__ __forceinline__ void lanes_meet() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A token by one wave, every score in 64 bits (expert e in lane e mod 64).  cs:
// room for the token's scores in LDS.
template <uint32_t R, bool BF16>
__device__ __forceinline__ void rank_token(const RouteArgs &a, uint64_t row, uint32_t lane, double *cs) {
    const uint32_t E = a.cfg.experts, G = a.cfg.groups, K = a.cfg.top_k;
    double s[R], c[R];
    scores<R, BF16>(a, row, lane, s);
    uint64_t key[R];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) {
        const uint32_t e = lane + 64u * i;
        c[i] = s[i] + (a.bias && e < E ? (double)a.bias[e] : 0.0);
        key[i] = e < E ? order_of(c[i]) : 0u;
    }
    if (G > 1) {
        // every group's best scores, one lane a group
        lanes_meet();
#pragma unroll
        for (uint32_t i = 0; i < R; ++i)
            if (lane + 64u * i < E) cs[lane + 64u * i] = c[i];
        lanes_meet();
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
        lanes_meet();
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

template <uint32_t R, bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void rank_kernel(RouteArgs a) {
    __shared__ double cs[kRouteWaves][R * 64];
    const uint32_t wave = threadIdx.x / 64;
    for (uint64_t row = (uint64_t)blockIdx.x * kRouteWaves + wave; row < a.tokens;
         row += (uint64_t)gridDim.x * kRouteWaves)
        rank_token<R, BF16>(a, row, lane_id(), cs[wave]);
}

// ---------------------------------------------------------------------------
// 16 lanes a token
// ---------------------------------------------------------------------------

constexpr uint32_t kRow = 16;                    // lanes of a token: a row of the wave, which DPP moves rotate
constexpr uint32_t kRowTokens = kLanes / kRow;   // tokens of a wave
constexpr uint32_t kCandidates = 16;

template <int N>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true);  // row_ror:N
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __uint_as_float(rotated<1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(rotated<2>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(rotated<4>(__float_as_uint(v))));
    return fmaxf(v, __uint_as_float(rotated<8>(__float_as_uint(v))));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(rotated<1>(__float_as_uint(v)));
    v += __uint_as_float(rotated<2>(__float_as_uint(v)));
    v += __uint_as_float(rotated<4>(__float_as_uint(v)));
    return v + __uint_as_float(rotated<8>(__float_as_uint(v)));
}
// Exclusive sum over the lanes of a row before this one (shifts inside the row
// bring zeros).
__device__ __forceinline__ uint32_t row_before(uint32_t v) {
    uint32_t s = v;
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x111, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x112, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x114, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x118, 0xF, 0xF, false);
    return s - v;
}

struct Candidate {
    double c;
    uint32_t id, pad;
};

template <uint32_t R>
struct RouteShared {
    union {
        float approx[kRowTokens][kRow * R + kRow * R / 32];  // a gap every 32: groups of 32 start in different banks
        Candidate cand[kRowTokens][kCandidates];
        double cs[R / 4 * 64];
    };
    uint16_t list[kRowTokens][kCandidates];
};

// The 32-bit scores a and what they certify, for the 64-bit scores c (softmax:
// e^(l - max), not divided by the sum, which comes here only with renormalised
// weights and without a bias: the order is the same and the sum cancels):
// |a - c| <= d(a) = 2^-22 + 2^-23 |a|.  With half steps h = 2^-24: the exponent x
// is off by at most 2.25 h |x|, which changes e^-|x| by at most 0.83 h since
// |x| e^-|x| < 0.37; the exponential adds 2 h, and for a sigmoid the sum and the
// reciprocal 3 h, of values of at most 1; adding the bias rounds by h |a|.
//   candidates  if t is the K-th largest a, K experts have c >= t - d(t), so
//               every expert among the K best has a >= t - 2 d(t) or so
//   groups      a group's score, the sum b1 + b2 of its two largest a, is off by at
//               most d(b1) + d(b2) and the sum's rounding, h (|b1| + |b2|): the sizes of
//               the addends, which may cancel, not that of the sum.  (a + d(a) and
//               a - d(a) grow with a, so this holds whichever two the c put first.)
//               The kept groups are certain when the lowest that one of them may be
//               lies above the highest that another may be.  The comparison takes
//               3 h (|b1| + |b2|) in place of 2 (for one score 2 h |b1| in place of 1),
//               for the roundings of its own sums, and a sixteenth more, for those of
//               the bounds.  Else the two experts of every group are scored in 64
//               bits, if they are certain themselves
constexpr float kOff = 0x1p-22f, kOffRel = 0x1p-23f;

template <uint32_t R, bool BF16>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, uint64_t first, RouteShared<R> &sh) {
    const uint32_t lane = lane_id(), sub = lane % kRow, tok = lane / kRow;
    const uint32_t E = a.cfg.experts, G = a.cfg.groups, K = a.cfg.top_k;
    const bool sigmoid = a.cfg.score == ZC_SCORE_SIGMOID;
    const float ninf = -__builtin_inff();
    const bool live = first + tok < a.tokens;
    const uint64_t row = live ? first + tok : a.tokens - 1;

    // experts sub * R .. sub * R + R - 1
    float l[R], v[R];
    const uint32_t e0 = sub * R;
    const uint64_t at = row * a.stride + e0;
    const bool wide = e0 + R <= E && (reinterpret_cast<uintptr_t>(a.logits) & (BF16 ? 7 : 15)) == 0 && a.stride % 4 == 0;
    float bias[R];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) bias[i] = 0.0f;
    if (a.bias) {
        if (e0 + R <= E && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
#pragma unroll
            for (uint32_t i = 0; i < R; i += 4) {
                const u32v4 w = *reinterpret_cast<const u32v4 *>(a.bias + e0 + i);
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) bias[i + j] = __uint_as_float(w[j]);
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < R; ++i) bias[i] = e0 + i < E ? a.bias[e0 + i] : 0.0f;
        }
    }
    if (wide) {
#pragma unroll
        for (uint32_t i = 0; i < R; i += 4) {
            if (BF16) {
                const u32v2 w = *reinterpret_cast<const u32v2 *>(static_cast<const uint16_t *>(a.logits) + at + i);
                l[i] = bf_lo(w[0]), l[i + 1] = bf_hi(w[0]), l[i + 2] = bf_lo(w[1]), l[i + 3] = bf_hi(w[1]);
            } else {
                const u32v4 w = *reinterpret_cast<const u32v4 *>(static_cast<const float *>(a.logits) + at + i);
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) l[i + j] = __uint_as_float(w[j]);
            }
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) l[i] = e0 + i < E ? logit<BF16>(a.logits, at + i) : ninf;
    }
    bool slow = false;
    float inv = 1.0f, top = 0.0f;
    if (sigmoid) {
#pragma unroll
        for (uint32_t i = 0; i < R; ++i)
            v[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -1.44269504f));
    } else {
        float m = l[0], sum = 0.0f;
#pragma unroll
        for (uint32_t i = 1; i < R; ++i) m = fmaxf(m, l[i]);
        top = row_max(m);
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) {
            v[i] = __builtin_amdgcn_exp2f((l[i] - top) * 1.44269504f);
            sum += v[i];
        }
        sum = row_sum(sum);
        slow = !(sum >= 1.0f && sum < 2048.0f);  // NaN or infinities, or nothing but -inf
        inv = __builtin_amdgcn_rcpf(sum);
    }
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) {
        v[i] += bias[i];
        v[i] = e0 + i < E && v[i] == v[i] ? v[i] : ninf;
    }

    if (G > 1) {
        const uint32_t per = E / G;
        float *mine = sh.approx[tok];
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) mine[e0 + i + (e0 + i) / 32] = v[i];
        lanes_meet();
        const bool two = a.cfg.group_score == 2 && per > 1;
        const float *group = mine;
        float score = ninf, off = 0.0f;
        if (sub < G) {
            float b1 = ninf, b2 = ninf;
#pragma unroll 8
            for (uint32_t j = 0; j < per; ++j) {
                const uint32_t e = sub * per + j;
                const float x = group[e + e / 32];
                b2 = fmaxf(b2, fminf(b1, x));
                b1 = fmaxf(b1, x);
            }
            score = two ? b1 + b2 : b1;
            off = 1.0625f * (two ? 2.0f * kOff + 1.5f * kOffRel * (fabsf(b1) + fabsf(b2)) : kOff + kOffRel * fabsf(b1));
        }
        // a group stays when fewer than group_top come before it: one other group a rotation of the row.  Every lane takes
        // part, those past the last group with their -inf: a rotation brings 0 from a lane that is switched off, and a 0
        // would come before a group whose score is negative
        const auto places = [&](auto mine_score, auto rotate) -> uint32_t {
            uint32_t before = 0;
            const auto meet = [&](auto o, uint32_t other) {
                before += o > mine_score || (o == mine_score && other < sub);
            };
            meet(rotate(std::integral_constant<int, 1>{}), (sub - 1) & 15);
            meet(rotate(std::integral_constant<int, 2>{}), (sub - 2) & 15);
            meet(rotate(std::integral_constant<int, 3>{}), (sub - 3) & 15);
            meet(rotate(std::integral_constant<int, 4>{}), (sub - 4) & 15);
            meet(rotate(std::integral_constant<int, 5>{}), (sub - 5) & 15);
            meet(rotate(std::integral_constant<int, 6>{}), (sub - 6) & 15);
            meet(rotate(std::integral_constant<int, 7>{}), (sub - 7) & 15);
            meet(rotate(std::integral_constant<int, 8>{}), (sub - 8) & 15);
            meet(rotate(std::integral_constant<int, 9>{}), (sub - 9) & 15);
            meet(rotate(std::integral_constant<int, 10>{}), (sub - 10) & 15);
            meet(rotate(std::integral_constant<int, 11>{}), (sub - 11) & 15);
            meet(rotate(std::integral_constant<int, 12>{}), (sub - 12) & 15);
            meet(rotate(std::integral_constant<int, 13>{}), (sub - 13) & 15);
            meet(rotate(std::integral_constant<int, 14>{}), (sub - 14) & 15);
            meet(rotate(std::integral_constant<int, 15>{}), (sub - 15) & 15);
            return before;
        };
        const auto row_any = [&](bool b) { return ((__ballot(b) >> (kRow * tok)) & 0xFFFFu) != 0; };
        const uint32_t place = places(score, [&](auto n) {
            return __uint_as_float(rotated<decltype(n)::value>(__float_as_uint(score)));
        });
        bool keep = sub < G && place < a.cfg.group_top;
        if (a.cfg.group_top < G) {
            const float low = -row_max(keep ? off - score : ninf), high = row_max(sub < G && !keep ? score + off : ninf);
            // (infinities have no distance from each other, and a group that holds those of both signs has no score)
            const bool unsure = row_any(sub < G && !(fabsf(score) < 3.0e38f)) || !(low > high);
            if (__ballot(unsure)) {
                float b1 = ninf, b2 = ninf, b3 = ninf;
                uint32_t i1 = 0, i2 = 0;
                if (sub < G)
                    for (uint32_t j = 0; j < per; ++j) {
                        const uint32_t e = sub * per + j;
                        const float x = group[e + e / 32];
                        if (x > b1) {
                            b3 = b2, b2 = b1, i2 = i1;
                            b1 = x, i1 = e;
                        } else if (x > b2) {
                            b3 = b2;
                            b2 = x, i2 = e;
                        } else if (x > b3) {
                            b3 = x;
                        }
                    }
                const float in = two ? b2 : b1, out = two ? b3 : b2;
                const bool sure = sub >= G || in - out > 2.0f * (2.0f * kOff + kOffRel * (fabsf(in) + fabsf(out))) ||
                                  (per == (two ? 2u : 1u) && fabsf(in) < 3.0e38f);
                const auto exact = [&](uint32_t e) -> double {
                    const double x = (double)logit<BF16>(a.logits, row * a.stride + e);
                    return sigmoid ? 1.0 / (1.0 + exp(-x)) + (a.bias ? (double)a.bias[e] : 0.0) : exp(x - (double)top);
                };
                double score64 = -__builtin_inf();
                if (sub < G) score64 = exact(i1) + (two ? exact(i2) : 0.0);
                const uint64_t bits = __builtin_bit_cast(uint64_t, score64);
                const uint32_t place64 = places(score64, [&](auto n) {
                    const uint64_t hi = rotated<decltype(n)::value>((uint32_t)(bits >> 32));
                    return __builtin_bit_cast(double, hi << 32 | rotated<decltype(n)::value>((uint32_t)bits));
                });
                if (unsure) {
                    keep = sub < G && place64 < a.cfg.group_top;
                    slow |= row_any(!sure || score64 != score64);
                }
            }
        }
        const uint32_t kept = (uint32_t)(__ballot(keep) >> (kRow * tok)) & 0xFFFFu;
        lanes_meet();
        const uint32_t magic = (1u << 20) / per + 1;  // e / per = e * magic >> 20 for e below 2^10
#pragma unroll
        for (uint32_t i = 0; i < R; ++i)
            if (!((kept >> (((e0 + i) * magic >> 20) & 31u)) & 1u)) v[i] = ninf;
    }

    // the K-th largest (equal ones count once, which only lowers it)
    float w[R], t = ninf;
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) w[i] = v[i];
    for (uint32_t k = 0; k < K; ++k) {
        float m[R / 4];
#pragma unroll
        for (uint32_t i = 0; i < R / 4; ++i)
            m[i] = fmaxf(fmaxf(w[4 * i], w[4 * i + 1]), fmaxf(w[4 * i + 2], w[4 * i + 3]));
#pragma unroll
        for (uint32_t i = 1; i < R / 4; ++i) m[0] = fmaxf(m[0], m[i]);
        t = row_max(m[0]);
#pragma unroll
        for (uint32_t i = 0; i < R; ++i) w[i] = w[i] == t ? ninf : w[i];
    }
    const float bound = t - 2.5f * (kOff + kOffRel * fabsf(t));
    uint32_t marks = 0;
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) marks |= v[i] >= bound ? 1u << i : 0u;
    const uint32_t n = (uint32_t)__builtin_popcount(marks), before = row_before(n);
    const uint32_t total = (uint32_t)__shfl((int)(before + n), (int)(lane | (kRow - 1)));
    slow |= !(fabsf(bound) < 3.0e38f) || total > kCandidates || total < K;
    if (!slow) {
        uint32_t slot = before;
        for (uint32_t rest = marks; rest; rest &= rest - 1) sh.list[tok][slot++] = (uint16_t)(e0 + __builtin_ctz(rest));
    }
    lanes_meet();
    const bool have = !slow && sub < total;
    const uint32_t id = have ? sh.list[tok][sub] : 0;
    const double x = have ? (double)logit<BF16>(a.logits, row * a.stride + id) : 0.0;
    // softmax: e^(l - max), which orders as the scores do
    const double s = sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top);
    const double c = sigmoid && a.bias && have ? s + (double)a.bias[id] : s;
    sh.cand[tok][sub] = Candidate{have ? c : -__builtin_inf(), have ? id : ~0u, 0u};
    lanes_meet();
    uint32_t rank = 0;
    for (uint32_t j = 0; j < kCandidates; ++j) {
        const Candidate o = sh.cand[tok][j];
        rank += o.c > c || (o.c == c && o.id < id);
    }
    const bool chosen = have && rank < K;
    const float p = chosen ? (float)(sigmoid ? s : s * (double)inv) : 0.0f;
    const float sum = row_sum(p);
    if (chosen && live) {
        const float weight = a.cfg.renormalise ? p / (sum + 1e-20f) : p;
        a.ids[row * K + rank] = (int32_t)id;
        a.weights[row * K + rank] = weight * a.cfg.scale;
    }
    // tokens that 32 bits cannot decide, one after another
    for (uint64_t left = __ballot(slow && live && sub == 0); left; left &= left - 1) {
        const uint32_t which = (uint32_t)__builtin_ctzll(left) / kRow;
        lanes_meet();
        rank_token<R / 4, BF16>(a, first + which, lane, sh.cs);
    }
}

// Four tokens a wave; the waves do not wait for each other.  Bound by the latency
// of a wave's steps, one after another: 1 token of 256 experts in 8 groups takes
// 7.1 us, 8192 tokens (two waves a SIMD) 10 to 13, where their bytes need 1.7; one
// wave a token with every score in 64 bits took 28.  No loop over tokens: around
// this body it costs a tenth of a call of one token (7.4 -> 8.3 us).
template <uint32_t R, bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
    __shared__ RouteShared<R> shared[kRouteWaves];
    const uint32_t wave = threadIdx.x / 64;
    const uint64_t first = a.first + ((uint64_t)blockIdx.x * kRouteWaves + wave) * kRowTokens;
    if (first < a.tokens) route_tokens<R, BF16>(a, first, shared[wave]);
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
// Bound by latency as the forward is: 8191 tokens of 128 experts take 7.0 us.
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

// 16 lanes a token where the 32-bit bound applies (see route_kernel), up to 512
// experts, 16 groups and 15 places; one wave a token else.
static bool certifiable(const RouteArgs &a) {
    const zc_route_config &c = a.cfg;
    return c.experts <= 512 && c.groups <= kRow && c.top_k < kCandidates &&
           (c.score == ZC_SCORE_SIGMOID || (c.renormalise && !a.bias));
}

template <uint32_t R, bool BF16>
static void launch_route(const RouteArgs &a, Launches &on) {
    const dim3 block(kRouteWaves * 64);
    if constexpr (R <= 8) {
        if (certifiable(a)) {
            // A grid holds less than 2^32 threads.
            constexpr uint64_t most = 1u << 20;
            RouteArgs part = a;
            for (uint64_t first = 0; first < a.tokens; first += most * kRouteWaves * kRowTokens) {
                const uint64_t blocks = ceil_div(a.tokens - first, kRouteWaves * kRowTokens);
                part.first = (uint32_t)first;
                on.launch((route_kernel<4 * R, BF16>), dim3((uint32_t)(blocks < most ? blocks : most)), block, part);
            }
            return;
        }
    }
    on.launch((rank_kernel<R, BF16>), dim3(route_blocks(a.tokens)), block, a);
}

template <uint32_t R>
static void launch_route(const RouteArgs &a, bool bf16, Launches &on) {
    if (bf16)
        launch_route<R, true>(a, on);
    else
        launch_route<R, false>(a, on);
}

template <uint32_t R>
static void launch_route_backward(const RouteBackArgs &a, bool bf16, Launches &on) {
    const dim3 grid(route_blocks(a.f.tokens)), block(kRouteWaves * 64);
    if (bf16)
        on.launch((route_backward_kernel<R, true>), grid, block, a);
    else
        on.launch((route_backward_kernel<R, false>), grid, block, a);
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
    Launches on(stream);
    if (cfg->experts <= 64)
        launch_route<1>(a, bf16, on);
    else if (cfg->experts <= 128)
        launch_route<2>(a, bf16, on);
    else if (cfg->experts <= 256)
        launch_route<4>(a, bf16, on);
    else if (cfg->experts <= 512)
        launch_route<8>(a, bf16, on);
    else
        launch_route<16>(a, bf16, on);
    return on.status();
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
    Launches on(stream);
    if (cfg->experts <= 64)
        launch_route_backward<1>(a, bf16, on);
    else if (cfg->experts <= 128)
        launch_route_backward<2>(a, bf16, on);
    else if (cfg->experts <= 256)
        launch_route_backward<4>(a, bf16, on);
    else if (cfg->experts <= 512)
        launch_route_backward<8>(a, bf16, on);
    else
        launch_route_backward<16>(a, bf16, on);
    return on.status();
}
