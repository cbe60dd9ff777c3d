// Balance of the experts, MI355X / gfx950: copies of every expert, balance loss and
// z loss of every sequence, and the logits' gradient:
//   loss = experts / (top_k n^2) sum_e c[e] sum_t p[t, e],  z = 1 / n sum_t lse(t)^2
//   d loss / d logit = experts / (top_k n^2) p_e (c_e - sum_j c_j p_j) [(1 - sigmoid_e) for sigmoid scores]
//   d z / d logit = 2 / n lse softmax_e
// Bound by reading the logits, and at a few thousand tokens by the latency of a
// token's steps.  A team of 16 lanes, or a wave, holds a token: lane l the experts l, l + its
// lanes, ...
#include <math.h>

#include <type_traits>

#include "zc_moe_device.h"

namespace zc {
namespace moe {

constexpr uint32_t kBWaves = 8;
constexpr uint32_t kBThreads = kBWaves * kLanes;

struct BalanceArgs {
    const void *logits, *add;
    void *dlogits;
    const int32_t *ids;
    const uint8_t *mask;
    const int32_t *offsets;
    uint32_t *parts;  // a tile's sums of p (floats), its counts, its z and its tokens: 2 experts + 2 words
    uint32_t *joins;  // a sequence's shares of the loss, z, tokens, and how many of its blocks are done
    int32_t *counts, *used;
    float *loss, *zloss;
    const float *dloss, *dzloss;
    uint64_t stride, add_stride, out_stride;
    uint32_t tokens, experts, top_k, sequences, tile_rows, run;
    double experts_each;  // experts / top_k
};

constexpr uint32_t kJoinZ = ZC_MAX_EXPERTS / kLanes, kJoinUsed = kJoinZ + 1, kJoinDone = kJoinUsed + 1, kJoinWords = kJoinDone + 1;

// Sum and maximum over a team, the same in all of its lanes: rotations of 8, 4, 2 and
// 1 inside a row of 16 lanes, and from row to row for a wave.
template <int BY>
__device__ __forceinline__ float rotated(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x120 + BY, 0xF, 0xF, false));
}
template <uint32_t LANES>
__device__ __forceinline__ float team_sum(float v) {
    if (LANES == kLanes) return wave_sum_f(v);
    v += rotated<8>(v);
    v += rotated<4>(v);
    v += rotated<2>(v);
    return v + rotated<1>(v);
}
template <uint32_t LANES>
__device__ __forceinline__ float team_max(float v) {
    v = fmaxf(v, rotated<8>(v));
    v = fmaxf(v, rotated<4>(v));
    v = fmaxf(v, rotated<2>(v));
    v = fmaxf(v, rotated<1>(v));
    if (LANES == kLanes) {
        v = fmaxf(v, __shfl_xor(v, 16));
        v = fmaxf(v, __shfl_xor(v, 32));
    }
    return v;
}

template <bool BF16>
__device__ __forceinline__ float value_at(const void *p, uint64_t i) {
    return BF16 ? bf_one(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
// A token's logits; -inf past the last expert.
template <bool BF16, uint32_t LANES, uint32_t V>
__device__ __forceinline__ void load_token(const BalanceArgs &a, uint64_t t, float (&l)[V]) {
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        const uint32_t e = lane_id() % LANES + LANES * i;
        l[i] = e < a.experts ? value_at<BF16>(a.logits, t * a.stride + e) : -__builtin_inff();
    }
}

// e^x to a unit or two of 32 bits: the product with log2(e) is carried on to its last digits, which the
// exponent of 2 alone would lose at |x| times as many.  NaN stays, and what is below e^-200 is 0.
__device__ __forceinline__ float exp_of(float v) {
    const float x = v < -200.0f ? -200.0f : v, t = x * 1.44269504f;
    const float rest = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269504f, -t)), e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, rest * 0.69314718f, e);
}

// Softmax of the team's logits, and the logarithm of its sum of exponentials: 0 and
// 0 where all are -inf.  NaN makes all of it NaN; +inf the softmax, and the logarithm is +inf.
template <uint32_t LANES, uint32_t V>
__device__ __forceinline__ float softmax(const float (&l)[V], float (&p)[V]) {
    float top = l[0];
#pragma unroll
    for (uint32_t i = 1; i < V; ++i) top = fmaxf(top, l[i]);
    top = team_max<LANES>(top);
    if (top == -__builtin_inff()) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        p[i] = exp_of(l[i] - top);
        sum += p[i];
    }
    sum = team_sum<LANES>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) p[i] *= inv;
    if (top == __builtin_inff()) {
        sum = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) sum += l[i] != l[i] ? l[i] : 0.0f;
        return top + team_sum<LANES>(sum);
    }
    return sum == 0.0f ? 0.0f : top + logf(sum);
}
// Sigmoids over their sum; rest: 1 - sigmoid.
template <uint32_t LANES, uint32_t V>
__device__ __forceinline__ void sigmoids(const float (&l)[V], float (&p)[V], float (&rest)[V]) {
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        const float t = exp_of(-fabsf(l[i])), r = __builtin_amdgcn_rcpf(1.0f + t), tr = t * r;
        p[i] = l[i] >= 0.0f ? r : tr;
        rest[i] = l[i] >= 0.0f ? tr : r;
        sum += p[i];
    }
    const float inv = 1.0f / (team_sum<LANES>(sum) + 1e-20f);
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) p[i] *= inv;
}

// The sums of one tile of a sequence's tokens.  Bound by the instructions of the tokens' steps: 65536 tokens,
// 160 experts, 37 sequences 38 us with a wave a token; its sums over the experts and its logarithm are shared by four with
// 16 lanes each: 19.5 us.
template <bool BF16, bool SIGMOID, uint32_t LANES, uint32_t V>
__global__ __launch_bounds__(kBThreads) void balance_tile_kernel(BalanceArgs a) {
    constexpr uint32_t kTeams = kLanes / LANES, kStep = kBWaves * kTeams;  // tokens of a wave, and of the block, at once
    __shared__ float sums[kBWaves][LANES * V];
    __shared__ uint32_t bins[LANES * V];
    __shared__ float zs[kBWaves];
    __shared__ uint32_t ns[kBWaves];
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t sub = lane % LANES;
    if (blockIdx.x == 0)  // no block of the next launch is done yet
        for (uint32_t q = threadIdx.x; q < a.sequences; q += kBThreads) a.joins[q * kJoinWords + kJoinDone] = 0;
    const Span sp = find_tile(a.offsets, a.sequences, a.tokens, a.tile_rows, [&](uint32_t) { return blockIdx.x; });
    if (!sp.found) return;
    const uint32_t t0 = sp.begin + sp.tile * a.tile_rows, t1 = min(t0 + a.tile_rows, sp.end);
    for (uint32_t e = threadIdx.x; e < LANES * V; e += kBThreads) bins[e] = 0;
    __syncthreads();
    float acc[V], z = 0.0f;
    uint32_t n = 0;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) acc[i] = 0.0f;
    const bool scored = a.loss || a.zloss;
    // a wave's next tokens are on their way while it works on these; those past the tile repeat its last one
    const uint32_t mine = lane / LANES;
    float next[V];
    uint32_t next_on = 0;
    const auto fetch = [&](uint32_t t) {
        const uint32_t u = min(t + mine, t1 - 1);
        if (scored) load_token<BF16, LANES, V>(a, u, next);
        next_on = a.mask ? a.mask[u] : 1;
    };
    fetch(t0 + wave * kTeams);
    const int32_t *ids = a.ids + (uint64_t)t0 * a.top_k;
    for (uint32_t i = threadIdx.x; i < (t1 - t0) * a.top_k; i += kBThreads) {
        const int32_t id = ids[i];
        if (id >= 0 && (uint32_t)id < a.experts && (!a.mask || a.mask[t0 + i / a.top_k])) atomicAdd(&bins[id], 1u);
    }
    for (uint32_t t = t0 + wave * kTeams; t < t1; t += kStep) {
        float l[V], p[V], rest[V], lse = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) l[i] = next[i];
        const bool live = t + mine < t1 && next_on;
        fetch(t + kStep);
        n += live;
        if (!scored) continue;
        if (!SIGMOID || a.zloss) lse = softmax<LANES, V>(l, p);
        if (SIGMOID) sigmoids<LANES, V>(l, p, rest);
        z = live ? fmaf(lse, lse, z) : z;
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) acc[i] += live ? p[i] : 0.0f;
    }
    // the teams of a wave, in order
    if (LANES == 16) {
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) {
            acc[i] += __shfl_xor(acc[i], 16);
            acc[i] += __shfl_xor(acc[i], 32);
        }
        z += __shfl_xor(z, 16);
        z += __shfl_xor(z, 32);
        n += (uint32_t)__shfl_xor((int)n, 16);
        n += (uint32_t)__shfl_xor((int)n, 32);
    }
    if (lane < LANES)
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) sums[wave][sub + LANES * i] = acc[i];
    if (lane == 0) {
        zs[wave] = z;
        ns[wave] = n;
    }
    __syncthreads();
    uint32_t *out = a.parts + (uint64_t)blockIdx.x * (2 * a.experts + 2);
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBThreads) {
        float s = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < kBWaves; ++w) s += sums[w][e];
        out[e] = __float_as_uint(s);
        out[a.experts + e] = bins[e];
    }
    if (threadIdx.x == 0) {
        float s = 0.0f;
        uint32_t m = 0;
#pragma unroll
        for (uint32_t w = 0; w < kBWaves; ++w) {
            s += zs[w];
            m += ns[w];
        }
        out[2 * a.experts] = __float_as_uint(s);
        out[2 * a.experts + 1] = m;
    }
}

// 64 experts of one sequence a block: its tiles' sums in order, in 16 runs of tiles side by side.  The last of a
// sequence's blocks to come to an end adds their shares of the loss, in the order of the experts: words that other blocks
// wrote go past the caches of the XCDs, and a count taken after them says that they are there.  (One block a
// sequence, 256 experts, 257 tiles: 8.9 us.)
constexpr uint32_t kJRuns = 16;
constexpr uint32_t kJThreads = kJRuns * kLanes;
__global__ __launch_bounds__(kJThreads) void balance_join_kernel(BalanceArgs a) {
    __shared__ float sums[kJRuns][kLanes];
    __shared__ uint32_t hits[kJRuns][kLanes];
    __shared__ float all_z;
    __shared__ uint32_t all_n;
    const uint32_t lane = lane_id(), run = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t s = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
    // the sequence's tiles
    uint32_t first = 0, tiles = 0;
    if (!a.offsets) {
        tiles = (a.tokens + a.tile_rows - 1) / a.tile_rows;
    } else {
        uint32_t high = 0;
        for (uint32_t g0 = 0; g0 <= s; g0 += kLanes) {
            const Groups r = load_groups(a.offsets, a.sequences, a.tokens, a.tile_rows, g0, high);
            if (s < g0 + kLanes) {
                const int l = (int)(s - g0);
                tiles = (uint32_t)__builtin_amdgcn_readlane((int)r.tiles, l);
                first += (uint32_t)__builtin_amdgcn_readlane((int)(r.tile_sum - r.tiles), l);
            } else {
                first += last_lane(r.tile_sum);
            }
            high = last_lane(r.end);
        }
    }
    const uint32_t e = slice * kLanes + lane, words = 2 * a.experts + 2;
    float p = 0.0f;
    uint32_t c = 0;
    if (e < a.experts) {
        const uint32_t i0 = (uint32_t)((uint64_t)tiles * run / kJRuns), i1 = (uint32_t)((uint64_t)tiles * (run + 1) / kJRuns);
        const uint32_t *src = a.parts + (uint64_t)(first + i0) * words + e;
#pragma unroll 8
        for (uint32_t i = i0; i < i1; ++i, src += words) {
            p += __uint_as_float(src[0]);
            c += src[a.experts];
        }
    }
    sums[run][lane] = p;
    hits[run][lane] = c;
    __syncthreads();
    if (run == 1 && slice == 0) {  // a lane's tiles, then the lanes
        float z = 0.0f;
        uint32_t n = 0;
        for (uint32_t i = lane; i < tiles; i += kLanes) {
            const uint32_t *src = a.parts + (uint64_t)(first + i) * words + 2 * a.experts;
            z += __uint_as_float(src[0]);
            n += src[1];
        }
        z = wave_sum_f(z);
        n = last_lane(scan_sum(n));
        if (lane == 0) {
            all_z = z;
            all_n = n;
        }
    }
    float mine = 0.0f;
    if (run == 0) {
#pragma unroll
        for (uint32_t r = 1; r < kJRuns; ++r) {
            p += sums[r][lane];
            c += hits[r][lane];
        }
        if (e < a.experts) a.counts[(uint64_t)s * a.experts + e] = (int32_t)c;
        mine = wave_sum_f((float)c * p);
    }
    __syncthreads();
    if (threadIdx.x) return;
    // one thread writes what the last block reads, and counts its block after that
    uint32_t *join = a.joins + s * kJoinWords;
    const auto leave = [&](uint32_t i, uint32_t v) { __hip_atomic_store(&join[i], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    leave(slice, __float_as_uint(mine));
    if (slice == 0) {
        leave(kJoinZ, __float_as_uint(all_z));
        leave(kJoinUsed, all_n);
    }
    const uint32_t before = __hip_atomic_fetch_add(&join[kJoinDone], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (before + 1 != slices) return;
    const auto word = [&](uint32_t i) { return __hip_atomic_load(&join[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    float share = 0.0f;
    for (uint32_t i = 0; i < slices; ++i) share += __uint_as_float(word(i));
    const float z = __uint_as_float(word(kJoinZ));
    const uint32_t n = word(kJoinUsed);
    a.used[s] = (int32_t)n;
    // (quotients in 64 bits: the sums' own error is all that they have)
    const double each = n ? 1.0 / (double)n : 0.0;
    if (a.loss) a.loss[s] = n ? (float)((double)share * each * each * a.experts_each) : 0.0f;
    if (a.zloss) a.zloss[s] = n ? (float)((double)z * each) : 0.0f;
}
// Without tokens there are no tiles.
__global__ __launch_bounds__(256) void balance_zero_kernel(BalanceArgs a) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < a.sequences * a.experts) a.counts[i] = 0;
    if (i >= a.sequences) return;
    a.used[i] = 0;
    if (a.loss) a.loss[i] = 0.0f;
    if (a.zloss) a.zloss[i] = 0.0f;
}

// A wave takes `run` consecutive tokens.  The sequence of token t ends at the first
// offset above t, whatever the offsets before it are; an index of 0, or none,
// means that no sequence holds it.  8192 tokens of 256 experts 9.0 us (17 MB), 65536 of 160 in 37 sequences 26 us
// (84 MB, 3.2 TB/s): bound by the exponentials, one a value, and the sums over the lanes beside the memory.
template <bool BF16, bool SIGMOID, uint32_t V>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceArgs a) {
    const uint32_t lane = lane_id();
    const uint64_t wave = (uint64_t)blockIdx.x * 4 + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint64_t first = wave * a.run;
    if (first >= a.tokens) return;
    const uint32_t t1 = (uint32_t)min((uint64_t)a.tokens, first + a.run);
    float f[V], slope = 0.0f, zslope = 0.0f;
    bool live = false;
    uint32_t until = 0;
    for (uint32_t t = (uint32_t)first; t < t1; ++t) {
        if (t >= until) {
            uint32_t at = a.sequences + 1;
            until = ~0u;
            if (!a.offsets) {
                at = 1;
            } else {
                for (uint32_t j0 = 0; j0 <= a.sequences; j0 += kLanes) {
                    const uint32_t j = j0 + lane;
                    const uint32_t o = j <= a.sequences ? clamp_row(a.offsets[j], a.tokens) : 0u;
                    const uint64_t above = __ballot(o > t);
                    if (above) {
                        const int l = __builtin_ctzll(above);
                        at = j0 + (uint32_t)l;
                        until = (uint32_t)__builtin_amdgcn_readlane((int)o, l);
                        break;
                    }
                }
            }
            live = at >= 1 && at <= a.sequences;
            if (live) {
                const uint32_t s = at - 1;
                const int32_t n = a.used[s];
                live = n > 0;
                const float each = live ? 1.0f / (float)n : 0.0f;
                slope = a.dloss ? a.dloss[s] * each : 0.0f;
                zslope = a.dzloss ? 2.0f * a.dzloss[s] * each : 0.0f;
                const float unit = each * ((float)a.experts / (float)a.top_k);
#pragma unroll
                for (uint32_t i = 0; i < V; ++i) {
                    const uint32_t e = lane + kLanes * i;
                    f[i] = e < a.experts ? (float)a.counts[(uint64_t)s * a.experts + e] * unit : 0.0f;
                }
            }
        }
        float d[V];
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) d[i] = 0.0f;
        if (live && (!a.mask || a.mask[t])) {
            float l[V], p[V], rest[V];
            load_token<BF16, kLanes, V>(a, t, l);
            if (!SIGMOID || a.dzloss) {
                const float lse = softmax<kLanes, V>(l, p);
#pragma unroll
                for (uint32_t i = 0; i < V; ++i) d[i] = p[i] * (lse * zslope);
            }
            if (a.dloss) {
                if (SIGMOID) sigmoids<kLanes, V>(l, p, rest);
                float fp = 0.0f;
#pragma unroll
                for (uint32_t i = 0; i < V; ++i) fp = fmaf(f[i], p[i], fp);
                fp = wave_sum_f(fp);
#pragma unroll
                for (uint32_t i = 0; i < V; ++i) {
                    const float g = p[i] * (f[i] - fp) * slope;
                    d[i] += SIGMOID ? g * rest[i] : g;
                }
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) {
            const uint32_t e = lane + kLanes * i;
            if (e >= a.experts) continue;
            if (a.add) d[i] += value_at<BF16>(a.add, t * a.add_stride + e);
            if (BF16)
                static_cast<uint16_t *>(a.dlogits)[t * a.out_stride + e] = bf_round(d[i]);
            else
                static_cast<float *>(a.dlogits)[t * a.out_stride + e] = d[i];
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// A tile's tokens: about 256 tiles, whose sums one block a sequence then joins.
static uint32_t tile_rows_of(uint64_t tokens) {
    const uint64_t rows = ceil_div(ceil_div(tokens, 256), 32) * 32;  // 32: eight waves of four tokens
    return (uint32_t)(rows ? rows : 32);
}
static uint64_t tiles_of(uint64_t tokens, uint64_t sequences) {
    return tokens / tile_rows_of(tokens) + (tokens < sequences ? tokens : sequences);
}

// Bytes of the tiles' sums, behind which the joins lie.
static uint64_t join_at(uint64_t tokens, uint64_t experts, uint64_t sequences) {
    return ceil_div(tiles_of(tokens, sequences) * (2 * experts + 2) * 4, 256) * 256;
}

template <uint32_t N>
using Width = std::integral_constant<uint32_t, N>;

static void launch_tiles(const BalanceArgs &a, bool bf16, bool sigmoid, dim3 grid, Launches &on) {
    const auto go = [&](auto lanes, auto width) {
        constexpr uint32_t L = decltype(lanes)::value, V = decltype(width)::value;
        on.launch(bf16 ? (sigmoid ? balance_tile_kernel<true, true, L, V> : balance_tile_kernel<true, false, L, V>)
                       : (sigmoid ? balance_tile_kernel<false, true, L, V> : balance_tile_kernel<false, false, L, V>),
                  grid, dim3(kBThreads), a);
    };
    // (past 256 experts 16 lanes would hold more than 16 each)
    const uint32_t v = (a.experts + 15) / 16;
    if (v <= 1) return go(Width<16>{}, Width<1>{});
    if (v <= 2) return go(Width<16>{}, Width<2>{});
    if (v <= 4) return go(Width<16>{}, Width<4>{});
    if (v <= 8) return go(Width<16>{}, Width<8>{});
    if (v <= 12) return go(Width<16>{}, Width<12>{});
    if (v <= 16) return go(Width<16>{}, Width<16>{});
    if (v <= 32) return go(Width<64>{}, Width<8>{});
    go(Width<64>{}, Width<16>{});
}
static void launch_backward(const BalanceArgs &a, bool bf16, bool sigmoid, dim3 grid, Launches &on) {
    const auto go = [&](auto width) {
        constexpr uint32_t V = decltype(width)::value;
        on.launch(bf16 ? (sigmoid ? balance_backward_kernel<true, true, V> : balance_backward_kernel<true, false, V>)
                       : (sigmoid ? balance_backward_kernel<false, true, V> : balance_backward_kernel<false, false, V>),
                  grid, dim3(256), a);
    };
    const uint32_t v = (a.experts + kLanes - 1) / kLanes;
    if (v <= 1) return go(Width<1>{});
    if (v <= 2) return go(Width<2>{});
    if (v <= 3) return go(Width<3>{});
    if (v <= 4) return go(Width<4>{});
    if (v <= 8) return go(Width<8>{});
    go(Width<16>{});
}

static bool balance_ok(const zc_route_config *cfg, uint32_t logits_type, uint64_t tokens, uint32_t sequences,
                       const int32_t *d_offsets) {
    return cfg && cfg->experts >= 1 && cfg->experts <= ZC_MAX_EXPERTS && cfg->top_k >= 1 &&
           cfg->top_k <= ZC_MAX_TOP_K && cfg->score <= ZC_SCORE_SIGMOID && logits_type <= ZC_BF16 &&
           tokens <= kMaxRows / cfg->top_k && sequences >= 1 && sequences <= ZC_MAX_SEQUENCES &&
           (d_offsets || sequences == 1);
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_balance_workspace_bytes(uint64_t tokens, uint32_t experts, uint32_t sequences) {
    if (tokens > kMaxRows || experts < 1 || experts > ZC_MAX_EXPERTS || sequences < 1 || sequences > ZC_MAX_SEQUENCES)
        return 0;
    return ceil_div(join_at(tokens, experts, sequences) + sequences * kJoinWords * 4, 256) * 256;
}

extern "C" zc_status zc_balance(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                                const zc_route_config *cfg, const int32_t *d_ids, const uint8_t *d_mask,
                                uint32_t sequences, const int32_t *d_offsets, void *d_workspace,
                                uint64_t workspace_bytes, int32_t *d_counts, int32_t *d_used, float *d_loss,
                                float *d_zloss, void *stream) {
    if (!balance_ok(cfg, logits_type, tokens, sequences, d_offsets) || !d_counts || !d_used) return ZC_ERR_INVALID_ARG;
    const bool losses = d_loss || d_zloss;
    if (losses && (logits_stride < cfg->experts || logits_stride > kMaxStride)) return ZC_ERR_INVALID_ARG;
    if (tokens && ((losses && !d_logits) || !d_ids || !d_workspace)) return ZC_ERR_INVALID_ARG;
    if ((losses && !aligned(d_logits, logits_type == ZC_F32 ? 4 : 2)) || !aligned(d_ids, 4) || !aligned(d_offsets, 4) ||
        !aligned(d_workspace, 16) || !aligned(d_counts, 4) || !aligned(d_used, 4) || !aligned(d_loss, 4) ||
        !aligned(d_zloss, 4))
        return ZC_ERR_MISALIGNED;
    if (tokens && workspace_bytes < zc_balance_workspace_bytes(tokens, cfg->experts, sequences)) return ZC_ERR_CAPACITY;
    BalanceArgs a = {};
    a.logits = d_logits;
    a.ids = d_ids;
    a.mask = d_mask;
    a.offsets = d_offsets;
    a.parts = static_cast<uint32_t *>(d_workspace);
    a.counts = d_counts;
    a.used = d_used;
    a.loss = d_loss;
    a.zloss = d_zloss;
    a.stride = logits_stride;
    a.tokens = (uint32_t)tokens;
    a.experts = cfg->experts;
    a.top_k = cfg->top_k;
    a.sequences = sequences;
    a.tile_rows = tile_rows_of(tokens);
    a.experts_each = (double)a.experts / (double)a.top_k;
    Launches on(stream);
    if (!tokens) {
        on.launch(balance_zero_kernel, dim3((uint32_t)ceil_div((uint64_t)sequences * a.experts, 256)), dim3(256), a);
        return on.status();
    }
    a.joins = a.parts + join_at(tokens, a.experts, sequences) / 4;
    const uint64_t tiles = d_offsets ? tiles_of(tokens, sequences) : ceil_div(tokens, a.tile_rows);
    launch_tiles(a, logits_type == ZC_BF16, cfg->score == ZC_SCORE_SIGMOID, dim3((uint32_t)tiles), on);
    on.launch(balance_join_kernel, dim3(sequences, (a.experts + kLanes - 1) / kLanes), dim3(kJThreads), a);
    return on.status();
}

extern "C" zc_status zc_balance_backward(const void *d_logits, uint32_t logits_type, uint64_t tokens,
                                         uint64_t logits_stride, const zc_route_config *cfg, const uint8_t *d_mask,
                                         uint32_t sequences, const int32_t *d_offsets, const int32_t *d_counts,
                                         const int32_t *d_used, const float *d_dloss, const float *d_dzloss,
                                         const void *d_add, uint64_t add_stride, void *d_dlogits,
                                         uint64_t dlogits_stride, void *stream) {
    if (!balance_ok(cfg, logits_type, tokens, sequences, d_offsets) || logits_stride < cfg->experts ||
        logits_stride > kMaxStride || dlogits_stride < cfg->experts || dlogits_stride > kMaxStride ||
        (d_add && (add_stride < cfg->experts || add_stride > kMaxStride)))
        return ZC_ERR_INVALID_ARG;
    if (!tokens) return ZC_OK;
    if (!d_logits || !d_counts || !d_used || !d_dlogits) return ZC_ERR_INVALID_ARG;
    const uint32_t size = logits_type == ZC_F32 ? 4 : 2;
    if (!aligned(d_logits, size) || !aligned(d_offsets, 4) || !aligned(d_counts, 4) || !aligned(d_used, 4) ||
        !aligned(d_dloss, 4) || !aligned(d_dzloss, 4) || !aligned(d_add, size) || !aligned(d_dlogits, size))
        return ZC_ERR_MISALIGNED;
    BalanceArgs a = {};
    a.logits = d_logits;
    a.mask = d_mask;
    a.offsets = d_offsets;
    a.counts = const_cast<int32_t *>(d_counts);
    a.used = const_cast<int32_t *>(d_used);
    a.dloss = d_dloss;
    a.dzloss = d_dzloss;
    a.add = d_add;
    a.dlogits = d_dlogits;
    a.stride = logits_stride;
    a.add_stride = add_stride;
    a.out_stride = dlogits_stride;
    a.tokens = (uint32_t)tokens;
    a.experts = cfg->experts;
    a.top_k = cfg->top_k;
    a.sequences = sequences;
    a.run = (uint32_t)ceil_div(tokens, 8192);
    const uint64_t blocks = ceil_div(ceil_div(tokens, a.run), 4);
    Launches on(stream);
    launch_backward(a, logits_type == ZC_BF16, cfg->score == ZC_SCORE_SIGMOID, dim3((uint32_t)blocks), on);
    return on.status();
}
