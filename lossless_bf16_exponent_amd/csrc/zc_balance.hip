// Balance of the experts, MI355X / gfx950: copies of every expert, balance loss and
// z loss of every sequence, and the logits' gradient:
//   loss = experts / (top_k n^2) sum_e c[e] sum_t p[t, e],  z = 1 / n sum_t lse(t)^2
//   d loss / d logit = experts / (top_k n^2) p_e (c_e - sum_j c_j p_j) [(1 - sigmoid_e) for sigmoid scores]
//   d z / d logit = 2 / n lse softmax_e
// Bound by reading the logits, and at a few thousand tokens by the latency of a
// token's steps: a wave holds a token, lane l the experts l, l + 64, ...
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
    int32_t *counts, *used;
    float *loss, *zloss;
    const float *dloss, *dzloss;
    uint64_t stride, add_stride, out_stride;
    uint32_t tokens, experts, top_k, sequences, tile_rows, run;
};

// Largest of the wave; a lane without a source keeps its own.
__device__ __forceinline__ float wave_max_f(float v) {
#define ZC_MOE_LARGER(ctrl, rows)                                                                       \
    v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(                                 \
                     (int)__float_as_uint(v), (int)__float_as_uint(v), ctrl, rows, 0xF, false)))
    ZC_MOE_LARGER(0x111, 0xF);
    ZC_MOE_LARGER(0x112, 0xF);
    ZC_MOE_LARGER(0x114, 0xF);
    ZC_MOE_LARGER(0x118, 0xF);
    ZC_MOE_LARGER(0x142, 0xA);
    ZC_MOE_LARGER(0x143, 0xC);
#undef ZC_MOE_LARGER
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

template <bool BF16>
__device__ __forceinline__ float value_at(const void *p, uint64_t i) {
    return BF16 ? bf_one(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
// A token's logits; -inf past the last expert.
template <bool BF16, uint32_t V>
__device__ __forceinline__ void load_token(const BalanceArgs &a, uint64_t t, float (&l)[V]) {
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        const uint32_t e = lane_id() + kLanes * i;
        l[i] = e < a.experts ? value_at<BF16>(a.logits, t * a.stride + e) : -__builtin_inff();
    }
}

// Softmax of the wave's logits, and the logarithm of its sum of exponentials: 0 and
// 0 where all are -inf.  NaN and +inf make all of it NaN.
template <uint32_t V>
__device__ __forceinline__ float softmax(const float (&l)[V], float (&p)[V]) {
    float top = l[0];
#pragma unroll
    for (uint32_t i = 1; i < V; ++i) top = fmaxf(top, l[i]);
    top = wave_max_f(top);
    if (top == -__builtin_inff()) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        p[i] = expf(l[i] - top);
        sum += p[i];
    }
    sum = wave_sum_f(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) p[i] *= inv;
    return sum == 0.0f ? 0.0f : top + logf(sum);
}
// Sigmoids over their sum; rest: 1 - sigmoid.
template <uint32_t V>
__device__ __forceinline__ void sigmoids(const float (&l)[V], float (&p)[V], float (&rest)[V]) {
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) {
        const float t = expf(-fabsf(l[i])), r = 1.0f / (1.0f + t), tr = t * r;
        p[i] = l[i] >= 0.0f ? r : tr;
        rest[i] = l[i] >= 0.0f ? tr : r;
        sum += p[i];
    }
    const float inv = 1.0f / (wave_sum_f(sum) + 1e-20f);
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) p[i] *= inv;
}

// The sums of one tile of a sequence's tokens.
template <bool BF16, bool SIGMOID, uint32_t V>
__global__ __launch_bounds__(kBThreads) void balance_tile_kernel(BalanceArgs a) {
    __shared__ float sums[kBWaves][kLanes * V];
    __shared__ uint32_t bins[kLanes * V];
    __shared__ float zs[kBWaves];
    __shared__ uint32_t ns[kBWaves];
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const Span sp = find_tile(a.offsets, a.sequences, a.tokens, a.tile_rows, [&](uint32_t) { return blockIdx.x; });
    if (!sp.found) return;
    const uint32_t t0 = sp.begin + sp.tile * a.tile_rows, t1 = min(t0 + a.tile_rows, sp.end);
    for (uint32_t e = threadIdx.x; e < kLanes * V; e += kBThreads) bins[e] = 0;
    __syncthreads();
    const uint64_t i1 = (uint64_t)t1 * a.top_k;
    for (uint64_t i = (uint64_t)t0 * a.top_k + threadIdx.x; i < i1; i += kBThreads) {
        const int32_t id = a.ids[i];
        if (id >= 0 && (uint32_t)id < a.experts && (!a.mask || a.mask[i / a.top_k])) atomicAdd(&bins[id], 1u);
    }
    float acc[V], z = 0.0f;
    uint32_t n = 0;
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) acc[i] = 0.0f;
    for (uint32_t t = t0 + wave; t < t1; t += kBWaves) {
        if (a.mask && !a.mask[t]) continue;
        ++n;
        if (!a.loss && !a.zloss) continue;
        float l[V], p[V];
        load_token<BF16, V>(a, t, l);
        if (!SIGMOID || a.zloss) {
            const float lse = softmax<V>(l, p);
            z = fmaf(lse, lse, z);
        }
        if (SIGMOID) {
            float rest[V];
            sigmoids<V>(l, p, rest);
        }
#pragma unroll
        for (uint32_t i = 0; i < V; ++i) acc[i] += p[i];
    }
#pragma unroll
    for (uint32_t i = 0; i < V; ++i) sums[wave][lane + kLanes * i] = acc[i];
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

// One sequence a block: its tiles' sums in order, in runs of tiles side by side.
constexpr uint32_t kJThreads = 1024;
__global__ __launch_bounds__(kJThreads) void balance_join_kernel(BalanceArgs a) {
    __shared__ float sums[kJThreads];
    __shared__ uint32_t hits[kJThreads];
    __shared__ float waves[kJThreads / kLanes];
    __shared__ float zs[kLanes];
    __shared__ uint32_t ns[kLanes];
    const uint32_t tid = threadIdx.x, lane = lane_id(), wave = tid / kLanes, s = blockIdx.x;
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
    const uint32_t width = (a.experts + kLanes - 1) / kLanes * kLanes, runs = kJThreads / width;
    const uint32_t run = tid / width, e = tid % width, words = 2 * a.experts + 2;
    float p = 0.0f;
    uint32_t c = 0;
    if (run < runs && e < a.experts) {
        const uint32_t i0 = (uint32_t)((uint64_t)tiles * run / runs), i1 = (uint32_t)((uint64_t)tiles * (run + 1) / runs);
        const uint32_t *src = a.parts + (uint64_t)(first + i0) * words + e;
#pragma unroll 4
        for (uint32_t i = i0; i < i1; ++i, src += words) {
            p += __uint_as_float(src[0]);
            c += src[a.experts];
        }
    }
    sums[tid] = p;
    hits[tid] = c;
    if (wave == 0) {  // a lane's tiles, then the lanes in order
        float z = 0.0f;
        uint32_t n = 0;
        for (uint32_t i = lane; i < tiles; i += kLanes) {
            const uint32_t *src = a.parts + (uint64_t)(first + i) * words + 2 * a.experts;
            z += __uint_as_float(src[0]);
            n += src[1];
        }
        zs[lane] = z;
        ns[lane] = n;
    }
    __syncthreads();
    float share = 0.0f;
    if (tid < a.experts) {
        for (uint32_t r = 1; r < runs; ++r) {
            p += sums[r * width + tid];
            c += hits[r * width + tid];
        }
        a.counts[(uint64_t)s * a.experts + tid] = (int32_t)c;
        share = (float)c * p;
    }
    share = wave_sum_f(share);
    if (lane == 0) waves[wave] = share;
    __syncthreads();
    if (tid) return;
    float z = 0.0f;
    uint32_t n = 0;
    for (uint32_t i = 0; i < kLanes; ++i) {
        z += zs[i];
        n += ns[i];
    }
    for (uint32_t w = 1; w < kJThreads / kLanes; ++w) share += waves[w];
    a.used[s] = (int32_t)n;
    const float each = n ? 1.0f / (float)n : 0.0f;
    if (a.loss) a.loss[s] = n ? share * each * each * ((float)a.experts / (float)a.top_k) : 0.0f;
    if (a.zloss) a.zloss[s] = n ? z * each : 0.0f;
}

// A wave takes `run` consecutive tokens.  The sequence of token t ends at the first
// offset above t, whatever the offsets before it are; an index of 0, or none,
// means that no sequence holds it.
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
            load_token<BF16, V>(a, t, l);
            if (!SIGMOID || a.dzloss) {
                const float lse = softmax<V>(l, p);
#pragma unroll
                for (uint32_t i = 0; i < V; ++i) d[i] = p[i] * (lse * zslope);
            }
            if (a.dloss) {
                if (SIGMOID) sigmoids<V>(l, p, rest);
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
    const uint64_t rows = ceil_div(ceil_div(tokens, 256), kBWaves) * kBWaves;
    return (uint32_t)(rows < 16 ? 16 : rows);
}
static uint64_t tiles_of(uint64_t tokens, uint64_t sequences) {
    return tokens / tile_rows_of(tokens) + (tokens < sequences ? tokens : sequences);
}

template <template <bool, bool, uint32_t> class Pick>
static void launch_width(const BalanceArgs &a, bool bf16, bool sigmoid, dim3 grid, dim3 block, Launches &on) {
    const auto go = [&](auto width) {
        constexpr uint32_t V = decltype(width)::value;
        on.launch(bf16 ? (sigmoid ? Pick<true, true, V>::kernel() : Pick<true, false, V>::kernel())
                       : (sigmoid ? Pick<false, true, V>::kernel() : Pick<false, false, V>::kernel()),
                  grid, block, a);
    };
    const uint32_t v = (a.experts + kLanes - 1) / kLanes;
    if (v <= 1)
        go(std::integral_constant<uint32_t, 1>{});
    else if (v <= 2)
        go(std::integral_constant<uint32_t, 2>{});
    else if (v <= 4)
        go(std::integral_constant<uint32_t, 4>{});
    else if (v <= 8)
        go(std::integral_constant<uint32_t, 8>{});
    else
        go(std::integral_constant<uint32_t, 16>{});
}
template <bool BF16, bool SIGMOID, uint32_t V>
struct Tile {
    static auto kernel() { return &balance_tile_kernel<BF16, SIGMOID, V>; }
};
template <bool BF16, bool SIGMOID, uint32_t V>
struct BalanceBackward {
    static auto kernel() { return &balance_backward_kernel<BF16, SIGMOID, V>; }
};

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
    return ceil_div((tiles_of(tokens, sequences) + 1) * (2 * (uint64_t)experts + 2) * 4, 256) * 256;
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
    Launches on(stream);
    const uint64_t tiles = d_offsets ? tiles_of(tokens, sequences) : ceil_div(tokens, a.tile_rows);
    if (tokens)
        launch_width<Tile>(a, logits_type == ZC_BF16, cfg->score == ZC_SCORE_SIGMOID, dim3((uint32_t)tiles),
                           dim3(kBThreads), on);
    on.launch(balance_join_kernel, dim3(sequences), dim3(kJThreads), a);
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
    launch_width<BalanceBackward>(a, logits_type == ZC_BF16, cfg->score == ZC_SCORE_SIGMOID, dim3((uint32_t)blocks),
                                  dim3(256), on);
    return on.status();
}
