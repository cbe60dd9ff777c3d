// What the norms' kernels share (gfx950): a row in a team's registers, its
// statistics, parameters, and the host's checks and shapes.
#pragma once

#include <type_traits>

#include "zc_moe_device.h"

namespace zc {
namespace moe {

struct Param {
    const void *p;
    uint32_t f32;
};
struct NormSide {
    Param w, b;
    uint32_t kind;
    float eps;
};
struct NormArgs {
    const void *x, *dr;  // stream_type; backward: x is the stored sum
    const uint16_t *z, *dy;
    void *r;             // stream_type: the sum, or the gradient of x
    uint16_t *y, *dz;
    uint8_t *yq, *ys;
    NormSide after, before;
    Param gate;
    const float *row_gate;
    float *drow_gate;
    float *parts;        // [kSums][parts rows][cols]
    uint64_t x_stride, z_stride, r_stride, y_stride, dr_stride, dy_stride, dz_stride, q_stride, qs_stride;
    uint64_t part_stride;  // floats of one sum's parts
    uint32_t rows, cols, sums;  // sums: which are asked for, a bit each
    uint32_t wide;  // any rows: the results' start on 16 bytes
    float scale, inv_cols;
};

enum Sum { kDW1, kDB1, kDGate, kDW2, kDB2, kSums };

// ---------------------------------------------------------------------------
// results and parameters
// ---------------------------------------------------------------------------

// wide: rows start on 16 bytes, so that a line is written by one instruction and
// need not stay in the L2 for the next.
__device__ __forceinline__ void store_bf(uint16_t *p, const u32v4 &w, uint32_t n, uint32_t wide) {
    if (wide)
        store_values<true>(p, w, n);
    else
        store_values<false>(p, w, n);
}
template <bool F32S>
__device__ __forceinline__ void store_stream(void *base, uint64_t at, uint32_t n, const float (&v)[8], uint32_t wide) {
    if (F32S)
        store_floats(static_cast<float *>(base) + at, n, v);
    else
        store_bf(static_cast<uint16_t *>(base) + at, pack8(v), n, wide);
}
// Parameters of columns c .. c + n - 1; `otherwise` where there are none.
__device__ __forceinline__ void load_param(const Param &q, uint32_t c, uint32_t n, float otherwise, float (&v)[8]) {
    if (!q.p) {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = otherwise;
    } else if (q.f32) {
        Eight<true> e;
        e.load(q.p, c, n, false);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = e[i];
    } else {
        Eight<false> e;
        e.load(q.p, c, n, false);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = e[i];
    }
}

// ---------------------------------------------------------------------------
// sums over a row
// ---------------------------------------------------------------------------

constexpr uint32_t kMaxWaves = 16;
constexpr float kMost = 3.40282347e38f;  // the largest float

// A team of TEAM lanes holds a row.  Sums of K values over it: over each wave,
// then over the waves in order.  Two places in turn, so that one barrier a sum is
// enough: a place is written again only after the barrier of the sum between.
template <uint32_t TEAM>
struct Team {
    float (*parts)[kMaxWaves][4];
    uint32_t turn;
    template <uint32_t K>
    __device__ __forceinline__ void sum(float (&v)[K]) {
        static_assert(K <= 4, "four a turn");
#pragma unroll
        for (uint32_t k = 0; k < K; ++k) v[k] = wave_sum_f(v[k]);
        if (TEAM == kLanes) return;
        const uint32_t wave = threadIdx.x / kLanes;
        if (lane_id() == 0)
#pragma unroll
            for (uint32_t k = 0; k < K; ++k) parts[turn][wave][k] = v[k];
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < K; ++k) v[k] = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < TEAM / kLanes; ++w)
#pragma unroll
            for (uint32_t k = 0; k < K; ++k) v[k] += parts[turn][w][k];
        turn ^= 1;
    }
};

// The normed value of v is (v / 2 - mean / 2) * k - off, in halves so that no difference leaves the range of a float: slope is
// 1 / deviation, k twice that, and off what rounding the mean left, which counts where the deviation is small beside the
// mean.  A constant row, whose normed values are 0, has a k of 0: lanes past its end hold zeros, which could leave the
// range.
struct Stat {
    float middle, off, k, slope;
};
constexpr Stat kNoNorm = {0.0f, 0.0f, 2.0f, 1.0f};
// A row's mean, rounded: without the pragma the product would go unrounded into one difference and rounded into another,
// and what the sums of the differences say of it would be of another mean.
__device__ __forceinline__ float mean_of(float sum, float inv_cols) {
#pragma clang fp contract(off)
    return sum * inv_cols;
}
// MEAN: there may be a mean.
template <bool MEAN = true>
__device__ __forceinline__ float normed(float v, const Stat &s) {
    return MEAN ? fmaf(fmaf(v, 0.5f, -s.middle), s.k, -s.off) : v * s.slope;
}
// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}
// What the mean's rounding left of a row's deviations, and the sum of their squares without it and with it.
struct Deviations {
    float rest, var, spread;
};
__device__ __forceinline__ Deviations beside_rest(float squares, float sum, float inv_cols) {
    // (where the difference is lost in rounding: not below 0, and NaN stays)
    const float rest = sum * inv_cols, left = fmaf(-rest, sum, squares);
    return {rest, left < 0.0f ? 0.0f : left, squares};
}
// Next to nothing is left beside the mean's rounding.
__device__ __forceinline__ bool lost(const Deviations &s) { return s.var < s.spread * 0x1p-16f; }
// Whether a row has to be measured again: where that is so, or squares leave the range of a float (above 2^120 in sum, infinities and
// NaN among them, or below 2^-80 with an eps that does not cover them).  Measured 2^-80 or 2^80 times as large it keeps all
// digits that matter.  (The same in all of a team's lanes, and rarely.)
__device__ __forceinline__ bool out_of_range(const Deviations &s, float eps) {
    const bool out = !(s.var <= 0x1p120f) || (s.var < 0x1p-80f && eps < 0x1p-58f) || lost(s);
    return __builtin_expect(__builtin_amdgcn_readfirstlane(out) != 0, 0);
}

// Keeps packed values packed: the compiler would unpack what does not change once for all rows.
template <bool F32>
__device__ __forceinline__ void stay_packed(Eight<F32> &v) {
    if (!F32) asm volatile("" : "+v"(v.w[0]));
}
template <bool F32, uint32_t CHUNKS>
__device__ __forceinline__ void apart(Eight<F32> (&v)[CHUNKS]) {
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) stay_packed(v[i]);
}
template <uint32_t CHUNKS>
__device__ __forceinline__ void apart(float (&)[CHUNKS][8]) {}

// A row's values in a team's lanes, with what it takes to measure them.
template <uint32_t TEAM, uint32_t CHUNKS, typename V>
struct Measured {
    V &v;
    const uint32_t (&n)[CHUNKS];
    Team<TEAM> &team;
    uint32_t kind;
    float eps, inv_cols, tail;
    bool in_tail;

    __device__ __forceinline__ float average(float unit) const {
        float t[1] = {tail * unit};
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) t[0] = fmaf(v[i][j], unit, t[0]);
        team.sum(t);
        return mean_of(t[0], inv_cols);
    }
    // Deviations `less` * `more` times as large: values and mean are made `less` times as large before the difference.
    __device__ __forceinline__ Deviations deviations(float mean, float less, float more) const {
        if (kind == ZC_NORM_LAYER) {
            const float middle = mean * less;
            const float last = in_tail ? fmaf(tail, less, -middle) * more : 0.0f;
            float u[2] = {last * last, last};
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float d = j < n[i] ? fmaf(v[i][j], less, -middle) * more : 0.0f;
                    u[0] = fmaf(d, d, u[0]);
                    u[1] += d;
                }
            team.sum(u);
            return beside_rest(u[0], u[1], inv_cols);
        }
        const float unit = less * more;
        float t[1] = {tail * unit * (tail * unit)};
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const float d = v[i][j] * unit;
                t[0] = fmaf(d, d, t[0]);
            }
        team.sum(t);
        return {0.0f, t[0], 0.0f};
    }
    // The statistics from a mean and the deviations from it, measured again where they have to be.
    __device__ __forceinline__ Stat settle(float mean, Deviations s) const {
        float unit = 1.0f;
        if (out_of_range(s, eps)) {
            apart(v);
            if (!(s.var <= 0x1p120f)) unit = 0x1p-80f;
            if (kind == ZC_NORM_LAYER && unit < 1.0f) {
                // (the values' sum may have left the range too, which their mean does not)
                const float small = average(unit);
                mean = fabsf(small) < 0x1p50f ? fminf(fmaxf(small / unit, -kMost), kMost) : small;
                s = deviations(mean, unit, 1.0f);
                apart(v);
            }
            // The mean takes what its rounding left: a constant row then has no deviation at all.  What still deviates does so by a
            // step of the mean at least, whose square is in range where the mean is not tiny itself.
            const bool centre = lost(s);
            if (centre) mean += s.rest / unit;
            if (s.var < 0x1p-80f && eps < 0x1p-58f && unit == 1.0f && !(centre && fabsf(mean) > 0x1p-20f)) unit = 0x1p80f;
            s = deviations(mean, fminf(unit, 1.0f), fmaxf(unit, 1.0f));
            if (s.var == 0.0f) unit = 1.0f, s.rest = 0.0f;  // no deviation: what is left is eps, as it is
        }
        // eps in the row's unit (for large rows it is nothing beside their squares)
        const float rs = __builtin_amdgcn_rsqf(fmaf(s.var, inv_cols, eps * unit * unit));
        // (one step of the mean as the only deviation makes a product of 2^33 at most)
        const float slope = rs * unit;
        return {uniform(0.5f * mean), s.rest * rs, fabsf(mean) * slope < 0x1p100f ? 2.0f * slope : 0.0f, uniform(slope)};
    }
};

template <uint32_t TEAM, uint32_t CHUNKS, typename V>
__device__ __forceinline__ Stat row_stat(V &v, const uint32_t (&n)[CHUNKS], uint32_t kind, float eps, float inv_cols,
                                         Team<TEAM> &team, float tail = 0.0f, bool in_tail = false) {
    const Measured<TEAM, CHUNKS, V> m = {v, n, team, kind, eps, inv_cols, tail, in_tail};
    const float mean = kind == ZC_NORM_LAYER ? m.average(1.0f) : 0.0f;
    return m.settle(mean, m.deviations(mean, 1.0f, 1.0f));
}

// ---------------------------------------------------------------------------
// rows through descriptors
// ---------------------------------------------------------------------------

// A row is reached through a descriptor of its own (buffer accesses take any value as their
// start): what lies past its end reads as 0 and is not written, without a branch, so that a load
// on its way is waited for by its place among the loads and stores and not by the end of them all.
// A descriptor of no bytes stands for an array that is not there.  `cols` are the row's
// whole pieces of 8; the values behind them are its tail, one a lane.
typedef __amdgpu_buffer_rsrc_t Row;
__device__ __forceinline__ Row row_of(const void *base, uint64_t at, uint32_t cols, uint32_t size) {
    // (word 3: plain 32-bit data)
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(static_cast<const uint8_t *>(base)) + at * size, 0,
                                             base ? (int)(cols * size) : 0, 0x00020000);
}
// ONCE: nothing reads it again, and rows start on 16 bytes, so that no line is shared by two accesses.
template <bool F32, bool ONCE>
__device__ __forceinline__ void load_row(Row r, uint32_t c, Eight<F32> &v) {
#pragma unroll
    for (uint32_t i = 0; i < (F32 ? 2 : 1); ++i)
        v.w[i] = __builtin_bit_cast(u32v4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(c * (F32 ? 4 : 2) + 16 * i), 0, ONCE ? 2 : 0));
}
template <bool F32, bool ONCE>
__device__ __forceinline__ void store_row(Row r, uint32_t c, const float (&v)[8]) {
    if (F32) {
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(
                u32v4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                      __float_as_uint(v[4 * i + 3])},
                r, (int)(c * 4 + 16 * i), 0, ONCE ? 2 : 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b128(pack8(v), r, (int)(c * 2), 0, ONCE ? 2 : 0);
    }
}

// One value of a row's tail.
template <bool F32>
__device__ __forceinline__ float load_tail(Row r, uint32_t c) {
    if (F32) return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)(c * 4), 0, 0));
    return bf_one((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(c * 2), 0, 0));
}
template <bool F32>
__device__ __forceinline__ void store_tail(Row r, uint32_t c, float v) {
    if (F32)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)(c * 4), 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(bf_round(v), r, (int)(c * 2), 0, 0);
}
__device__ __forceinline__ float keep_tail(const Param &q, uint32_t c, bool on, float otherwise) {
    if (!on) return 0.0f;
    if (!q.p) return otherwise;
    return q.f32 ? static_cast<const float *>(q.p)[c] : bf_one(static_cast<const uint16_t *>(q.p)[c]);
}

// A parameter's values of a lane for all rows: floats, or BF16 pairs where every
// parameter is BF16.  `otherwise` where there is no parameter, 0 past the row's end.
template <bool F32>
__device__ __forceinline__ void keep_param(const Param &q, uint32_t c, uint32_t n, float otherwise, Eight<F32> &v) {
    float w[8];
    load_param(q, c, n, otherwise, w);
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) w[i] = n ? w[i] : 0.0f;
    if (F32) {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v.w[i / 4 % (F32 ? 2 : 1)][i & 3] = __float_as_uint(w[i]);
    } else {
        v.w[0] = pack8(w);
    }
}

constexpr uint32_t block_threads(uint32_t team) { return team < 256 ? 256 : team; }
constexpr uint32_t block_teams(uint32_t team) { return team < 256 ? 256 / team : 1; }
// Waves that a SIMD holds of the forward kernel of whole rows, whatever its team.
constexpr uint32_t kRowsWaves = 4;

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// A row's team: the fewest lanes that hold it in registers.
struct Shape {
    uint32_t team, chunks;
};
inline Shape shape_of(uint64_t cols) {
    if (cols <= 512) return {64, 1};
    if (cols <= 1024) return {64, 2};
    if (cols <= 2048) return {256, 1};
    if (cols <= 4096) return {512, 1};
    if (cols <= 8192) return {512, 2};
    return {1024, 2};
}
// Blocks of the backward pass: each keeps sums over its rows.
inline uint64_t backward_blocks(uint64_t rows, const Shape &s) {
    const uint64_t most = s.team > 256 ? 256 : 512, need = ceil_div(rows, block_teams(s.team));
    return need < most ? need : most;
}

// Calls go(team, chunks) with the shape as constants.
template <typename Go>
inline void with_shape(const Shape &s, Go go) {
    typedef std::integral_constant<uint32_t, 1> C1;
    typedef std::integral_constant<uint32_t, 2> C2;
    if (s.team == 64)
        s.chunks == 1 ? go(std::integral_constant<uint32_t, 64>{}, C1{}) : go(std::integral_constant<uint32_t, 64>{}, C2{});
    else if (s.team == 256)
        go(std::integral_constant<uint32_t, 256>{}, C1{});
    else if (s.team == 512)
        s.chunks == 1 ? go(std::integral_constant<uint32_t, 512>{}, C1{}) : go(std::integral_constant<uint32_t, 512>{}, C2{});
    else
        go(std::integral_constant<uint32_t, 1024>{}, C2{});
}
inline bool finite(float v) { return v - v == 0.0f; }
inline bool side_ok(const zc_norm_params &p) {
    return p.kind == ZC_NORM_NONE ||
           (p.kind <= ZC_NORM_LAYER && p.type <= ZC_BF16 && finite(p.eps) && p.eps >= 0x1p-126f);
}
inline bool param_aligned(const void *p, uint32_t type) { return aligned(p, type == ZC_F32 ? 4 : 2); }
inline bool side_aligned(const zc_norm_params &p) {
    return p.kind == ZC_NORM_NONE || (param_aligned(p.d_weight, p.type) && param_aligned(p.d_bias, p.type));
}
inline NormSide side(const zc_norm_params &p) {
    return {{p.d_weight, p.type == ZC_F32}, {p.d_bias, p.type == ZC_F32}, p.kind, p.eps};
}
inline bool stride_ok(const void *p, uint64_t stride, uint64_t cols) {
    return !p || (stride >= cols && stride <= kMaxStride);
}
// Rows that start on 16 bytes.
inline bool wide8(const void *p, uint64_t stride, bool f32 = false) {
    return !p || (aligned(p, 16) && stride % (f32 ? 4 : 8) == 0);
}

inline zc_status check(const zc_norm_config *cfg, uint32_t stream_type, uint64_t rows, uint64_t cols, bool branch) {
    if (!cfg || stream_type > ZC_BF16 || rows > kMaxRows || cols > ZC_NORM_MAX_COLS || !side_ok(cfg->before))
        return ZC_ERR_INVALID_ARG;
    if (branch && (!side_ok(cfg->after) || !finite(cfg->scale) || (cfg->d_gate && cfg->gate_type > ZC_BF16)))
        return ZC_ERR_INVALID_ARG;
    if (!side_aligned(cfg->before)) return ZC_ERR_MISALIGNED;
    if (branch && (!side_aligned(cfg->after) || !param_aligned(cfg->d_gate, cfg->gate_type) || !aligned(cfg->d_row_gate, 4)))
        return ZC_ERR_MISALIGNED;
    return ZC_OK;
}

inline NormArgs common(const zc_norm_config &cfg, uint64_t rows, uint64_t cols, bool branch) {
    NormArgs a = {};
    a.before = side(cfg.before);
    if (branch) {
        a.after = side(cfg.after);
        a.gate = {cfg.d_gate, cfg.gate_type == ZC_F32};
        a.row_gate = cfg.d_row_gate;
        a.scale = cfg.scale;
    }
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.inv_cols = 1.0f / (float)cols;
    return a;
}

// Whether a parameter that is read is not BF16.
inline bool any_float(const zc_norm_config &c, bool branch) {
    const auto has = [](const zc_norm_params &p) { return p.kind != ZC_NORM_NONE && (p.d_weight || p.d_bias) && p.type == ZC_F32; };
    return has(c.before) || (branch && (has(c.after) || (c.d_gate && c.gate_type == ZC_F32)));
}

}  // namespace moe
}  // namespace zc
