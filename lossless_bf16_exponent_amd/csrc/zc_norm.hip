// Norms on both sides of a block with its gate and the residual sum, and their
// gradients, MI355X / gfx950:
//   h = N1(z);  r = x + scale * row_gate[t] * gate[c] * h;  y = N2(r)
// Bound by memory: a row stays in registers between its statistics and its
// results, so every array is read once and written once.
#include <math.h>

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
    uint32_t wide;
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

// The normed value of v is (v * unit - mean - rest) * rs; rest is what rounding
// the mean left of it, which counts where the deviation is small beside the mean.
// unit is 1 unless the squares
// would leave the range of a float: above 2^120 in sum (infinities and NaN among
// them), or below 2^-80 with an eps that does not cover them; the row is then
// taken 2^-80 or 2^80 times as large, which is exact for all values that matter.
struct Stat {
    float mean, rest, rs, unit;
};
__device__ __forceinline__ float normed(float v, const Stat &s) { return (fmaf(v, s.unit, -s.mean) - s.rest) * s.rs; }

template <uint32_t TEAM, uint32_t CHUNKS, typename V>
__device__ __forceinline__ Stat row_stat(const V &v, const uint32_t (&n)[CHUNKS], uint32_t kind, float eps,
                                         float inv_cols, Team<TEAM> &team) {
    Stat s = {0.0f, 0.0f, 1.0f, 1.0f};
    float var = 0.0f;
    const auto measure = [&]() {
        s.mean = s.rest = 0.0f;
        if (kind == ZC_NORM_LAYER) {
            float t[1] = {0.0f};
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) t[0] = fmaf(v[i][j], s.unit, t[0]);
            team.sum(t);
            s.mean = t[0] * inv_cols;
            float u[2] = {0.0f, 0.0f};
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float d = j < n[i] ? fmaf(v[i][j], s.unit, -s.mean) : 0.0f;
                    u[0] = fmaf(d, d, u[0]);
                    u[1] += d;
                }
            team.sum(u);
            s.rest = u[1] * inv_cols;
            // (where the difference is lost in rounding: not below 0, and NaN stays)
            const float left = fmaf(-s.rest, u[1], u[0]);
            var = left < 0.0f ? 0.0f : left;
        } else {
            float t[1] = {0.0f};
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float d = v[i][j] * s.unit;
                    t[0] = fmaf(d, d, t[0]);
                }
            team.sum(t);
            var = t[0];
        }
    };
    measure();
    if (!(var <= 0x1p120f) || (var < 0x1p-80f && eps < 0x1p-58f)) {
        s.unit = var < 1.0f ? 0x1p80f : 0x1p-80f;
        measure();
    }
    // eps in the row's unit (for large rows it is nothing beside their squares)
    s.rs = __builtin_amdgcn_rsqf(fmaf(var, inv_cols, eps * s.unit * s.unit));
    return s;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr uint32_t block_threads(uint32_t team) { return team < 256 ? 256 : team; }
constexpr uint32_t block_teams(uint32_t team) { return team < 256 ? 256 / team : 1; }

template <bool F32S, uint32_t TEAM, uint32_t CHUNKS>
__global__ __launch_bounds__(block_threads(TEAM)) void norm_kernel(NormArgs a) {
    __shared__ float parts[2][kMaxWaves][4];
    Team<TEAM> team = {parts, 0};
    const uint32_t sub = threadIdx.x % TEAM;
    uint32_t n[CHUNKS];
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const uint32_t c = (i * TEAM + sub) * 8;
        n[i] = c < a.cols ? min(a.cols - c, 8u) : 0u;
    }
    for (uint64_t row = (uint64_t)blockIdx.x * block_teams(TEAM) + threadIdx.x / TEAM; row < a.rows;
         row += (uint64_t)gridDim.x * block_teams(TEAM)) {
        Eight<F32S> x[CHUNKS];
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) x[i].load(a.x, row * a.x_stride + (i * TEAM + sub) * 8, n[i], true);
        float v[CHUNKS][8];
        if (a.z) {
            Eight<false> z[CHUNKS];
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) z[i].load(a.z, row * a.z_stride + (i * TEAM + sub) * 8, n[i], true);
            const float share = a.row_gate ? a.scale * a.row_gate[row] : a.scale;
            const bool on = a.after.kind != ZC_NORM_NONE;
            Stat s = {0.0f, 0.0f, 1.0f, 1.0f};
            if (on) s = row_stat<TEAM, CHUNKS>(z, n, a.after.kind, a.after.eps, a.inv_cols, team);
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                const uint32_t c = (i * TEAM + sub) * 8;
                float h[8], p[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) h[j] = z[i][j];
                if (on) {
#pragma unroll
                    for (uint32_t j = 0; j < 8; ++j) h[j] = normed(h[j], s);
                    if (a.after.w.p) {
                        load_param(a.after.w, c, n[i], 1.0f, p);
#pragma unroll
                        for (uint32_t j = 0; j < 8; ++j) h[j] *= p[j];
                    }
                    if (a.after.b.p) {
                        load_param(a.after.b, c, n[i], 0.0f, p);
#pragma unroll
                        for (uint32_t j = 0; j < 8; ++j) h[j] += p[j];
                    }
                }
                if (a.gate.p) {
                    load_param(a.gate, c, n[i], 1.0f, p);
#pragma unroll
                    for (uint32_t j = 0; j < 8; ++j) h[j] *= p[j];
                }
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) v[i][j] = j < n[i] ? fmaf(share, h[j], x[i][j]) : 0.0f;
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) v[i][j] = x[i][j];
        }
        if (a.r)
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
                store_stream<F32S>(a.r, row * a.r_stride + (i * TEAM + sub) * 8, n[i], v[i], a.wide);
        if (!a.y && !a.yq) continue;
        if (a.before.kind != ZC_NORM_NONE) {
            const Stat s = row_stat<TEAM, CHUNKS>(v, n, a.before.kind, a.before.eps, a.inv_cols, team);
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                const uint32_t c = (i * TEAM + sub) * 8;
                float w[8], b[8];
                load_param(a.before.w, c, n[i], 1.0f, w);
                load_param(a.before.b, c, n[i], 0.0f, b);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) v[i][j] = j < n[i] ? fmaf(normed(v[i][j], s), w[j], b[j]) : 0.0f;
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            const uint32_t c = (i * TEAM + sub) * 8;
            const u32v4 w = pack8(v[i]);
            if (a.y) store_bf(a.y + row * a.y_stride + c, w, n[i], a.wide);
            // 16 lanes hold a block of 128; lanes past the last block have nothing to keep, whole blocks at a time
            if (a.yq && c < a.q_stride) {
                uint8_t *s = a.ys + row * a.qs_stride;
                keep8(w, a.yq + row * a.q_stride + c, s + c / kBlock, sub % kKeepLanes);
                const uint32_t pad = c / kBlock + sub % kKeepLanes;
                if (c / kBlock + 1 == a.q_stride / kBlock && sub % kKeepLanes > 0 && pad < a.qs_stride) s[pad] = 0;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// With v^ the normed value and u = dy * w the gradient there, that of v is
//   1 / deviation * (u - v^ mean(u v^) [- mean(u) for LAYER]).
// A team's lanes keep their columns from row to row, so the sums over the rows
// stay in registers until the team's last row and leave as one part a team; a
// second launch adds the parts in order.  BIAS: with the biases' sums.  Columns past
// the end read as 0 and have a gradient of 0, so they add nothing.
template <bool F32S, bool BIAS, uint32_t TEAM, uint32_t CHUNKS>
__global__ __launch_bounds__(block_threads(TEAM)) void norm_backward_kernel(NormArgs a) {
    __shared__ float parts[2][kMaxWaves][4];
    Team<TEAM> team = {parts, 0};
    const uint32_t sub = threadIdx.x % TEAM, index = blockIdx.x * block_teams(TEAM) + threadIdx.x / TEAM;
    uint32_t n[CHUNKS];
    float dw1[CHUNKS][8], dgate[CHUNKS][8], dw2[CHUNKS][8], db1[BIAS ? CHUNKS : 1][8], db2[BIAS ? CHUNKS : 1][8];
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const uint32_t c = (i * TEAM + sub) * 8;
        n[i] = c < a.cols ? min(a.cols - c, 8u) : 0u;
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            dw1[i][j] = dgate[i][j] = dw2[i][j] = 0.0f;
            if (BIAS) db1[BIAS ? i : 0][j] = db2[BIAS ? i : 0][j] = 0.0f;
        }
    }
    const bool pre = a.before.kind != ZC_NORM_NONE, post = a.after.kind != ZC_NORM_NONE;
    for (uint64_t row = index; row < a.rows; row += (uint64_t)gridDim.x * block_teams(TEAM)) {
        Eight<F32S> x[CHUNKS], dr[CHUNKS];
        Eight<false> dy[CHUNKS], z[CHUNKS];
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            const uint32_t c = (i * TEAM + sub) * 8;
            if (a.dy && pre) x[i].load(a.x, row * a.x_stride + c, n[i], true);
            dr[i].clear();
            dy[i].clear();
            if (a.dy) dy[i].load(a.dy, row * a.dy_stride + c, n[i], true);
            if (a.dr) dr[i].load(a.dr, row * a.dr_stride + c, n[i], true);
            if (a.z) z[i].load(a.z, row * a.z_stride + c, n[i], true);
        }
        float g[CHUNKS][8];  // the gradient of r
        if (a.dy && pre) {
            const Stat s = row_stat<TEAM, CHUNKS>(x, n, a.before.kind, a.before.eps, a.inv_cols, team);
            float t[2] = {0.0f, 0.0f};
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                float w[8];
                load_param(a.before.w, (i * TEAM + sub) * 8, n[i], 1.0f, w);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float v = normed(x[i][j], s);
                    dw2[i][j] = fmaf(dy[i][j], v, dw2[i][j]);
                    if (BIAS) db2[BIAS ? i : 0][j] += dy[i][j];
                    g[i][j] = dy[i][j] * w[j];
                    t[0] = fmaf(g[i][j], v, t[0]);
                    t[1] += g[i][j];
                }
            }
            team.sum(t);
            const float m0 = t[0] * a.inv_cols, m1 = a.before.kind == ZC_NORM_LAYER ? t[1] * a.inv_cols : 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    g[i][j] = fmaf((fmaf(-normed(x[i][j], s), m0, g[i][j]) - m1) * s.rs, s.unit, dr[i][j]);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) g[i][j] = dr[i][j] + dy[i][j];
        }
        if (a.r)
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
                store_stream<F32S>(a.r, row * a.r_stride + (i * TEAM + sub) * 8, n[i], g[i], a.wide);
        if (!a.z) {
            if (a.drow_gate && sub == 0) a.drow_gate[row] = 0.0f;
            continue;
        }
        const float rg = a.row_gate ? a.row_gate[row] : 1.0f;
        Stat s = {0.0f, 0.0f, 1.0f, 1.0f};
        if (post) s = row_stat<TEAM, CHUNKS>(z, n, a.after.kind, a.after.eps, a.inv_cols, team);
        float t[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            const uint32_t c = (i * TEAM + sub) * 8;
            float gate[8], w[8], h[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                g[i][j] = c + j < a.cols ? a.scale * g[i][j] : 0.0f;  // at gate * row_gate * h
                h[j] = z[i][j];
                w[j] = 1.0f;
            }
            if (post) {
                load_param(a.after.w, c, n[i], 1.0f, w);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) h[j] = normed(h[j], s) * w[j];
                if (a.after.b.p) {
                    float b[8];
                    load_param(a.after.b, c, n[i], 0.0f, b);
#pragma unroll
                    for (uint32_t j = 0; j < 8; ++j) h[j] += b[j];
                }
            }
            load_param(a.gate, c, n[i], 1.0f, gate);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                dgate[i][j] = fmaf(rg * g[i][j], h[j], dgate[i][j]);
                t[0] = fmaf(gate[j] * g[i][j], h[j], t[0]);
                const float dh = rg * gate[j] * g[i][j], v = normed(z[i][j], s);
                dw1[i][j] = fmaf(dh, v, dw1[i][j]);
                if (BIAS) db1[BIAS ? i : 0][j] += dh;
                g[i][j] = dh * w[j];
                t[1] = fmaf(g[i][j], v, t[1]);
                t[2] += g[i][j];
            }
        }
        if (a.drow_gate || (post && a.dz)) team.sum(t);
        if (a.drow_gate && sub == 0) a.drow_gate[row] = t[0];
        if (!a.dz) continue;
        const float m0 = t[1] * a.inv_cols, m1 = a.after.kind == ZC_NORM_LAYER ? t[2] * a.inv_cols : 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            if (post)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    g[i][j] = (fmaf(-normed(z[i][j], s), m0, g[i][j]) - m1) * s.rs * s.unit;
            store_bf(a.dz + row * a.dz_stride + (i * TEAM + sub) * 8, pack8(g[i]), n[i], a.wide);
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const auto leave = [&](uint32_t sum, const float (&v)[8]) {
            if (a.sums >> sum & 1)
                store_floats(a.parts + sum * a.part_stride + (uint64_t)index * a.cols + (i * TEAM + sub) * 8, n[i], v);
        };
        leave(kDW1, dw1[i]);
        leave(kDGate, dgate[i]);
        leave(kDW2, dw2[i]);
        if (BIAS) {
            leave(kDB1, db1[BIAS ? i : 0]);
            leave(kDB2, db2[BIAS ? i : 0]);
        }
    }
}

// The parts of the sums over the rows, added in order: 64 columns a block, their
// parts cut into 16 runs.
struct SumArgs {
    const float *parts;
    float *out[kSums];
    uint64_t part_stride;
    uint32_t count, cols, live;  // live: sums that have parts; the others are zeros
};
constexpr uint32_t kSumRuns = 16;
__global__ __launch_bounds__(kLanes * kSumRuns) void norm_sums_kernel(SumArgs a) {
    __shared__ float run[kSumRuns][kLanes];
    float *out = a.out[blockIdx.y];
    if (!out) return;
    const uint32_t c = blockIdx.x * kLanes + lane_id(), w = threadIdx.x / kLanes;
    float v = 0.0f;
    if (c < a.cols && (a.live >> blockIdx.y & 1)) {
        const uint32_t i0 = (uint32_t)((uint64_t)a.count * w / kSumRuns), i1 = (uint32_t)((uint64_t)a.count * (w + 1) / kSumRuns);
        const float *src = a.parts + blockIdx.y * a.part_stride + (uint64_t)i0 * a.cols + c;
#pragma unroll 8
        for (uint32_t i = i0; i < i1; ++i, src += a.cols) v += *src;
    }
    run[w][lane_id()] = v;
    __syncthreads();
    if (w || c >= a.cols) return;
#pragma unroll
    for (uint32_t i = 1; i < kSumRuns; ++i) v += run[i][lane_id()];
    out[c] = v;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// A row's team: the fewest lanes that hold it in registers.
struct Shape {
    uint32_t team, chunks;
};
static Shape shape_of(uint64_t cols) {
    if (cols <= 512) return {64, 1};
    if (cols <= 1024) return {64, 2};
    if (cols <= 2048) return {256, 1};
    if (cols <= 4096) return {512, 1};
    if (cols <= 8192) return {512, 2};
    return {1024, 2};
}
// Blocks of the backward pass: each keeps sums over its rows.
static uint64_t backward_blocks(uint64_t rows, const Shape &s) {
    const uint64_t most = s.team > 256 ? 256 : 512, need = ceil_div(rows, block_teams(s.team));
    return need < most ? need : most;
}

// Calls go(team, chunks) with the shape as constants.
template <typename Go>
static void with_shape(const Shape &s, Go go) {
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
static void launch_forward(const NormArgs &a, const Shape &s, bool f32, dim3 grid, Launches &on) {
    with_shape(s, [&](auto team, auto chunks) {
        constexpr uint32_t T = decltype(team)::value, C = decltype(chunks)::value;
        on.launch(f32 ? norm_kernel<true, T, C> : norm_kernel<false, T, C>, grid, dim3(block_threads(T)), a);
    });
}
static void launch_backward(const NormArgs &a, const Shape &s, bool f32, bool bias, dim3 grid, Launches &on) {
    with_shape(s, [&](auto team, auto chunks) {
        constexpr uint32_t T = decltype(team)::value, C = decltype(chunks)::value;
        on.launch(f32 ? (bias ? norm_backward_kernel<true, true, T, C> : norm_backward_kernel<true, false, T, C>)
                      : (bias ? norm_backward_kernel<false, true, T, C> : norm_backward_kernel<false, false, T, C>),
                  grid, dim3(block_threads(T)), a);
    });
}

static bool finite(float v) { return v - v == 0.0f; }
static bool side_ok(const zc_norm_params &p) {
    return p.kind == ZC_NORM_NONE ||
           (p.kind <= ZC_NORM_LAYER && p.type <= ZC_BF16 && finite(p.eps) && p.eps >= 0x1p-126f);
}
static bool param_aligned(const void *p, uint32_t type) { return aligned(p, type == ZC_F32 ? 4 : 2); }
static bool side_aligned(const zc_norm_params &p) {
    return p.kind == ZC_NORM_NONE || (param_aligned(p.d_weight, p.type) && param_aligned(p.d_bias, p.type));
}
static NormSide side(const zc_norm_params &p) {
    return {{p.d_weight, p.type == ZC_F32}, {p.d_bias, p.type == ZC_F32}, p.kind, p.eps};
}
static bool stride_ok(const void *p, uint64_t stride, uint64_t cols) {
    return !p || (stride >= cols && stride <= kMaxStride);
}
static bool wide8(const void *p, uint64_t stride) { return !p || (aligned(p, 16) && stride % 8 == 0); }  // of BF16 rows

static zc_status check(const zc_norm_config *cfg, uint32_t stream_type, uint64_t rows, uint64_t cols, bool branch) {
    if (!cfg || stream_type > ZC_BF16 || rows > kMaxRows || cols > ZC_NORM_MAX_COLS || !side_ok(cfg->before))
        return ZC_ERR_INVALID_ARG;
    if (branch && (!side_ok(cfg->after) || !finite(cfg->scale) || (cfg->d_gate && cfg->gate_type > ZC_BF16)))
        return ZC_ERR_INVALID_ARG;
    if (!side_aligned(cfg->before)) return ZC_ERR_MISALIGNED;
    if (branch && (!side_aligned(cfg->after) || !param_aligned(cfg->d_gate, cfg->gate_type) || !aligned(cfg->d_row_gate, 4)))
        return ZC_ERR_MISALIGNED;
    return ZC_OK;
}

static NormArgs common(const zc_norm_config &cfg, uint64_t rows, uint64_t cols) {
    NormArgs a = {};
    a.after = side(cfg.after);
    a.before = side(cfg.before);
    a.gate = {cfg.d_gate, cfg.gate_type == ZC_F32};
    a.row_gate = cfg.d_row_gate;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.scale = cfg.scale;
    a.inv_cols = 1.0f / (float)cols;
    return a;
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" zc_status zc_norm(const void *d_x, uint32_t stream_type, uint64_t rows, uint64_t cols, uint64_t x_stride,
                             const void *d_z, uint64_t z_stride, const zc_norm_config *cfg, void *d_r,
                             uint64_t r_stride, void *d_y, uint64_t y_stride, void *d_yq, uint8_t *d_yq_scales,
                             void *stream) {
    const zc_status bad = check(cfg, stream_type, rows, cols, d_z != nullptr);
    if (bad == ZC_ERR_INVALID_ARG || x_stride < cols || x_stride > kMaxStride || !stride_ok(d_z, z_stride, cols) ||
        !stride_ok(d_r, r_stride, cols) || !stride_ok(d_y, y_stride, cols) || !d_yq != !d_yq_scales)
        return ZC_ERR_INVALID_ARG;
    if (bad) return bad;
    if (!rows || !cols || (!d_r && !d_y && !d_yq)) return ZC_OK;
    if (!d_x) return ZC_ERR_INVALID_ARG;
    const uint32_t size = stream_type == ZC_F32 ? 4 : 2;
    if (!aligned(d_x, size) || !aligned(d_z, 2) || !aligned(d_r, size) || !aligned(d_y, 2) || !aligned(d_yq, 16) ||
        !aligned(d_yq_scales, 4))
        return ZC_ERR_MISALIGNED;
    NormArgs a = common(*cfg, rows, cols);
    a.x = d_x;
    a.z = static_cast<const uint16_t *>(d_z);
    a.r = d_r;
    a.y = static_cast<uint16_t *>(d_y);
    a.yq = static_cast<uint8_t *>(d_yq);
    a.ys = d_yq_scales;
    a.x_stride = x_stride;
    a.z_stride = z_stride;
    a.r_stride = r_stride;
    a.y_stride = y_stride;
    a.q_stride = stride8(cols);
    a.qs_stride = scale_stride(cols);
    a.wide = cols % 8 == 0 && wide8(d_r, r_stride) && wide8(d_y, y_stride);
    const Shape s = shape_of(cols);
    const uint64_t blocks = ceil_div(rows, block_teams(s.team));
    Launches on(stream);
    launch_forward(a, s, stream_type == ZC_F32, dim3((uint32_t)(blocks < (1u << 20) ? blocks : 1u << 20)), on);
    return on.status();
}

extern "C" uint64_t zc_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols) {
    if (rows > kMaxRows || cols > ZC_NORM_MAX_COLS || !rows || !cols) return 0;
    const Shape s = shape_of(cols);
    return ceil_div(backward_blocks(rows, s) * block_teams(s.team) * cols * kSums * 4, 256) * 256;
}

extern "C" zc_status zc_norm_backward(const void *d_r, uint32_t stream_type, uint64_t rows, uint64_t cols,
                                      uint64_t r_stride, const void *d_z, uint64_t z_stride,
                                      const zc_norm_config *cfg, const void *d_dr, uint64_t dr_stride,
                                      const void *d_dy, uint64_t dy_stride, void *d_dx, uint64_t dx_stride,
                                      void *d_dz, uint64_t dz_stride, const zc_norm_grads *grads, void *d_workspace,
                                      uint64_t workspace_bytes, void *stream) {
    const zc_status bad = check(cfg, stream_type, rows, cols, d_z != nullptr);
    if (bad == ZC_ERR_INVALID_ARG || r_stride < cols || r_stride > kMaxStride || !stride_ok(d_z, z_stride, cols) ||
        !stride_ok(d_dr, dr_stride, cols) || !stride_ok(d_dy, dy_stride, cols) || !stride_ok(d_dx, dx_stride, cols) ||
        !stride_ok(d_dz, dz_stride, cols) || (d_dz && !d_z))
        return ZC_ERR_INVALID_ARG;
    if (bad) return bad;
    if (!cols) return ZC_OK;
    SumArgs sum = {};
    float *const row_gate = grads ? grads->d_row_gate : nullptr;
    if (grads) {
        sum.out[kDW1] = grads->d_weight_after;
        sum.out[kDB1] = grads->d_bias_after;
        sum.out[kDGate] = grads->d_gate;
        sum.out[kDW2] = grads->d_weight_before;
        sum.out[kDB2] = grads->d_bias_before;
    }
    uint32_t asked = 0;
    for (uint32_t k = 0; k < kSums; ++k) {
        if (!aligned(sum.out[k], 4)) return ZC_ERR_MISALIGNED;
        asked |= (uint32_t)(sum.out[k] != nullptr) << k;
    }
    if (!asked && (!rows || (!d_dx && !d_dz && !row_gate))) return ZC_OK;
    const uint32_t size = stream_type == ZC_F32 ? 4 : 2;
    if (!aligned(d_r, size) || !aligned(d_z, 2) || !aligned(d_dr, size) || !aligned(d_dy, 2) || !aligned(d_dx, size) ||
        !aligned(d_dz, 2) || !aligned(row_gate, 4) || !aligned(d_workspace, 16))
        return ZC_ERR_MISALIGNED;
    NormArgs a = common(*cfg, rows, cols);
    a.x = d_r;
    a.z = static_cast<const uint16_t *>(d_z);
    a.dr = d_dr;
    a.dy = static_cast<const uint16_t *>(d_dy);
    a.r = d_dx;
    a.dz = static_cast<uint16_t *>(d_dz);
    a.drow_gate = row_gate;
    a.x_stride = r_stride;
    a.z_stride = z_stride;
    a.dr_stride = dr_stride;
    a.dy_stride = dy_stride;
    a.r_stride = dx_stride;
    a.dz_stride = dz_stride;
    // which sums have anything to add: the rest are zeros
    uint32_t live = 0;
    if (d_z) live |= 1u << kDGate | (a.after.kind != ZC_NORM_NONE ? 1u << kDW1 | 1u << kDB1 : 0u);
    if (d_dy && a.before.kind != ZC_NORM_NONE) live |= 1u << kDW2 | 1u << kDB2;
    if (!rows) live = 0;
    a.sums = asked & live;
    const Shape s = shape_of(cols);
    const uint64_t blocks = rows ? backward_blocks(rows, s) : 0, count = blocks * block_teams(s.team);
    a.part_stride = sum.part_stride = count * cols;
    sum.count = (uint32_t)count;
    sum.cols = (uint32_t)cols;
    sum.live = a.sums;
    if (rows && !d_r) return ZC_ERR_INVALID_ARG;
    if (a.sums) {
        if (!d_workspace) return ZC_ERR_INVALID_ARG;
        if (workspace_bytes < zc_norm_backward_workspace_bytes(rows, cols)) return ZC_ERR_CAPACITY;
        a.parts = static_cast<float *>(d_workspace);
        sum.parts = a.parts;
    }
    a.wide = cols % 8 == 0 && wide8(d_dx, dx_stride) && wide8(d_dz, dz_stride);
    Launches on(stream);
    if (rows && (a.sums || d_dx || d_dz || row_gate))
        launch_backward(a, s, stream_type == ZC_F32, a.sums & (1u << kDB1 | 1u << kDB2), dim3((uint32_t)blocks), on);
    if (asked) on.launch(norm_sums_kernel, dim3((uint32_t)ceil_div(cols, kLanes), kSums), dim3(kLanes * kSumRuns), sum);
    return on.status();
}
