// Gradients of the norms on both sides of a block, its gate and the residual sum,
// MI355X / gfx950.  Bound by memory: every array is read once and written once, and
// the sums over the rows are kept in registers.
#include "zc_norm.h"

namespace zc {
namespace moe {

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

// Both halves' statistics at once: x before the norm `before`, z before the norm `after`.
// MEAN: one of them may be a LAYER norm.
template <bool MEAN, uint32_t TEAM, uint32_t CHUNKS, typename X, typename Z>
__device__ __forceinline__ void both_stats(X &x, Z &z, const uint32_t (&n)[CHUNKS], const NormArgs &a, bool pre,
                                           bool post, Stat &sx, Stat &sz, Team<TEAM> &team, float xt, float zt, bool in_tail) {
    const Measured<TEAM, CHUNKS, X> mx = {x, n, team, MEAN ? a.before.kind : ZC_NORM_RMS, a.before.eps, a.inv_cols, xt, in_tail};
    const Measured<TEAM, CHUNKS, Z> mz = {z, n, team, MEAN ? a.after.kind : ZC_NORM_RMS, a.after.eps, a.inv_cols, zt, in_tail};
    const bool lx = MEAN && pre && a.before.kind == ZC_NORM_LAYER, lz = MEAN && post && a.after.kind == ZC_NORM_LAYER;
    float mean[2] = {0.0f, 0.0f};
    Deviations s[2];
    if (MEAN && (lx || lz)) {
        float u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float m[2] = {xt, zt};
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                m[0] += x[i][j];
                m[1] += z[i][j];
            }
        team.sum(m);
        mean[0] = lx ? mean_of(m[0], a.inv_cols) : 0.0f;
        mean[1] = lz ? mean_of(m[1], a.inv_cols) : 0.0f;
        u[2] = in_tail ? xt - mean[0] : 0.0f;
        u[3] = in_tail ? zt - mean[1] : 0.0f;
        u[0] = u[2] * u[2];
        u[1] = u[3] * u[3];
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const float dx = n[i] ? x[i][j] - mean[0] : 0.0f, dz = n[i] ? z[i][j] - mean[1] : 0.0f;
                u[0] = fmaf(dx, dx, u[0]);
                u[1] = fmaf(dz, dz, u[1]);
                u[2] += dx;
                u[3] += dz;
            }
        team.sum(u);
        s[0] = beside_rest(u[0], lx ? u[2] : 0.0f, a.inv_cols);
        s[1] = beside_rest(u[1], lz ? u[3] : 0.0f, a.inv_cols);
    } else {
        float t[2] = {xt * xt, zt * zt};
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                t[0] = fmaf(x[i][j], x[i][j], t[0]);
                t[1] = fmaf(z[i][j], z[i][j], t[1]);
            }
        team.sum(t);
        s[0] = {0.0f, t[0], 0.0f};
        s[1] = {0.0f, t[1], 0.0f};
    }
    if (pre) sx = mx.settle(mean[0], s[0]);
    if (post) sz = mz.settle(mean[1], s[1]);
}

// With v^ the normed value and u = dy * w the gradient there, that of v is
//   1 / deviation * (u - v^ mean(u v^) [- mean(u) for LAYER]).
// A team's lanes keep their columns from row to row, so the sums over the rows
// stay in registers until the team's last row and leave as one part a team; a
// second launch adds the parts in order.  The next row's loads are on their way while a row is worked on,
// and weights and gate stay in registers.  Values past a row's end read as 0, have a gradient of 0, and add nothing.
//
// ANY: with biases, means and the rows' gates; without, about 34 instructions a value, which bound the kernel
// beside the memory: 8192 x 7168 takes 178 us with ANY and 128 without, 5.5 TB/s, past what a large copy
// reaches (246 without the loads ahead, and with loads under conditions).  Its registers would not hold the parameters
// beside five sums: ANY has them as floats in LDS, or, of rows past 8192, in memory.  WIDE: as in the forward kernel.
template <bool F32S, bool F32P, bool WIDE, bool ANY, uint32_t TEAM, uint32_t CHUNKS>
__global__ __launch_bounds__(block_threads(TEAM)) void norm_backward_kernel(NormArgs a) {
    __shared__ float parts[2][kMaxWaves][4];
    Team<TEAM> team = {parts, 0};
    const uint32_t sub = threadIdx.x % TEAM, whole = a.cols / 8 * 8, ct = whole + sub;
    const bool in_tail = !WIDE && ct < a.cols;
    const uint32_t index = (uint32_t)__builtin_amdgcn_readfirstlane(blockIdx.x * block_teams(TEAM) + threadIdx.x / TEAM);
    uint32_t n[CHUNKS];
    float dw1[CHUNKS][8], dgate[CHUNKS][8], dw2[CHUNKS][8], db1[ANY ? CHUNKS : 1][8], db2[ANY ? CHUNKS : 1][8];
    enum { kW1, kB1, kGate, kW2, kParams };
    constexpr bool kInLds = ANY && TEAM * CHUNKS <= 1024;
    constexpr uint32_t kRegs = ANY ? 1 : CHUNKS;
    Eight<F32P> w1[kRegs], gate[kRegs], w2[kRegs];
    // (a lane's values in two places, so that lanes side by side read 16 bytes side by side)
    __shared__ alignas(16) float kept[kInLds ? kParams : 1][2][kInLds ? TEAM * CHUNKS * 4 : 4];
    const bool pre = a.dy && a.before.kind != ZC_NORM_NONE, post = a.z && a.after.kind != ZC_NORM_NONE;
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const uint32_t c = (i * TEAM + sub) * 8;
        n[i] = c < whole ? 8u : 0u;
        if (!ANY) {
            keep_param<F32P>(post ? a.after.w : Param{}, c, n[i], 1.0f, w1[ANY ? 0 : i]);
            keep_param<F32P>(a.z ? a.gate : Param{}, c, n[i], 1.0f, gate[ANY ? 0 : i]);
            keep_param<F32P>(pre ? a.before.w : Param{}, c, n[i], 1.0f, w2[ANY ? 0 : i]);
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            dw1[i][j] = dgate[i][j] = dw2[i][j] = 0.0f;
            if (ANY) db1[ANY ? i : 0][j] = db2[ANY ? i : 0][j] = 0.0f;
        }
    }
    const auto param = [&](uint32_t k) -> Param {
        return k == kGate ? (a.z ? a.gate : Param{}) : k == kW2 ? (pre ? a.before.w : Param{}) : !post ? Param{} : k == kW1 ? a.after.w : a.after.b;
    };
    if constexpr (kInLds) {
        for (uint32_t q = threadIdx.x; q < TEAM * CHUNKS; q += block_threads(TEAM))
#pragma unroll
            for (uint32_t k = 0; k < kParams; ++k) {
                Eight<true> v;
                keep_param<true>(param(k), 8 * q, 8 * q < whole ? 8u : 0u, k == kB1 ? 0.0f : 1.0f, v);
                *reinterpret_cast<u32v4 *>(&kept[k][0][4 * q]) = v.w[0];
                *reinterpret_cast<u32v4 *>(&kept[k][1][4 * q]) = v.w[1];
            }
        __syncthreads();
    }
    // parameter k of a lane's chunk i
    const auto values = [&](auto k_t, uint32_t i, float (&v)[8]) {
        constexpr uint32_t k = decltype(k_t)::value;
        if constexpr (kInLds) {
            const float *at = &kept[k][0][(i * TEAM + sub) * 4];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) v[j] = at[j / 4 * (TEAM * CHUNKS * 4) + (j & 3)];
        } else if constexpr (ANY) {
            load_param(param(k), (i * TEAM + sub) * 8, n[i], k == kB1 ? 0.0f : 1.0f, v);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) v[j] = n[i] ? v[j] : 0.0f;
        } else {
            const Eight<F32P> &e = k == kW1 ? w1[i % kRegs] : k == kGate ? gate[i % kRegs] : w2[i % kRegs];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) v[j] = k == kB1 ? 0.0f : e[j];
        }
    };
    typedef std::integral_constant<uint32_t, kW1> W1;
    typedef std::integral_constant<uint32_t, kB1> B1;
    typedef std::integral_constant<uint32_t, kGate> Gate;
    typedef std::integral_constant<uint32_t, kW2> W2;
    const float w1t = keep_tail(post ? a.after.w : Param{}, ct, in_tail, 1.0f);
    const float b1t = ANY ? keep_tail(post ? a.after.b : Param{}, ct, in_tail, 0.0f) : 0.0f;
    const float gatet = keep_tail(a.z ? a.gate : Param{}, ct, in_tail, 1.0f);
    const float w2t = keep_tail(pre ? a.before.w : Param{}, ct, in_tail, 1.0f);
    float dw1t = 0.0f, db1t = 0.0f, dgatet = 0.0f, dw2t = 0.0f, db2t = 0.0f;
    struct Loaded {
        Eight<F32S> x[CHUNKS], dr[CHUNKS];
        Eight<false> z[CHUNKS], dy[CHUNKS];
        float xt, drt, zt, dyt;
    };
    const auto fetch = [&](uint32_t t, Loaded &v) {
        constexpr uint32_t size = F32S ? 4 : 2;
        const Row rx = row_of(a.x, t * a.x_stride, whole, size), rz = row_of(a.z, t * a.z_stride, whole, 2);
        const Row rd = row_of(a.dr, t * a.dr_stride, whole, size), ry = row_of(a.dy, t * a.dy_stride, whole, 2);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            const uint32_t c = (i * TEAM + sub) * 8;
            load_row<F32S, WIDE>(rx, c, v.x[i]);
            load_row<false, WIDE>(rz, c, v.z[i]);
            load_row<false, WIDE>(ry, c, v.dy[i]);
            load_row<F32S, WIDE>(rd, c, v.dr[i]);
        }
        v.xt = v.drt = v.zt = v.dyt = 0.0f;
        if (!WIDE) {
            v.xt = load_tail<F32S>(row_of(a.x, t * a.x_stride, a.cols, size), ct);
            v.zt = load_tail<false>(row_of(a.z, t * a.z_stride, a.cols, 2), ct);
            v.dyt = load_tail<false>(row_of(a.dy, t * a.dy_stride, a.cols, 2), ct);
            v.drt = load_tail<F32S>(row_of(a.dr, t * a.dr_stride, a.cols, size), ct);
        }
    };
    const uint32_t step = gridDim.x * block_teams(TEAM);
    uint32_t row = index;
    Loaded v;
    if (row < a.rows) fetch(row, v);
    while (row < a.rows) {
        Loaded next;
        fetch(row + step < a.rows ? row + step : a.rows - 1, next);
#pragma unroll
        for (uint32_t i = 0; i < kRegs; ++i) {
            stay_packed(w1[i]);
            stay_packed(gate[i]);
            stay_packed(w2[i]);
        }
        const float rg = ANY && a.row_gate ? a.row_gate[row] : 1.0f;
        Stat sx = kNoNorm, sz = kNoNorm;
        if (pre || post) both_stats<ANY, TEAM, CHUNKS>(v.x, v.z, n, a, pre, post, sx, sz, team, v.xt, v.zt, in_tail);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            stay_packed(v.x[i]);
            stay_packed(v.z[i]);
            stay_packed(v.dy[i]);
            stay_packed(v.dr[i]);
        }
        float g[CHUNKS][8];  // the gradient of r
        float gt = 0.0f;
        if (pre) {
            float t[2] = {0.0f, 0.0f};
            const float ht = WIDE ? 0.0f : normed<ANY>(v.xt, sx);
            if (!WIDE) {
                dw2t = fmaf(v.dyt, ht, dw2t);
                if (ANY) db2t += v.dyt;
                gt = v.dyt * w2t;
                t[0] = gt * ht;
                if (ANY) t[1] = gt;
            }
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                float w[8];
                values(W2{}, i, w);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float h = normed<ANY>(v.x[i][j], sx), d = v.dy[i][j];
                    dw2[i][j] = fmaf(d, h, dw2[i][j]);
                    if (ANY) db2[ANY ? i : 0][j] += d;
                    g[i][j] = d * w[j];
                    t[0] = fmaf(g[i][j], h, t[0]);
                    if (ANY) t[1] += g[i][j];
                }
            }
            float m0, m1 = 0.0f;
            if (ANY) {
                team.sum(t);
                m0 = t[0] * a.inv_cols;
                if (a.before.kind == ZC_NORM_LAYER) m1 = t[1] * a.inv_cols;
            } else {
                float u[1] = {t[0]};
                team.sum(u);
                m0 = u[0] * a.inv_cols;
            }
            if (!WIDE) {
                const float u = fmaf(-ht, m0, gt);
                gt = fmaf(ANY ? u - m1 : u, sx.slope, v.drt);
            }
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) stay_packed(v.x[i]);
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float u = fmaf(-normed<ANY>(v.x[i][j], sx), m0, g[i][j]);
                    g[i][j] = fmaf(ANY ? u - m1 : u, sx.slope, v.dr[i][j]);
                }
        } else {
            gt = v.drt + v.dyt;
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) g[i][j] = v.dr[i][j] + v.dy[i][j];
        }
        const Row rr = row_of(a.r, row * a.r_stride, whole, F32S ? 4 : 2);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) store_row<F32S, WIDE>(rr, (i * TEAM + sub) * 8, g[i]);
        if (!WIDE) store_tail<F32S>(row_of(a.r, row * a.r_stride, a.cols, F32S ? 4 : 2), ct, gt);
        const float share = ANY ? a.scale * rg : a.scale;
        float t[3] = {0.0f, 0.0f, 0.0f};
        const float zht = WIDE ? 0.0f : normed<ANY>(v.zt, sz);
        if (!WIDE) {
            const float e = in_tail ? gt : 0.0f, q = e * fmaf(zht, w1t, b1t), dh = gatet * e * share;
            dgatet = fmaf(share, q, dgatet);
            if (ANY) t[2] = gatet * q;
            dw1t = fmaf(dh, zht, dw1t);
            if (ANY) db1t += dh;
            gt = dh * w1t;
            t[0] = gt * zht;
            if (ANY) t[1] = gt;
        }
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            float b[8], w[8], gate_v[8];
            values(W1{}, i, w);
            values(Gate{}, i, gate_v);
            values(B1{}, i, b);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const float zh = normed<ANY>(v.z[i][j], sz);  // z itself without a norm
                const float h = ANY ? fmaf(zh, w[j], b[j]) : zh * w[j];
                const float e = ANY ? (n[i] ? g[i][j] : 0.0f) : g[i][j], q = e * h;
                dgate[i][j] = fmaf(share, q, dgate[i][j]);
                if (ANY) t[2] = fmaf(gate_v[j], q, t[2]);
                const float dh = gate_v[j] * e * share;
                dw1[i][j] = fmaf(dh, zh, dw1[i][j]);
                if (ANY) db1[ANY ? i : 0][j] += dh;
                g[i][j] = dh * w[j];
                t[0] = fmaf(g[i][j], zh, t[0]);
                if (ANY) t[1] += g[i][j];
            }
        }
        float m0 = 0.0f, m1 = 0.0f;
        if (ANY) {
            if (a.drow_gate || post) team.sum(t);
            if (a.drow_gate && sub == 0) a.drow_gate[row] = a.z ? a.scale * t[2] : 0.0f;
            m0 = t[0] * a.inv_cols;
            if (a.after.kind == ZC_NORM_LAYER) m1 = t[1] * a.inv_cols;
        } else if (post) {
            float u[1] = {t[0]};
            team.sum(u);
            m0 = u[0] * a.inv_cols;
        }
        const Row rz = row_of(a.dz, row * a.dz_stride, whole, 2);
        if (!WIDE) {
            if (post) {
                const float u = fmaf(-zht, m0, gt);
                gt = (ANY ? u - m1 : u) * sz.slope;
            }
            store_tail<false>(row_of(a.dz, row * a.dz_stride, a.cols, 2), ct, gt);
        }
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            stay_packed(v.z[i]);
            if (post)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float u = fmaf(-normed<ANY>(v.z[i][j], sz), m0, g[i][j]);
                    g[i][j] = (ANY ? u - m1 : u) * sz.slope;
                }
            store_row<false, WIDE>(rz, (i * TEAM + sub) * 8, g[i]);
        }
        row += step;
        v = next;
    }
    const auto part = [&](uint32_t sum, uint32_t c) { return a.parts + sum * a.part_stride + (uint64_t)index * a.cols + c; };
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const auto leave = [&](uint32_t sum, const float (&s)[8]) {
            if (a.sums >> sum & 1) store_floats(part(sum, (i * TEAM + sub) * 8), n[i], s);
        };
        leave(kDW1, dw1[i]);
        leave(kDGate, dgate[i]);
        leave(kDW2, dw2[i]);
        if (ANY) {
            leave(kDB1, db1[ANY ? i : 0]);
            leave(kDB2, db2[ANY ? i : 0]);
        }
    }
    if (!in_tail) return;
    const auto leave = [&](uint32_t sum, float s) {
        if (a.sums >> sum & 1) *part(sum, ct) = s;
    };
    leave(kDW1, dw1t);
    leave(kDGate, dgatet);
    leave(kDW2, dw2t);
    if (ANY) {
        leave(kDB1, db1t);
        leave(kDB2, db2t);
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
// 64 columns of one sum a block, its parts in order, in 16 runs side by side: 256 parts of three sums of 7168 columns
// 4.9 us (22 MB), of five of 5125 6.1: a launch and the latency of 16 loads in a row.
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

static void launch_backward(const NormArgs &a, const Shape &s, bool wide, bool f32, bool f32p, bool any, dim3 grid,
                            Launches &on) {
    with_shape(s, [&](auto team, auto chunks) {
        constexpr uint32_t T = decltype(team)::value, C = decltype(chunks)::value;
        const auto pick = [&](auto f32_t, auto any_t) {
            constexpr bool S = decltype(f32_t)::value, A = decltype(any_t)::value;
            // (with ANY the parameters' type in registers does not matter)
            on.launch(f32p && !A ? (wide ? norm_backward_kernel<S, !A, true, A, T, C> : norm_backward_kernel<S, !A, false, A, T, C>)
                                 : (wide ? norm_backward_kernel<S, false, true, A, T, C> : norm_backward_kernel<S, false, false, A, T, C>),
                      grid, dim3(block_threads(T)), a);
        };
        if (f32)
            any ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
        else
            any ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
    });
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

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
    NormArgs a = common(*cfg, rows, cols, d_z != nullptr);
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
    const bool f32 = stream_type == ZC_F32;
    const bool wide = cols % 8 == 0 && wide8(d_dx, dx_stride, f32) && wide8(d_dz, dz_stride) && wide8(d_r, r_stride, f32) &&
                      wide8(d_dr, dr_stride, f32) && wide8(d_dy, dy_stride) && wide8(d_z, z_stride);
    const bool any = a.sums & (1u << kDB1 | 1u << kDB2) || a.before.kind == ZC_NORM_LAYER || a.after.kind == ZC_NORM_LAYER ||
                     (a.after.kind != ZC_NORM_NONE && a.after.b.p) || a.row_gate || row_gate;
    Launches on(stream);
    if (rows && (a.sums || d_dx || d_dz || row_gate))
        launch_backward(a, s, wide, f32, any_float(*cfg, d_z != nullptr), any, dim3((uint32_t)blocks), on);
    if (asked) on.launch(norm_sums_kernel, dim3((uint32_t)ceil_div(cols, kLanes), kSums), dim3(kLanes * kSumRuns), sum);
    return on.status();
}
