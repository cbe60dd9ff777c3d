// Norms on both sides of a block with its gate and the residual sum, MI355X / gfx950:
//   h = N1(z);  r = x + scale * row_gate[t] * gate[c] * h;  y = N2(r)
// Bound by memory: a row stays in registers between its statistics and its
// results, so every array is read once and written once.
#include "zc_norm.h"

namespace zc {
namespace moe {

// ---------------------------------------------------------------------------
// rows of any length with their 8-bit blocks
// ---------------------------------------------------------------------------

// The lanes hold their columns as the 8-bit blocks want them, the ragged last ones too.  8192 x 7165, norms on both sides and a gate:
// 220 us (528 MB), bound by loads that wait for each other; aligned rows take 96.
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
            Stat s = kNoNorm;
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
// all others
// ---------------------------------------------------------------------------

// A team takes rows in turn, the next row's loads on their way while it works on one;
// weights and gate stay in registers.  WIDE: rows start on 16 bytes and have no tail.  Q: with
// the 8-bit blocks of y (WIDE only).  8192 x 7168, norms on both sides and a gate: 82 us, 5.7 TB/s, past what
// a large copy reaches; without the loads ahead and with loads under conditions 158.
template <bool F32S, bool F32P, bool WIDE, bool Q, uint32_t TEAM, uint32_t CHUNKS>
__global__ __launch_bounds__(block_threads(TEAM), kRowsWaves) void norm_rows_kernel(NormArgs a) {
    __shared__ float parts[2][kMaxWaves][4];
    Team<TEAM> team = {parts, 0};
    const uint32_t sub = threadIdx.x % TEAM, whole = a.cols / 8 * 8, ct = whole + sub;
    const bool in_tail = !WIDE && ct < a.cols;
    uint32_t n[CHUNKS];
    Eight<F32P> w1[CHUNKS], gate[CHUNKS], w2[CHUNKS];
    const bool post = a.z && a.after.kind != ZC_NORM_NONE, pre = a.before.kind != ZC_NORM_NONE;
#pragma unroll
    for (uint32_t i = 0; i < CHUNKS; ++i) {
        const uint32_t c = (i * TEAM + sub) * 8;
        n[i] = c < whole ? 8u : 0u;
        keep_param<F32P>(post ? a.after.w : Param{}, c, n[i], 1.0f, w1[i]);
        keep_param<F32P>(a.z ? a.gate : Param{}, c, n[i], 1.0f, gate[i]);
        keep_param<F32P>(pre ? a.before.w : Param{}, c, n[i], 1.0f, w2[i]);
    }
    const float w1t = keep_tail(post ? a.after.w : Param{}, ct, in_tail, 1.0f), b1t = keep_tail(post ? a.after.b : Param{}, ct, in_tail, 0.0f);
    const float gatet = keep_tail(a.z ? a.gate : Param{}, ct, in_tail, 1.0f);
    const float w2t = keep_tail(pre ? a.before.w : Param{}, ct, in_tail, 1.0f), b2t = keep_tail(pre ? a.before.b : Param{}, ct, in_tail, 0.0f);
    const uint32_t step = gridDim.x * block_teams(TEAM);
    uint32_t row = (uint32_t)__builtin_amdgcn_readfirstlane(blockIdx.x * block_teams(TEAM) + threadIdx.x / TEAM);
    if (row >= a.rows) return;
    Eight<F32S> x[CHUNKS];
    Eight<false> z[CHUNKS];
    float xt = 0.0f, zt = 0.0f;
    const auto fetch = [&](uint32_t t, Eight<F32S> (&vx)[CHUNKS], Eight<false> (&vz)[CHUNKS], float &tx, float &tz) {
        const Row rx = row_of(a.x, t * a.x_stride, whole, F32S ? 4 : 2), rz = row_of(a.z, t * a.z_stride, whole, 2);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            load_row<false, WIDE>(rz, (i * TEAM + sub) * 8, vz[i]);
            load_row<F32S, WIDE>(rx, (i * TEAM + sub) * 8, vx[i]);
        }
        if (!WIDE) {
            tz = load_tail<false>(row_of(a.z, t * a.z_stride, a.cols, 2), ct);
            tx = load_tail<F32S>(row_of(a.x, t * a.x_stride, a.cols, F32S ? 4 : 2), ct);
        }
    };
    fetch(row, x, z, xt, zt);
    for (;;) {
        // past the last row: that one again, so that no branch stands around the loads
        const uint32_t after = row + step < a.rows ? row + step : a.rows - 1;
        Eight<F32S> nx[CHUNKS];
        Eight<false> nz[CHUNKS];
        float nxt = 0.0f, nzt = 0.0f;
        fetch(after, nx, nz, nxt, nzt);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            stay_packed(w1[i]);
            stay_packed(gate[i]);
            stay_packed(w2[i]);
        }
        float v[CHUNKS][8];
        const float share = a.row_gate ? a.scale * a.row_gate[row] : a.scale;
        Stat s = kNoNorm;
        if (post) s = row_stat<TEAM, CHUNKS>(z, n, a.after.kind, a.after.eps, a.inv_cols, team, zt, in_tail);
        float vt = 0.0f;
        if (!WIDE) vt = a.z ? fmaf(share, gatet * (post ? fmaf(normed(zt, s), w1t, b1t) : zt), xt) : xt;
        if (!WIDE) vt = in_tail ? vt : 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            stay_packed(x[i]);
            stay_packed(z[i]);
            float b[8];
            if (post && a.after.b.p) load_param(a.after.b, (i * TEAM + sub) * 8, n[i], 0.0f, b);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                float h = z[i][j];
                if (post) {
                    h = normed(h, s) * w1[i][j];
                    if (a.after.b.p) h += b[j];
                }
                v[i][j] = a.z ? fmaf(share, gate[i][j] * h, x[i][j]) : x[i][j];
            }
        }
        const Row rr = row_of(a.r, row * a.r_stride, whole, F32S ? 4 : 2);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) store_row<F32S, WIDE>(rr, (i * TEAM + sub) * 8, v[i]);
        if (!WIDE) store_tail<F32S>(row_of(a.r, row * a.r_stride, a.cols, F32S ? 4 : 2), ct, vt);
        if (pre) {
            s = row_stat<TEAM, CHUNKS>(v, n, a.before.kind, a.before.eps, a.inv_cols, team, vt, in_tail);
            if (!WIDE) vt = fmaf(normed(vt, s), w2t, b2t);
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                float b[8];
                if (a.before.b.p) load_param(a.before.b, (i * TEAM + sub) * 8, n[i], 0.0f, b);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    v[i][j] = normed(v[i][j], s) * w2[i][j];
                    if (a.before.b.p) v[i][j] += b[j];
                }
            }
        }
        const Row ry = row_of(a.y, row * a.y_stride, whole, 2);
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) store_row<false, WIDE>(ry, (i * TEAM + sub) * 8, v[i]);
        if (!WIDE) store_tail<false>(row_of(a.y, row * a.y_stride, a.cols, 2), ct, vt);
        if (Q)
#pragma unroll
            for (uint32_t i = 0; i < CHUNKS; ++i) {
                const uint32_t c = (i * TEAM + sub) * 8;
                if (c >= a.q_stride) continue;
                const u32v4 w = n[i] ? pack8(v[i]) : u32v4{0u, 0u, 0u, 0u};
                uint8_t *q = a.ys + row * a.qs_stride;
                keep8(w, a.yq + row * a.q_stride + c, q + c / kBlock, sub % kKeepLanes);
                const uint32_t pad = c / kBlock + sub % kKeepLanes;
                if (c / kBlock + 1 == a.q_stride / kBlock && sub % kKeepLanes > 0 && pad < a.qs_stride) q[pad] = 0;
            }
        row += step;
        if (row >= a.rows) return;
#pragma unroll
        for (uint32_t i = 0; i < CHUNKS; ++i) {
            x[i] = nx[i];
            z[i] = nz[i];
        }
        xt = nxt;
        zt = nzt;
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static void launch_norm(const NormArgs &a, const Shape &s, bool f32, Launches &on) {
    const uint64_t blocks = ceil_div(a.rows, block_teams(s.team));
    const dim3 grid((uint32_t)(blocks < (1u << 20) ? blocks : 1u << 20));
    with_shape(s, [&](auto team, auto chunks) {
        constexpr uint32_t T = decltype(team)::value, C = decltype(chunks)::value;
        on.launch(f32 ? norm_kernel<true, T, C> : norm_kernel<false, T, C>, grid, dim3(block_threads(T)), a);
    });
}
static void launch_rows(const NormArgs &a, const Shape &s, bool f32, bool f32p, bool wide, Launches &on) {
    // as many blocks as the device holds at once
    const uint64_t blocks = ceil_div(a.rows, block_teams(s.team)), most = 256 * (4 * kRowsWaves * kLanes / block_threads(s.team));
    const dim3 grid((uint32_t)(blocks < most ? blocks : most));
    with_shape(s, [&](auto team, auto chunks) {
        constexpr uint32_t T = decltype(team)::value, C = decltype(chunks)::value;
        const auto pick = [&](auto wide_t, auto q_t) {
            constexpr bool W = decltype(wide_t)::value, Q = decltype(q_t)::value;
            on.launch(f32 ? (f32p ? norm_rows_kernel<true, true, W, Q, T, C> : norm_rows_kernel<true, false, W, Q, T, C>)
                          : (f32p ? norm_rows_kernel<false, true, W, Q, T, C> : norm_rows_kernel<false, false, W, Q, T, C>),
                      grid, dim3(block_threads(T)), a);
        };
        if (a.yq)
            pick(std::true_type{}, std::true_type{});
        else
            wide ? pick(std::true_type{}, std::false_type{}) : pick(std::false_type{}, std::false_type{});
    });
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
    NormArgs a = common(*cfg, rows, cols, d_z != nullptr);
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
    const bool f32 = stream_type == ZC_F32;
    a.wide = cols % 8 == 0 && wide8(d_r, r_stride, f32) && wide8(d_y, y_stride);
    const Shape s = shape_of(cols);
    Launches on(stream);
    const bool wide = a.wide && wide8(d_x, x_stride, f32) && wide8(d_z, z_stride);
    if (a.yq && !wide)
        launch_norm(a, s, f32, on);
    else
        launch_rows(a, s, f32, any_float(*cfg, d_z != nullptr), wide, on);
    return on.status();
}

