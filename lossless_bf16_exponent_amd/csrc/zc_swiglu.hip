// Gated activation with an 8-bit checkpoint of its input, and its gradient from
// that checkpoint, MI355X / gfx950.  Bound by memory.
#include "zc_moe_device.h"

namespace zc {
namespace moe {

constexpr uint32_t kGThreads = 256;
constexpr uint32_t kGLanes = 16;  // lanes of a block of 128 columns, 8 values each
constexpr uint32_t kGBlocks = kGThreads / kGLanes;

struct GateArgs {
    const uint16_t *gu;
    const uint16_t *dh;
    uint16_t *h;      // forward
    uint16_t *dgu;    // backward
    uint8_t *hq, *hs, *kept, *ks;
    uint64_t stride, h_stride;  // of gu or dgu; of h or dh
    uint64_t q_stride, hss, kss;
    uint32_t rows, cols, blocks;
};

// sigmoid(g) = s * unit and 1 - sigmoid(g) from t = e^-|g| <= 1: neither overflows,
// nor loses digits to a subtraction.  The hardware exponential and reciprocal (1
// ulp of 32 bits) are far finer than the BF16 results.  Below e^-87 t has few
// digits in 32 bits or none, and g t times a large value is a normal number
// again.  A wave that holds a gate past 80 (FAR) therefore takes t 2^64 higher
// there, and a sigmoid that is t keeps that factor until the products are made
// (unit; 1 else); 1 + t is then 1, and g t nothing beside 1.  NaN stays NaN.
constexpr float kFar = 80.0f;
struct Sigmoid {
    float s, rest, unit;
};
template <bool FAR>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
    const float a = fabsf(g);
    const bool far = FAR && a > kFar;
    const float t = __builtin_amdgcn_exp2f(FAR ? fmaf(a, -1.44269504f, far ? 64.0f : 0.0f) : a * -1.44269504f);
    const float r = __builtin_amdgcn_rcpf(1.0f + (far ? 0.0f : t)), tr = t * r;
    Sigmoid o;
    o.s = g >= 0.0f ? r : tr;
    o.rest = g >= 0.0f ? (far ? 0.0f : tr) : r;
    o.unit = far && g < 0.0f ? 0x1p-64f : 1.0f;
    return o;
}
// Whether a lane of the wave holds a gate past kFar.
__device__ __forceinline__ bool any_far(const float (&g)[8]) {
    float m = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) m = fmaxf(m, fabsf(g[i]));
    return __ballot(m > kFar) != 0;
}
template <bool FAR>
__device__ __forceinline__ u32v4 gated8(const float (&g)[8], const u32v4 &u) {
    u32v4 h;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const Sigmoid a = sigmoid<FAR>(g[2 * i]), b = sigmoid<FAR>(g[2 * i + 1]);
        h[i] = bf_pack(g[2 * i] * a.s * bf_lo(u[i]) * a.unit, g[2 * i + 1] * b.s * bf_hi(u[i]) * b.unit);
    }
    return h;
}
template <bool FAR>
__device__ __forceinline__ void gradients8(const float (&g)[8], const float (&u)[8], const u32v4 &dh, float (&dg)[8],
                                           float (&du)[8]) {
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
        const float d = (i & 1) ? bf_hi(dh[i / 2]) : bf_lo(dh[i / 2]);
        const Sigmoid o = sigmoid<FAR>(g[i]);
        dg[i] = d * u[i] * (o.s * fmaf(g[i], o.rest, 1.0f)) * o.unit;
        du[i] = d * (g[i] * o.s) * o.unit;
    }
}

// The 8 values' 8-bit form under the block's scale (16 lanes a block); lane 0
// writes the scale.
__device__ __forceinline__ void keep8(const u32v4 &w, uint8_t *q, uint8_t *s, uint32_t sub) {
    uint32_t m = 0;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) m = finite_max(m, w[i]);
    m = group_max<kGLanes>(m);
    typedef Fp8<ZC_FP8_E4M3> F;
    const uint32_t byte = scale_byte(m, F::kTop);
    const float inv = scale_inverse(byte);
    uint2 r;
    r.x = F::pack4(bf_lo(w[0]) * inv, bf_hi(w[0]) * inv, bf_lo(w[1]) * inv, bf_hi(w[1]) * inv);
    r.y = F::pack4(bf_lo(w[2]) * inv, bf_hi(w[2]) * inv, bf_lo(w[3]) * inv, bf_hi(w[3]) * inv);
    *reinterpret_cast<uint2 *>(q) = r;
    if (sub == 0) *s = (uint8_t)byte;
}

// Everything is read once and written once: non-temporal accesses (65536 x 2048
// forward 198 -> 181 us, backward 197 -> 178 us).  Now 181 and 171 us, 5.9 and 6.3
// TB/s, past what a large copy reaches.  16 lanes of eight values a block of 128.
template <bool WIDE>
__global__ __launch_bounds__(kGThreads) void swiglu_kernel(GateArgs a) {
    const uint32_t sub = threadIdx.x % kGLanes;
    const uint64_t all = (uint64_t)a.rows * a.blocks;
    for (uint64_t b = (uint64_t)blockIdx.x * kGBlocks + threadIdx.x / kGLanes; b < all;
         b += (uint64_t)gridDim.x * kGBlocks) {
        const uint32_t row = (uint32_t)(b / a.blocks), kb = (uint32_t)(b % a.blocks);
        const uint32_t c = kb * kBlock + sub * 8, n = c < a.cols ? a.cols - c : 0u;
        const uint16_t *src = a.gu + (uint64_t)row * a.stride + c;
        const u32v4 g = load_values<WIDE>(src, n), u = load_values<WIDE>(src + a.cols, n);
        if (a.kept) {
            uint8_t *q = a.kept + (uint64_t)row * 2 * a.q_stride + c, *s = a.ks + (uint64_t)row * a.kss;
            keep8(g, q, s + kb, sub);
            keep8(u, q + a.q_stride, s + a.blocks + kb, sub);
            if (kb + 1 == a.blocks && 2 * a.blocks + sub < a.kss) s[2 * a.blocks + sub] = 0;
        }
        if (!a.h && !a.hq) continue;
        float gf[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) gf[i] = (i & 1) ? bf_hi(g[i / 2]) : bf_lo(g[i / 2]);
        const u32v4 h = any_far(gf) ? gated8<true>(gf, u) : gated8<false>(gf, u);
        if (a.h) store_values<WIDE>(a.h + (uint64_t)row * a.h_stride + c, h, n);
        if (a.hq) {
            uint8_t *s = a.hs + (uint64_t)row * a.hss;
            keep8(h, a.hq + (uint64_t)row * a.q_stride + c, s + kb, sub);
            if (kb + 1 == a.blocks && sub > 0 && kb + sub < a.hss) s[kb + sub] = 0;
        }
    }
}

template <bool WIDE>
__global__ __launch_bounds__(kGThreads) void swiglu_backward_kernel(GateArgs a) {
    const uint32_t sub = threadIdx.x % kGLanes;
    const uint64_t all = (uint64_t)a.rows * a.blocks;
    typedef Fp8<ZC_FP8_E4M3> F;
    for (uint64_t b = (uint64_t)blockIdx.x * kGBlocks + threadIdx.x / kGLanes; b < all;
         b += (uint64_t)gridDim.x * kGBlocks) {
        const uint32_t row = (uint32_t)(b / a.blocks), kb = (uint32_t)(b % a.blocks);
        const uint32_t c = kb * kBlock + sub * 8, n = c < a.cols ? a.cols - c : 0u;
        const uint8_t *q = a.kept + (uint64_t)row * 2 * a.q_stride + c, *s = a.ks + (uint64_t)row * a.kss;
        const u32v2 gq = *reinterpret_cast<const u32v2 *>(q);
        const u32v2 uq = *reinterpret_cast<const u32v2 *>(q + a.q_stride);
        const float gs = scale_value(s[kb]), us = scale_value(s[a.blocks + kb]);
        const u32v4 dh = load_values<WIDE>(a.dh + (uint64_t)row * a.h_stride + c, n);
        float g[8], u[8], dg[8], du[8];
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            g[4 * i] = F::value<0>(gq[i]);
            g[4 * i + 1] = F::value<1>(gq[i]);
            g[4 * i + 2] = F::value<2>(gq[i]);
            g[4 * i + 3] = F::value<3>(gq[i]);
            u[4 * i] = F::value<0>(uq[i]);
            u[4 * i + 1] = F::value<1>(uq[i]);
            u[4 * i + 2] = F::value<2>(uq[i]);
            u[4 * i + 3] = F::value<3>(uq[i]);
        }
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            g[i] *= gs;
            u[i] *= us;
        }
        if (any_far(g))
            gradients8<true>(g, u, dh, dg, du);
        else
            gradients8<false>(g, u, dh, dg, du);
        u32v4 wg, wu;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            wg[i] = bf_pack(dg[2 * i], dg[2 * i + 1]);
            wu[i] = bf_pack(du[2 * i], du[2 * i + 1]);
        }
        uint16_t *dst = a.dgu + (uint64_t)row * a.stride + c;
        store_values<WIDE>(dst, wg, n);
        store_values<WIDE>(dst + a.cols, wu, n);
    }
}

static uint32_t gate_grid(const GateArgs &a) {
    const uint64_t units = ceil_div((uint64_t)a.rows * a.blocks, kGBlocks);
    return (uint32_t)(units < (1u << 20) ? units : (1u << 20));
}
static bool wide8(const void *p, uint64_t stride) { return aligned(p, 16) && stride % 8 == 0; }

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" zc_status zc_swiglu(const void *d_gate_up, uint64_t rows, uint64_t cols, uint64_t stride, void *d_h,
                               uint64_t h_stride, void *d_hq, uint8_t *d_hq_scales, void *d_kept,
                               uint8_t *d_kept_scales, void *stream) {
    if (rows > kMaxRows || cols > kMaxCols / 2 || stride < 2 * cols || stride > kMaxStride ||
        (d_h && (h_stride < cols || h_stride > kMaxStride)) || !d_hq != !d_hq_scales || !d_kept != !d_kept_scales)
        return ZC_ERR_INVALID_ARG;
    if (!rows || !cols || (!d_h && !d_hq && !d_kept)) return ZC_OK;
    if (!d_gate_up) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_gate_up, 2) || !aligned(d_h, 2) || !aligned(d_hq, 16) || !aligned(d_hq_scales, 4) ||
        !aligned(d_kept, 16) || !aligned(d_kept_scales, 4))
        return ZC_ERR_MISALIGNED;
    GateArgs a = {};
    a.gu = static_cast<const uint16_t *>(d_gate_up);
    a.h = static_cast<uint16_t *>(d_h);
    a.hq = static_cast<uint8_t *>(d_hq);
    a.hs = d_hq_scales;
    a.kept = static_cast<uint8_t *>(d_kept);
    a.ks = d_kept_scales;
    a.stride = stride;
    a.h_stride = h_stride;
    a.q_stride = stride8(cols);
    a.hss = scale_stride(cols);
    a.kss = scale_stride(2 * a.q_stride);
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.blocks = (uint32_t)ceil_div(cols, kBlock);
    Launches on(stream);
    if (cols % 8 == 0 && wide8(d_gate_up, stride) && (!d_h || wide8(d_h, h_stride)))
        on.launch(swiglu_kernel<true>, dim3(gate_grid(a)), dim3(kGThreads), a);
    else
        on.launch(swiglu_kernel<false>, dim3(gate_grid(a)), dim3(kGThreads), a);
    return on.status();
}

extern "C" zc_status zc_swiglu_backward(const void *d_kept, const uint8_t *d_kept_scales, uint64_t rows,
                                        uint64_t cols, const void *d_dh, uint64_t dh_stride, void *d_dgate_up,
                                        uint64_t stride, void *stream) {
    if (rows > kMaxRows || cols > kMaxCols / 2 || stride < 2 * cols || stride > kMaxStride || dh_stride < cols ||
        dh_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!rows || !cols) return ZC_OK;
    if (!d_kept || !d_kept_scales || !d_dh || !d_dgate_up) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_kept, 16) || !aligned(d_kept_scales, 4) || !aligned(d_dh, 2) || !aligned(d_dgate_up, 2))
        return ZC_ERR_MISALIGNED;
    GateArgs a = {};
    a.kept = static_cast<uint8_t *>(const_cast<void *>(d_kept));
    a.ks = const_cast<uint8_t *>(d_kept_scales);
    a.dh = static_cast<const uint16_t *>(d_dh);
    a.dgu = static_cast<uint16_t *>(d_dgate_up);
    a.stride = stride;
    a.h_stride = dh_stride;
    a.q_stride = stride8(cols);
    a.kss = scale_stride(2 * a.q_stride);
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.blocks = (uint32_t)ceil_div(cols, kBlock);
    Launches on(stream);
    if (cols % 8 == 0 && wide8(d_dh, dh_stride) && wide8(d_dgate_up, stride))
        on.launch(swiglu_backward_kernel<true>, dim3(gate_grid(a)), dim3(kGThreads), a);
    else
        on.launch(swiglu_backward_kernel<false>, dim3(gate_grid(a)), dim3(kGThreads), a);
    return on.status();
}
