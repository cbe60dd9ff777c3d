// Grouped products of 8-bit floating point with a power-of-two scale for each
// block of 128, MI355X / gfx950:
//   forward   out[r, c] = sum over k of A[r, k] B_g[c, k], rows r of group g
//   gradient  out[g, i, j] = sum over the rows r of group g of A[i, r] B[j, r]
// The scaled matrix instructions apply the scales: 2^(a - 127) 2^(b - 127) for
// every lane's 32 values, in the 32-bit sum, at no cost of their own.
#include "zc_moe_device.h"

namespace zc {
namespace moe {

typedef int i32v8 __attribute__((ext_vector_type(8)));
typedef float f32v16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));

struct MatArgs {
    const uint8_t *a, *as, *b, *bs;
    const int32_t *offsets;
    void *out;
    uint64_t lda, ldas, ldb, ldbs;       // bytes of a row
    uint64_t b_group, bs_group;          // bytes of a group's matrix and scales (forward)
    uint64_t ldo, out_group;             // elements
    uint32_t m, n, rows, blocks, groups;  // blocks of 128 along the contraction (forward); rows split into groups
    uint32_t b_shift;                    // rows of B that share a row of scales, as a shift
};

constexpr uint32_t kMThreads = 256;
constexpr uint32_t kSimpleTile = 128;

// sum_mode FULL: 32 8-bit values of a lane, times their scale, as BF16: exact,
// since a BF16 has the exponents of a float and more digits than any 8-bit type.
// (The conversion takes its scale from a float's exponent.)
template <int F>
__device__ __forceinline__ void widen(const i32v8 &w, uint32_t scale, bf16v8 (&out)[4]) {
    const float s = __uint_as_float(scale << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16v2 lo, hi;
            if (F == 0) {
                lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[2 * i + j], s, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[2 * i + j], s, true);
            } else {
                lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w[2 * i + j], s, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w[2 * i + j], s, true);
            }
            out[i][4 * j] = lo[0];
            out[i][4 * j + 1] = lo[1];
            out[i][4 * j + 2] = hi[0];
            out[i][4 * j + 3] = hi[1];
        }
}

template <int FA, int FB>
__device__ __forceinline__ f32v16 mfma(const i32v8 &a, const i32v8 &b, const f32v16 &c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, FA, FB, 0, (int)sa, 0, (int)sb);
}

// 128 x 128 tile, four waves of 64 x 64, one block of 128 along the contraction
// at a time through LDS.
template <bool WGRAD, int FA, int FB, bool OUT_BF16, bool FULL>
__global__ __launch_bounds__(kMThreads) void simple_kernel(MatArgs p) {
    __shared__ alignas(16) uint8_t sa[kSimpleTile][kBlock + 16];
    __shared__ alignas(16) uint8_t sb[kSimpleTile][kBlock + 16];
    const uint32_t tid = threadIdx.x, lane = lane_id(), wave = tid / kLanes;
    const uint32_t wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    const uint32_t ntiles = (p.n + kSimpleTile - 1) / kSimpleTile;
    const uint32_t nt = blockIdx.x % ntiles, mt = blockIdx.x / ntiles;
    Span sp;
    uint32_t m0, m1, kb0, kb1;
    const uint8_t *b = p.b, *bs = p.bs;
    uint64_t out0 = 0;
    if (WGRAD) {
        const uint32_t mtiles = (p.m + kSimpleTile - 1) / kSimpleTile;
        sp = find_group(p.offsets, p.groups, p.rows, mt / mtiles);
        m0 = (mt % mtiles) * kSimpleTile;
        m1 = p.m;
        kb0 = sp.blocks0;
        kb1 = kb0 + (sp.end - sp.begin + kBlock - 1) / kBlock;
        out0 = (uint64_t)sp.group * p.out_group;
    } else {
        sp = find_tile(p.offsets, p.groups, p.rows, kSimpleTile, mt);
        if (!sp.found) return;
        m0 = sp.begin + sp.tile * kSimpleTile;
        m1 = sp.end;
        kb0 = 0;
        kb1 = p.blocks;
        b += sp.group * p.b_group;
        bs += sp.group * p.bs_group;
    }
    const uint32_t n0 = nt * kSimpleTile;
    f32v16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t r = i * 32 + tid / 8, c = (tid % 8) * 16;
            const uint32_t ra = min(m0 + r, m1 - 1), rb = min(n0 + r, p.n - 1);
            *reinterpret_cast<u32v4 *>(&sa[r][c]) =
                *reinterpret_cast<const u32v4 *>(p.a + (uint64_t)ra * p.lda + (uint64_t)kb * kBlock + c);
            *reinterpret_cast<u32v4 *>(&sb[r][c]) =
                *reinterpret_cast<const u32v4 *>(b + (uint64_t)rb * p.ldb + (uint64_t)kb * kBlock + c);
        }
        __syncthreads();
        uint32_t ea[2], eb[2];
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            const uint32_t ra = min(m0 + wm + 32 * i + lane % 32, m1 - 1);
            const uint32_t rb = min(n0 + wn + 32 * i + lane % 32, p.n - 1);
            ea[i] = p.as[(uint64_t)ra * p.ldas + kb];
            eb[i] = bs[(uint64_t)(rb >> p.b_shift) * p.ldbs + kb];
        }
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {
            i32v8 fa[2], fb[2];
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                fa[i] = *reinterpret_cast<const i32v8 *>(&sa[wm + 32 * i + lane % 32][half * 64 + (lane / 32) * 32]);
                fb[i] = *reinterpret_cast<const i32v8 *>(&sb[wn + 32 * i + lane % 32][half * 64 + (lane / 32) * 32]);
            }
            // B in the place of the left matrix: a lane then holds four consecutive columns of one row
            if (FULL) {
                bf16v8 wa[2][4], wb[2][4];
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    widen<FA>(fa[i], ea[i], wa[i]);
                    widen<FB>(fb[i], eb[i], wb[i]);
                }
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
                        for (uint32_t q = 0; q < 4; ++q)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j][q], wa[i][q], acc[i][j], 0, 0, 0);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < 2; ++j) acc[i][j] = mfma<FB, FA>(fb[j], fa[i], acc[i][j], eb[j], ea[i]);
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
            for (uint32_t e = 0; e < 16; ++e) {
                const uint32_t r = m0 + wm + 32 * i + lane % 32;
                const uint32_t c = n0 + wn + 32 * j + 8 * (e / 4) + 4 * (lane / 32) + e % 4;
                if (r < m1 && c < p.n) {
                    const uint64_t o = out0 + (uint64_t)r * p.ldo + c;
                    if (OUT_BF16)
                        static_cast<uint16_t *>(p.out)[o] = bf_round(acc[i][j][e]);
                    else
                        static_cast<float *>(p.out)[o] = acc[i][j][e];
                }
            }
}

template <bool WGRAD, int FA, int FB, bool FULL>
static void launch_out(const MatArgs &p, bool bf16, uint32_t grid, hipStream_t st) {
    if (bf16)
        hipLaunchKernelGGL((simple_kernel<WGRAD, FA, FB, true, FULL>), dim3(grid), dim3(kMThreads), 0, st, p);
    else
        hipLaunchKernelGGL((simple_kernel<WGRAD, FA, FB, false, FULL>), dim3(grid), dim3(kMThreads), 0, st, p);
}

template <bool WGRAD, int FA, int FB>
static void launch_sum(const MatArgs &p, bool bf16, bool full, uint32_t grid, hipStream_t st) {
    if (full)
        launch_out<WGRAD, FA, FB, true>(p, bf16, grid, st);
    else
        launch_out<WGRAD, FA, FB, false>(p, bf16, grid, st);
}

template <bool WGRAD>
static zc_status launch(const MatArgs &p, uint32_t ta, uint32_t tb, bool bf16, bool full, hipStream_t st) {
    const uint64_t ntiles = ceil_div(p.n, kSimpleTile);
    const uint64_t mtiles = WGRAD ? ceil_div(p.m, kSimpleTile) * p.groups
                                  : p.rows / kSimpleTile + (p.rows < p.groups ? p.rows : p.groups);
    if (ntiles * mtiles > 0xFFFFFFu) return ZC_ERR_INVALID_ARG;
    const uint32_t grid = (uint32_t)(ntiles * mtiles);
    const int fa = ta == ZC_FP8_E5M2, fb = tb == ZC_FP8_E5M2;
    if (!fa && !fb) launch_sum<WGRAD, 0, 0>(p, bf16, full, grid, st);
    if (!fa && fb) launch_sum<WGRAD, 0, 1>(p, bf16, full, grid, st);
    if (fa && !fb) launch_sum<WGRAD, 1, 0>(p, bf16, full, grid, st);
    if (fa && fb) launch_sum<WGRAD, 1, 1>(p, bf16, full, grid, st);
    return launched();
}

static bool types_ok(uint32_t ta, uint32_t tb, uint32_t to, uint32_t sum) {
    return is_fp8(ta) && is_fp8(tb) && (to == ZC_F32 || to == ZC_BF16) && sum <= ZC_FP8_SUM_FULL;
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_fp8_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, uint32_t groups) {
    (void)m;
    (void)n;
    (void)k;
    (void)groups;
    return 0;
}

extern "C" zc_status zc_fp8_matmul(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t m,
                                   const void *d_b, const uint8_t *d_b_scales, uint32_t b_type, uint64_t n,
                                   uint64_t k, uint32_t groups, const int32_t *d_offsets, void *d_out,
                                   uint32_t out_type, uint64_t out_stride, uint32_t sum_mode,
                                   void *d_workspace, uint64_t workspace_bytes, void *stream) {
    (void)workspace_bytes;
    if (!types_ok(a_type, b_type, out_type, sum_mode) || m > kMaxRows || n > kMaxCols || k > kMaxCols || groups == 0 ||
        groups > ZC_MAX_EXPERTS || (!d_offsets && groups != 1) || out_stride < n || out_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!m || !n) return ZC_OK;
    if (!d_out || (k && (!d_a || !d_a_scales || !d_b || !d_b_scales))) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_a, 16) || !aligned(d_a_scales, 16) || !aligned(d_b, 16) || !aligned(d_b_scales, 16) ||
        !aligned(d_offsets, 4) || !aligned(d_out, out_type == ZC_F32 ? 4 : 2) || !aligned(d_workspace, 16))
        return ZC_ERR_MISALIGNED;
    MatArgs p = {};
    p.a = static_cast<const uint8_t *>(d_a);
    p.as = d_a_scales;
    p.b = static_cast<const uint8_t *>(d_b);
    p.bs = d_b_scales;
    p.offsets = d_offsets;
    p.out = d_out;
    p.lda = p.ldb = stride8(k);
    p.ldas = p.ldbs = scale_stride(k);
    p.b_group = n * p.ldb;
    p.bs_group = ceil_div(n, kBlock) * p.ldbs;
    p.ldo = out_stride;
    p.m = p.rows = (uint32_t)m;
    p.n = (uint32_t)n;
    p.blocks = (uint32_t)ceil_div(k, kBlock);
    p.groups = groups;
    p.b_shift = 7;
    return launch<false>(p, a_type, b_type, out_type == ZC_BF16, sum_mode == ZC_FP8_SUM_FULL,
                         static_cast<hipStream_t>(stream));
}

extern "C" zc_status zc_fp8_matmul_wgrad(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t n,
                                         const void *d_b, const uint8_t *d_b_scales, uint32_t b_type, uint64_t k,
                                         uint64_t padded_rows, uint64_t rows, uint32_t groups,
                                         const int32_t *d_offsets, void *d_out, uint32_t out_type,
                                         uint32_t sum_mode, void *stream) {
    if (!types_ok(a_type, b_type, out_type, sum_mode) || rows > kMaxRows || n > kMaxCols || k > kMaxCols || groups == 0 ||
        groups > ZC_MAX_EXPERTS || (!d_offsets && groups != 1) || padded_rows % kBlock ||
        padded_rows > kMaxRows + ZC_MOE_ROW_SLACK)
        return ZC_ERR_INVALID_ARG;
    if (padded_rows < zc_fp8_padded_rows(rows, groups)) return ZC_ERR_CAPACITY;
    if (!n || !k) return ZC_OK;
    if (!d_out || (rows && (!d_a || !d_a_scales || !d_b || !d_b_scales))) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_a, 16) || !aligned(d_a_scales, 16) || !aligned(d_b, 16) || !aligned(d_b_scales, 16) ||
        !aligned(d_offsets, 4) || !aligned(d_out, out_type == ZC_F32 ? 4 : 2))
        return ZC_ERR_MISALIGNED;
    MatArgs p = {};
    p.a = static_cast<const uint8_t *>(d_a);
    p.as = d_a_scales;
    p.b = static_cast<const uint8_t *>(d_b);
    p.bs = d_b_scales;
    p.offsets = d_offsets;
    p.out = d_out;
    p.lda = p.ldb = padded_rows;
    p.ldas = p.ldbs = scale_stride(padded_rows);
    p.ldo = k;
    p.out_group = n * k;
    p.m = (uint32_t)n;
    p.n = (uint32_t)k;
    p.rows = (uint32_t)rows;
    p.groups = groups;
    p.b_shift = 0;
    return launch<true>(p, a_type, b_type, out_type == ZC_BF16, sum_mode == ZC_FP8_SUM_FULL,
                         static_cast<hipStream_t>(stream));
}
