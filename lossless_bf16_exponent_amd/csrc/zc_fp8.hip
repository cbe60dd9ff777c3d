// BF16 to 8-bit blocks of 128 with a power-of-two scale, along the rows, as
// 128 x 128 squares, and transposed (blocks along the tokens), MI355X / gfx950.
// All of it is bound by memory: every value is read once and written once.
#include "zc_moe_device.h"

namespace zc {
namespace moe {

constexpr uint32_t kQThreads = 256;
constexpr uint32_t kLanesPerBlock = 16;  // 8 values a lane
constexpr uint32_t kQBlocks = kQThreads / kLanesPerBlock;

struct QuantArgs {
    const uint16_t *x;
    uint8_t *q, *scales;
    uint64_t xs, qs, ss;
    uint32_t rows, cols, blocks;  // blocks of 128 in a row
};

// Eight values of a row from column c (a multiple of 8) as four pairs; values
// past the end are zeros.
template <bool WIDE>
__device__ __forceinline__ u32v4 load8(const uint16_t *row, uint32_t c, uint32_t cols) {
    return load_values<WIDE>(row + c, c < cols ? cols - c : 0u);
}

template <uint32_t TYPE>
__device__ __forceinline__ uint2 pack8(const u32v4 &w, float inv) {
    uint2 r;
    r.x = Fp8<TYPE>::pack4(bf_lo(w[0]) * inv, bf_hi(w[0]) * inv, bf_lo(w[1]) * inv, bf_hi(w[1]) * inv);
    r.y = Fp8<TYPE>::pack4(bf_lo(w[2]) * inv, bf_hi(w[2]) * inv, bf_lo(w[3]) * inv, bf_hi(w[3]) * inv);
    return r;
}

// Blocks along the rows: 16 lanes a block, one 16-byte load and one 8-byte store
// a lane.  Bound by memory: 65536 x 7168 values take 250 to 267 us, 5.3 to 5.6
// TB/s.  The bytes of a row's scales past its last block are zeroed by the lanes
// of the last block.
template <uint32_t TYPE, bool WIDE>
__global__ __launch_bounds__(kQThreads) void quantize_kernel(QuantArgs a) {
    const uint32_t sub = threadIdx.x % kLanesPerBlock;
    const uint64_t all = (uint64_t)a.rows * a.blocks;
    for (uint64_t b = (uint64_t)blockIdx.x * kQBlocks + threadIdx.x / kLanesPerBlock; b < all;
         b += (uint64_t)gridDim.x * kQBlocks) {
        const uint32_t row = (uint32_t)(b / a.blocks), kb = (uint32_t)(b % a.blocks);
        const uint32_t c = kb * kBlock + sub * 8;
        const u32v4 w = load8<WIDE>(a.x + (uint64_t)row * a.xs, c, a.cols);
        uint32_t m = 0;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) m = finite_max(m, w[i]);
        m = group_max<kLanesPerBlock>(m);
        const uint32_t byte = scale_byte(m, Fp8<TYPE>::kTop);
        *reinterpret_cast<uint2 *>(a.q + (uint64_t)row * a.qs + c) = pack8<TYPE>(w, scale_inverse(byte));
        uint8_t *s = a.scales + (uint64_t)row * a.ss;
        if (sub == 0) s[kb] = (uint8_t)byte;
        if (kb + 1 == a.blocks && sub > 0 && kb + sub < a.ss) s[kb + sub] = 0;
    }
}

// 128 x 128 squares, one block of threads each: a thread holds 64 values.  4096 x
// 7168 values take 17.4 us, 5.1 TB/s.
template <uint32_t TYPE, bool WIDE>
__global__ __launch_bounds__(kQThreads) void quantize_square_kernel(QuantArgs a) {
    __shared__ uint32_t part[kQThreads / kLanes];
    const uint32_t sub = threadIdx.x % kLanesPerBlock, r0 = threadIdx.x / kLanesPerBlock;
    const uint32_t row_blocks = (a.rows + kBlock - 1) / kBlock;
    for (uint64_t b = blockIdx.x; b < (uint64_t)row_blocks * a.blocks; b += gridDim.x) {
        const uint32_t rb = (uint32_t)(b / a.blocks), kb = (uint32_t)(b % a.blocks);
        const uint32_t c = kb * kBlock + sub * 8;
        u32v4 w[kBlock / kQBlocks];
        uint32_t m = 0;
#pragma unroll
        for (uint32_t j = 0; j < kBlock / kQBlocks; ++j) {
            const uint32_t row = rb * kBlock + j * kQBlocks + r0;
            w[j] = u32v4{0u, 0u, 0u, 0u};
            if (row < a.rows) w[j] = load8<WIDE>(a.x + (uint64_t)row * a.xs, c, a.cols);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) m = finite_max(m, w[j][i]);
        }
        m = group_max<64>(m);
        __syncthreads();
        if (lane_id() == 0) part[threadIdx.x / kLanes] = m;
        __syncthreads();
        m = max(max(part[0], part[1]), max(part[2], part[3]));
        const uint32_t byte = scale_byte(m, Fp8<TYPE>::kTop);
        const float inv = scale_inverse(byte);
#pragma unroll
        for (uint32_t j = 0; j < kBlock / kQBlocks; ++j) {
            const uint32_t row = rb * kBlock + j * kQBlocks + r0;
            if (row < a.rows)
                *reinterpret_cast<uint2 *>(a.q + (uint64_t)row * a.qs + c) = pack8<TYPE>(w[j], inv);
        }
        uint8_t *s = a.scales + (uint64_t)rb * a.ss;
        if (threadIdx.x == 0) s[kb] = (uint8_t)byte;
        if (kb + 1 == a.blocks && threadIdx.x > 0 && kb + threadIdx.x < a.ss) s[kb + threadIdx.x] = 0;
    }
}

// ---------------------------------------------------------------------------
// transposed, blocks along the tokens
// ---------------------------------------------------------------------------

struct TransArgs {
    const void *x;
    const uint8_t *xscales;
    const int32_t *offsets;
    uint8_t *q, *scales;
    uint64_t xs, xss, qs, ss;  // qs: padded rows
    uint32_t rows, cols, groups, col_tiles;
    uint64_t units;  // tiles of 128 tokens by col_tiles, at most
};

// Columns of a tile: 128 bytes of a source row.
template <uint32_t SRC>
constexpr uint32_t kTCols = SRC == ZC_BF16 ? 64 : 128;

// A tile of one block of 128 tokens and 64 (8-bit source: 128) columns: read by
// rows, whole lines, into LDS as BF16 (an 8-bit checkpoint's values fit BF16: few
// digits, and the exponents of BF16), and quantised by columns: eight lanes a
// column, 16 tokens each, which then write its 128 bytes as one line.  (Four
// threads a column in four waves, 32 bytes each: 1.3 and 1.2 times as long.)
// 8192 tokens in 8 groups take 26 us from 4096 columns of BF16 (3.9 TB/s, of 5.2
// that a copy reaches) and 42 from 7168 of 8 bits (2.8 TB/s), which are also unpacked.
// Rows past the group's end are zeros.
template <uint32_t SRC, uint32_t TYPE, bool WIDE>
__global__ __launch_bounds__(kQThreads) void quantize_t_kernel(TransArgs a) {
    constexpr uint32_t COLS = kTCols<SRC>;
    __shared__ uint16_t tile[kBlock][COLS + 2];
    const uint32_t tid = threadIdx.x;
    for (uint64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const uint32_t ct = (uint32_t)(unit % a.col_tiles), t = (uint32_t)(unit / a.col_tiles);
        const Span sp = find_tile(a.offsets, a.groups, a.rows, kBlock, [&](uint32_t) { return t; });
        if (!sp.found) return;  // the whole block: no tile after this one exists either
        const uint32_t row0 = sp.begin + sp.tile * kBlock, c0 = ct * COLS;
        const uint32_t rows = min(sp.end - row0, kBlock);
#pragma unroll
        for (uint32_t j = 0; j < kBlock / 32; ++j) {
            const uint32_t r = j * 32 + tid / 8;
            if (SRC == ZC_BF16) {
                const uint16_t *x = static_cast<const uint16_t *>(a.x);
                const uint32_t c = (tid % 8) * 8;
                u32v4 w = {0u, 0u, 0u, 0u};
                if (r < rows && c0 + c < a.cols) w = load8<WIDE>(x + (uint64_t)(row0 + r) * a.xs, c0 + c, a.cols);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(&tile[r][c + 2 * i]) = w[i];
            } else {
                typedef Fp8<SRC == ZC_BF16 ? ZC_FP8_E4M3 : SRC> F;
                const uint8_t *x = static_cast<const uint8_t *>(a.x);
                const uint32_t c = (tid % 8) * 16;
                u32v4 w = {0u, 0u, 0u, 0u};
                float s = 0.0f;
                if (r < rows) {  // xs: the row's bytes, a multiple of 128, zeros past cols
                    w = __builtin_nontemporal_load(reinterpret_cast<const u32v4 *>(x + (uint64_t)(row0 + r) * a.xs + c0 + c));
                    s = scale_value(a.xscales[(uint64_t)(row0 + r) * a.xss + c0 / kBlock]);
                }
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    *reinterpret_cast<uint32_t *>(&tile[r][c + 4 * i]) =
                        bf_pack(F::template value<0>(w[i]) * s, F::template value<1>(w[i]) * s);
                    *reinterpret_cast<uint32_t *>(&tile[r][c + 4 * i + 2]) =
                        bf_pack(F::template value<2>(w[i]) * s, F::template value<3>(w[i]) * s);
                }
            }
        }
        __syncthreads();
        const uint32_t block = sp.blocks0 + sp.tile, piece = tid % 8;
#pragma unroll
        for (uint32_t j = 0; j < COLS / 32; ++j) {
            const uint32_t c = j * 32 + tid / 8;
            uint32_t v[8], m = 0;
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                v[i] = tile[16 * piece + 2 * i][c] | ((uint32_t)tile[16 * piece + 2 * i + 1][c] << 16);
                m = finite_max(m, v[i]);
            }
            m = group_max<8>(m);
            const uint32_t byte = scale_byte(m, Fp8<TYPE>::kTop);
            const float inv = scale_inverse(byte);
            if (c0 + c < a.cols) {
                u32v4 w;
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    w[i] = Fp8<TYPE>::pack4(bf_lo(v[2 * i]) * inv, bf_hi(v[2 * i]) * inv, bf_lo(v[2 * i + 1]) * inv,
                                            bf_hi(v[2 * i + 1]) * inv);
                *reinterpret_cast<u32v4 *>(a.q + (uint64_t)(c0 + c) * a.qs + (uint64_t)block * kBlock + 16 * piece) = w;
                if (piece == 0) a.scales[(uint64_t)(c0 + c) * a.ss + block] = (uint8_t)byte;
            }
        }
        __syncthreads();
    }
}

// 128 x 128 squares transposed, scales included: one block of threads a square.
// 32 matrices of 4096 x 7168 take 506 us, 3.7 TB/s: a dword of LDS is read for
// every byte.
struct SquareArgs {
    const uint8_t *q, *s;
    uint8_t *qt, *st;
    uint32_t rows, cols, row_blocks, col_blocks;
    uint64_t batch;
};

__global__ __launch_bounds__(kQThreads) void transpose_kernel(SquareArgs a) {
    __shared__ uint32_t tile[kBlock][kBlock / 4 + 1];
    const uint64_t per = (uint64_t)a.row_blocks * a.col_blocks;
    for (uint64_t unit = blockIdx.x; unit < a.batch * per; unit += gridDim.x) {
        const uint64_t batch = unit / per;
        const uint32_t rb = (uint32_t)(unit % per / a.col_blocks), cb = (uint32_t)(unit % a.col_blocks);
        const uint64_t qs = (uint64_t)a.col_blocks * kBlock, qts = (uint64_t)a.row_blocks * kBlock;
        const uint64_t ss = (a.col_blocks + 3) / 4 * 4, sts = (a.row_blocks + 3) / 4 * 4;
        const uint8_t *q = a.q + batch * a.rows * qs;
        uint8_t *qt = a.qt + batch * a.cols * qts;
        for (uint32_t i = threadIdx.x; i < kBlock * kBlock / 4; i += kQThreads) {
            const uint32_t r = i / (kBlock / 4), c = i % (kBlock / 4), row = rb * kBlock + r;
            tile[r][c] = row < a.rows ? *reinterpret_cast<const uint32_t *>(q + (uint64_t)row * qs + cb * kBlock + 4 * c) : 0u;
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < kBlock * kBlock / 4; i += kQThreads) {
            const uint32_t c = i / (kBlock / 4), r = 4 * (i % (kBlock / 4)), col = cb * kBlock + c;
            uint32_t w = 0;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) w |= ((tile[r + j][c / 4] >> (8 * (c % 4))) & 0xFFu) << (8 * j);
            if (col < a.cols) *reinterpret_cast<uint32_t *>(qt + (uint64_t)col * qts + rb * kBlock + r) = w;
        }
        uint8_t *st = a.st + batch * a.col_blocks * sts + cb * sts;
        if (threadIdx.x == 0) st[rb] = a.s[batch * a.row_blocks * ss + rb * ss + cb];
        if (rb + 1 == a.row_blocks && threadIdx.x > 0 && rb + threadIdx.x < sts) st[rb + threadIdx.x] = 0;
        __syncthreads();
    }
}

static uint32_t grid_of(uint64_t units) { return (uint32_t)(units < (1u << 20) ? units : (1u << 20)); }

template <uint32_t TYPE>
static void launch_quantize(const QuantArgs &a, bool square, bool wide, Launches &on) {
    const dim3 block(kQThreads);
    if (square) {
        const dim3 grid(grid_of(ceil_div(a.rows, kBlock) * a.blocks));
        if (wide)
            on.launch((quantize_square_kernel<TYPE, true>), grid, block, a);
        else
            on.launch((quantize_square_kernel<TYPE, false>), grid, block, a);
    } else {
        const dim3 grid(grid_of(ceil_div((uint64_t)a.rows * a.blocks, kQBlocks)));
        if (wide)
            on.launch((quantize_kernel<TYPE, true>), grid, block, a);
        else
            on.launch((quantize_kernel<TYPE, false>), grid, block, a);
    }
}

template <uint32_t SRC, uint32_t TYPE>
static void launch_quantize_t(const TransArgs &a, bool wide, uint32_t grid, Launches &on) {
    if (wide)
        on.launch((quantize_t_kernel<SRC, TYPE, true>), dim3(grid), dim3(kQThreads), a);
    else
        on.launch((quantize_t_kernel<SRC, TYPE, false>), dim3(grid), dim3(kQThreads), a);
}

template <uint32_t SRC>
static void launch_quantize_t(uint32_t type, const TransArgs &a, bool wide, uint32_t grid, Launches &on) {
    if (type == ZC_FP8_E4M3)
        launch_quantize_t<SRC, ZC_FP8_E4M3>(a, wide, grid, on);
    else
        launch_quantize_t<SRC, ZC_FP8_E5M2>(a, wide, grid, on);
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_fp8_stride(uint64_t cols) { return cols > kMaxCols ? 0 : stride8(cols); }
extern "C" uint64_t zc_fp8_scale_stride(uint64_t cols) { return cols > kMaxRows + ZC_MOE_ROW_SLACK ? 0 : scale_stride(cols); }

extern "C" uint64_t zc_fp8_padded_rows(uint64_t rows, uint32_t groups) {
    if (rows > kMaxRows || groups == 0 || groups > ZC_MAX_EXPERTS) return 0;
    // each group adds at most 127 rows, and only a group with rows adds any
    const uint64_t used = rows < groups ? rows : groups;
    return (rows + 127 * used) / kBlock * kBlock;
}

extern "C" zc_status zc_fp8_quantize(const void *d_x, uint64_t rows, uint64_t cols, uint64_t x_stride, uint32_t type,
                                     uint32_t block_rows, void *d_q, uint8_t *d_scales, void *stream) {
    if (!is_fp8(type) || (block_rows != 1 && block_rows != kBlock) || rows > kMaxRows || cols > kMaxCols ||
        x_stride < cols || x_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!rows || !cols) return ZC_OK;
    if (!d_x || !d_q || !d_scales) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_x, 2) || !aligned(d_q, 16) || !aligned(d_scales, 4)) return ZC_ERR_MISALIGNED;
    const QuantArgs a = {static_cast<const uint16_t *>(d_x), static_cast<uint8_t *>(d_q), d_scales, x_stride,
                         stride8(cols), scale_stride(cols), (uint32_t)rows, (uint32_t)cols,
                         (uint32_t)ceil_div(cols, kBlock)};
    const bool wide = aligned(d_x, 16) && x_stride % 8 == 0 && cols % 8 == 0;
    Launches on(stream);
    if (type == ZC_FP8_E4M3)
        launch_quantize<ZC_FP8_E4M3>(a, block_rows != 1, wide, on);
    else
        launch_quantize<ZC_FP8_E5M2>(a, block_rows != 1, wide, on);
    return on.status();
}

extern "C" zc_status zc_fp8_quantize_t(const void *d_x, const uint8_t *d_x_scales, uint32_t x_type, uint64_t rows,
                                       uint64_t cols, uint64_t x_stride, uint32_t groups, const int32_t *d_offsets,
                                       uint32_t type, void *d_q, uint8_t *d_scales, uint64_t padded_rows,
                                       void *stream) {
    if (!is_fp8(type) || (x_type != ZC_BF16 && !is_fp8(x_type)) || rows > kMaxRows || cols > kMaxCols ||
        x_stride < cols || x_stride > kMaxStride || groups == 0 || groups > ZC_MAX_EXPERTS ||
        (!d_offsets && groups != 1) || padded_rows % kBlock || padded_rows > kMaxRows + ZC_MOE_ROW_SLACK ||
        (x_type != ZC_BF16 && x_stride != stride8(cols)))
        return ZC_ERR_INVALID_ARG;
    if (padded_rows < zc_fp8_padded_rows(rows, groups)) return ZC_ERR_CAPACITY;
    if (!rows || !cols) return ZC_OK;
    if (!d_x || !d_q || !d_scales || (x_type != ZC_BF16 && !d_x_scales)) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_x, x_type == ZC_BF16 ? 2 : 16) || !aligned(d_x_scales, x_type == ZC_BF16 ? 1 : 4) || !aligned(d_q, 16) || !aligned(d_scales, 4) ||
        !aligned(d_offsets, 4))
        return ZC_ERR_MISALIGNED;
    TransArgs a = {d_x, d_x_scales, d_offsets, static_cast<uint8_t *>(d_q), d_scales, x_stride, scale_stride(cols),
                   padded_rows, scale_stride(padded_rows), (uint32_t)rows, (uint32_t)cols, groups,
                   (uint32_t)ceil_div(cols, x_type == ZC_BF16 ? kTCols<ZC_BF16> : kTCols<ZC_FP8_E4M3>), 0};
    a.units = zc_fp8_padded_rows(rows, groups) / kBlock * a.col_tiles;
    const uint32_t grid = grid_of(a.units);
    const bool wide = aligned(d_x, 16) && x_stride % 8 == 0 && cols % 8 == 0;
    Launches on(stream);
    if (x_type == ZC_BF16)
        launch_quantize_t<ZC_BF16>(type, a, wide, grid, on);
    else if (x_type == ZC_FP8_E4M3)
        launch_quantize_t<ZC_FP8_E4M3>(type, a, true, grid, on);
    else
        launch_quantize_t<ZC_FP8_E5M2>(type, a, true, grid, on);
    return on.status();
}

extern "C" zc_status zc_fp8_transpose(const void *d_q, const uint8_t *d_scales, uint64_t batch, uint64_t rows,
                                      uint64_t cols, void *d_qt, uint8_t *d_scales_t, void *stream) {
    if (rows > kMaxCols || cols > kMaxCols || batch > ZC_MAX_EXPERTS) return ZC_ERR_INVALID_ARG;
    if (!batch || !rows || !cols) return ZC_OK;
    if (!d_q || !d_scales || !d_qt || !d_scales_t) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_q, 16) || !aligned(d_scales, 4) || !aligned(d_qt, 16) || !aligned(d_scales_t, 4))
        return ZC_ERR_MISALIGNED;
    const SquareArgs a = {static_cast<const uint8_t *>(d_q), d_scales, static_cast<uint8_t *>(d_qt), d_scales_t,
                          (uint32_t)rows, (uint32_t)cols, (uint32_t)ceil_div(rows, kBlock),
                          (uint32_t)ceil_div(cols, kBlock), batch};
    Launches on(stream);
    on.launch(transpose_kernel, dim3(grid_of(batch * a.row_blocks * a.col_blocks)), dim3(kQThreads), a);
    return on.status();
}
