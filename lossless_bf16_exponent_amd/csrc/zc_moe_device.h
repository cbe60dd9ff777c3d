// Device and host helpers shared by the mixture-of-experts kernels (gfx950):
// BF16 and 8-bit conversions, the block scale, wave-wide reductions, and the
// lookup of a tile's expert in offsets that live on the device.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "zc_moe.h"

namespace zc {
namespace moe {

constexpr uint32_t kLanes = 64;
constexpr uint32_t kBlock = ZC_FP8_BLOCK;

typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4a2 __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any BF16 value

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return a / b + (a % b != 0); }
inline uint64_t stride8(uint64_t cols) { return ceil_div(cols, kBlock) * kBlock; }
inline uint64_t scale_stride(uint64_t cols) { return ceil_div(ceil_div(cols, kBlock), 4) * 4; }
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool is_fp8(uint32_t t) { return t == ZC_FP8_E4M3 || t == ZC_FP8_E5M2; }

// Row counts fit 31 bits with room to round up; row lengths are bounded so
// that a row's bytes fit 32 bits.
constexpr uint64_t kMaxRows = 0x7FFFFFFFull - ZC_MOE_ROW_SLACK;
constexpr uint64_t kMaxCols = 1ull << 28;
constexpr uint64_t kMaxStride = 1ull << 40;

// The launches of one call on its stream, up to the first that fails, once its
// arguments are accepted.  What another call left pending in the HIP runtime is
// dropped, and the status is that which the launches themselves return: a question
// after them would cost a call 0.1 us more.
class Launches {
  public:
    explicit Launches(void *stream) : stream_(static_cast<hipStream_t>(stream)) { (void)hipGetLastError(); }
    template <typename... P>
    void launch(void (*kernel)(P...), dim3 grid, dim3 block, std::common_type_t<P>... args) {
        void *at[] = {&args...};
        if (error_ == hipSuccess)
            error_ = hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, at, 0, stream_);
    }
    zc_status status() const {
        if (error_ == hipSuccess) return ZC_OK;
        (void)hipGetLastError();  // it is reported here and not again
        return ZC_ERR_HIP;
    }

  private:
    hipStream_t stream_;
    hipError_t error_ = hipSuccess;
};

// ---------------------------------------------------------------------------
// numbers
// ---------------------------------------------------------------------------

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf_one(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// Two floats as a pair of BF16, to nearest with ties to even (the conversion
// instruction of gfx950; NaN stays NaN).
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    const b2 r = __builtin_convertvector(v, b2);
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint16_t bf_round(float a) { return (uint16_t)bf_pack(a, 0.0f); }

// The scale byte of a block from the bits of its largest finite BF16 magnitude
// (15 bits).  The largest value of both 8-bit types is 1.75 times a power of
// two (2^8, 2^15), so the exponent of the scale is the magnitude's own minus 8
// (or 15), plus one when its mantissa is above 1.75 (96 of 128): adding 31
// carries into the exponent exactly then.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax15, uint32_t top) {
    const uint32_t e = (amax15 + 31u) >> 7;
    return e > top ? e - top : 0u;
}
// 1 / scale = 2^(127 - byte), byte 0..247.
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// scale = 2^(byte - 127) (byte 0 is a subnormal number).
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

template <uint32_t TYPE>
struct Fp8;
template <>
struct Fp8<ZC_FP8_E4M3> {
    static constexpr uint32_t kTop = 8;
    static constexpr int kFormat = 0;  // the matrix instructions' code of the type
    __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    template <int I>
    __device__ __forceinline__ static float value(uint32_t w) {
        return __builtin_amdgcn_cvt_f32_fp8((int)w, I);
    }
};
template <>
struct Fp8<ZC_FP8_E5M2> {
    static constexpr uint32_t kTop = 15;
    static constexpr int kFormat = 1;
    __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
        int w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    template <int I>
    __device__ __forceinline__ static float value(uint32_t w) {
        return __builtin_amdgcn_cvt_f32_bf8((int)w, I);
    }
};

// Larger magnitude (15 bits) of a BF16 pair, infinities and NaN left out.
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t pair) {
    const uint32_t a = pair & 0x7FFFu, b = (pair >> 16) & 0x7FFFu;
    m = max(m, a < 0x7F80u ? a : 0u);
    return max(m, b < 0x7F80u ? b : 0u);
}

// Eight BF16 values as four pairs, of which the first n exist (the others read
// as zeros and are not written).  WIDE: the array starts on 16 bytes and n is 0 or
// 8 or more.  Else a row may start at any value: the memory unit takes 16 bytes
// at any address, and only a row's last values go one by one.
template <bool WIDE>
__device__ __forceinline__ u32v4 load_values(const uint16_t *p, uint32_t n) {
    u32v4 w = {0u, 0u, 0u, 0u};
    if (n >= 8) {
        if (WIDE)
            w = __builtin_nontemporal_load(reinterpret_cast<const u32v4 *>(p));
        else
            w = __builtin_nontemporal_load(reinterpret_cast<const u32v4a2 *>(p));
    } else if (!WIDE && n) {
#pragma unroll
        for (uint32_t i = 0; i < 7; ++i) w[i / 2] |= (i < n ? (uint32_t)p[i] : 0u) << (16 * (i & 1));
    }
    return w;
}
template <bool WIDE>
__device__ __forceinline__ void store_values(uint16_t *p, const u32v4 &w, uint32_t n) {
    if (n >= 8) {
        if (WIDE)
            __builtin_nontemporal_store(w, reinterpret_cast<u32v4 *>(p));
        else
            *reinterpret_cast<u32v4a2 *>(p) = w;
    } else if (!WIDE && n) {
#pragma unroll
        for (uint32_t i = 0; i < 7; ++i)
            if (i < n) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// ---------------------------------------------------------------------------
// waves
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t lane_id() { return threadIdx.x & (kLanes - 1); }

// Maximum / sum over the 2^k lanes of an aligned group of WIDTH lanes.
template <int WIDTH>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
    for (int s = 1; s < WIDTH; s <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, s));
    return v;
}
template <int WIDTH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int s = 1; s < WIDTH; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// Sum over the wave, in an order of its own that does not change.
__device__ __forceinline__ float wave_sum_f(float v) {
#define ZC_MOE_ADD(ctrl, rows) \
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xF, false))
    ZC_MOE_ADD(0x111, 0xF);  // shifts of 1, 2, 4, 8 lanes inside the rows of 16; then a row's last lane into the rows after it
    ZC_MOE_ADD(0x112, 0xF);
    ZC_MOE_ADD(0x114, 0xF);
    ZC_MOE_ADD(0x118, 0xF);
    ZC_MOE_ADD(0x142, 0xA);
    ZC_MOE_ADD(0x143, 0xC);
#undef ZC_MOE_ADD
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Inclusive scans over the wave in DPP moves: shifts of 1, 2, 4 and 8 lanes
// inside the rows of 16, then the last lane of a row into the rows after it.  A
// lane without a source keeps 0.
#define ZC_MOE_SCAN(name, combine)                                                                            \
    __device__ __forceinline__ uint32_t name(uint32_t v) {                                                    \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));             \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));             \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));             \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));             \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));             \
        v = combine(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));             \
        return v;                                                                                             \
    }
__device__ __forceinline__ uint32_t add_u32(uint32_t a, uint32_t b) { return a + b; }
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
ZC_MOE_SCAN(scan_sum, add_u32)
ZC_MOE_SCAN(scan_max, max_u32)
#undef ZC_MOE_SCAN

// ---------------------------------------------------------------------------
// groups of rows
// ---------------------------------------------------------------------------

struct Span {
    uint32_t group;
    uint32_t begin, end;  // the group's rows
    uint32_t tile;        // index of the tile within the group
    uint32_t blocks0;     // blocks of 128 rows of the groups before it, each group rounded up
    bool found;
};

__device__ __forceinline__ uint32_t clamp_row(int32_t v, uint32_t rows) {
    return v < 0 ? 0u : min((uint32_t)v, rows);
}

// 64 groups of a list, one a lane: rows, tiles and blocks, and their running
// sums.  The offsets are clamped to 0..rows and to ascending order (a running
// maximum, `high` so far), so that no value of them leads outside the arrays.
struct Groups {
    uint32_t begin, end, tiles, blocks, tile_sum, block_sum;
    bool in;
};
__device__ __forceinline__ Groups load_groups(const int32_t *offsets, uint32_t groups, uint32_t rows,
                                              uint32_t tile_rows, uint32_t g0, uint32_t high) {
    Groups r;
    const uint32_t g = g0 + lane_id();
    r.in = g < groups;
    const uint32_t o0 = r.in ? clamp_row(offsets[g], rows) : 0u;
    const uint32_t o1 = r.in ? clamp_row(offsets[g + 1], rows) : 0u;
    r.begin = max(scan_max(o0), high);
    r.end = r.in ? max(r.begin, o1) : r.begin;
    const uint32_t n = r.end - r.begin;
    r.tiles = (n + tile_rows - 1) / tile_rows;
    r.blocks = (n + kBlock - 1) / kBlock;
    r.tile_sum = scan_sum(r.tiles);
    r.block_sum = scan_sum(r.blocks);
    return r;
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kLanes - 1);
}
// Tile t among these 64 groups, whose first tile and block are the given ones.
__device__ __forceinline__ bool tile_among(const Groups &r, uint32_t g0, uint32_t tiles0, uint32_t blocks0, uint32_t t,
                                           Span &s) {
    const uint32_t first = tiles0 + r.tile_sum - r.tiles;
    const uint64_t hit = __ballot(r.in && t >= first && t < first + r.tiles);
    if (!hit) return false;
    const int l = __builtin_ctzll(hit);
    s.group = g0 + (uint32_t)l;
    s.begin = (uint32_t)__builtin_amdgcn_readlane((int)r.begin, l);
    s.end = (uint32_t)__builtin_amdgcn_readlane((int)r.end, l);
    s.tile = t - (uint32_t)__builtin_amdgcn_readlane((int)first, l);
    s.blocks0 = blocks0 + (uint32_t)__builtin_amdgcn_readlane((int)(r.block_sum - r.blocks), l);
    s.found = true;
    return true;
}

// The tile that pick(total tiles) names, when every group's rows are cut into
// tiles of `tile_rows` and the tiles of all groups are counted in order; not
// found when it names none of them.  offsets NULL: one group of all rows.  The
// whole wave calls this; the result is uniform.  Up to 64 groups cost one load.
template <typename Pick>
__device__ __forceinline__ Span find_tile(const int32_t *offsets, uint32_t groups, uint32_t rows, uint32_t tile_rows,
                                          Pick pick) {
    Span s = {0, 0, rows, 0, 0, false};
    if (!offsets) {
        const uint32_t total = (rows + tile_rows - 1) / tile_rows;
        s.tile = pick(total);
        s.found = s.tile < total;
        return s;
    }
    if (groups <= kLanes) {
        const Groups r = load_groups(offsets, groups, rows, tile_rows, 0, 0);
        tile_among(r, 0, 0, 0, pick(last_lane(r.tile_sum)), s);
        return s;
    }
    uint32_t total = 0, high = 0;
    for (uint32_t g0 = 0; g0 < groups; g0 += kLanes) {
        const Groups r = load_groups(offsets, groups, rows, tile_rows, g0, high);
        total += last_lane(r.tile_sum);
        high = last_lane(r.end);
    }
    const uint32_t t = pick(total);
    uint32_t tiles = 0, blocks = 0;
    high = 0;
    for (uint32_t g0 = 0; g0 < groups; g0 += kLanes) {
        const Groups r = load_groups(offsets, groups, rows, tile_rows, g0, high);
        if (tile_among(r, g0, tiles, blocks, t, s)) return s;
        tiles += last_lane(r.tile_sum);
        blocks += last_lane(r.block_sum);
        high = last_lane(r.end);
    }
    return s;
}

// Group g's rows and first block, for kernels whose grid is indexed by group.
__device__ __forceinline__ Span find_group(const int32_t *offsets, uint32_t groups, uint32_t rows, uint32_t g) {
    Span s = {g, 0, rows, 0, 0, true};
    if (!offsets) return s;
    uint32_t blocks = 0, high = 0;
    for (uint32_t g0 = 0; g0 <= g; g0 += kLanes) {
        const Groups r = load_groups(offsets, groups, rows, kBlock, g0, high);
        if (g < g0 + kLanes) {
            const int l = (int)(g - g0);
            s.begin = (uint32_t)__builtin_amdgcn_readlane((int)r.begin, l);
            s.end = (uint32_t)__builtin_amdgcn_readlane((int)r.end, l);
            s.blocks0 = blocks + (uint32_t)__builtin_amdgcn_readlane((int)(r.block_sum - r.blocks), l);
        }
        blocks += last_lane(r.block_sum);
        high = last_lane(r.end);
    }
    return s;
}

}  // namespace moe
}  // namespace zc
