// BF16 products with an epilogue, and the gradients of their operands, MI355X / gfx950:
//   forward  out[r, c] = sum_k A[r, k] W[c, k]      both operands along the contraction
//   dgrad    dx[r, j]  = sum_c dpre[r, c] W[c, j]   the right operand across it
//   wgrad    dw[c, j]  = sum_r dpre[r, c] A[r, j]   both across it
// An operand that lies across the contraction comes out of LDS through the
// transposing reads of gfx950, so that nothing is transposed in memory.
#include <math.h>

#include <type_traits>

#include "zc_lds.h"
#include "zc_moe_device.h"

namespace zc {
namespace moe {

typedef float f32v16 __attribute__((ext_vector_type(16)));
typedef float f32v4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef short s16v4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16v4 lds_s16v4;

struct Epilogue {
    const void *bias, *res;
    uint16_t *pre;
    void *out;
    uint64_t res_stride, pre_stride, out_stride;
    uint32_t bias_f32, res_f32, out_f32, act;
    float scale;
};

struct ProductArgs {
    const uint16_t *a, *b;
    uint64_t lda, ldb;  // elements
    uint32_t m, n, k;   // results' rows and columns, contraction
    uint32_t blocks;    // blocks of 64 along the contraction
    uint32_t direct;    // of which the first so many may be loaded whole, 16 bytes at a time
    uint32_t whole;     // so many tiles take all of it; of those that follow, each is `splits` parts
    uint32_t splits;
    float *parts;       // the sums of the parts, tile by tile
    Epilogue e;
};

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// Left and right of 0 the activations are each other's mirror image: beside v or 1, and v * 0 or 0, stands a tail that is even in v.
// A tail comes as the product of `s` and `t`, both as small as its root, so that where the exponential has no digits left,
// each meets a factor of its own before they meet each other: a large gradient keeps the tail's digits, and finite values have finite
// products.  What stands beside a tail is bounded (`x`), so that infinities give the limits; NaN comes through the tail.

// sigmoid(-|v|) = s * t and sigmoid(|v|) = r from e^-|v| = m 4^h, a whole number h, |log2 m| <= 1: the whole part is taken off the
// exponent exactly, and 32 bits of it are left for m.  h is rounded by adding a number whose last bit is 1, and its lowest bits
// become t's exponent.  The hardware's exponential and reciprocal are off by a unit of 32 bits: the sigmoid by less than 7 half
// steps at any v.  (8192 x 4096 x 7168 with SILU: 50 of 410 us; the library's exponential and a division took 76.)
struct Sigmoid {
    float s, t, r, x;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float v) {
    constexpr float kWhole = 12582912.0f;  // 1.5 * 2^23
    Sigmoid g;
    g.x = fminf(fabsf(v), 174.0f);  // from there on h is -126, and m goes on to 0
    const float y = fmaf(g.x, -0.721347520f, kWhole), h2 = fmaf(2.0f, y, -2.0f * kWhole);
    const float m = __builtin_amdgcn_exp2f(fmaf(fabsf(v), -1.92596299e-8f, fmaf(fabsf(v), -1.44269502f, -h2)));
    g.t = __uint_as_float((__float_as_uint(y) << 23) + 0x3F800000u);
    const float mt = m * g.t;
    g.r = __builtin_amdgcn_rcpf(fmaf(mt, g.t, 1.0f));
    g.s = mt * g.r;
    return g;
}
// The normal distribution's tail beyond |v| is m * t^2, with t = e^(-v^2 / 4) and,
// for x = |v| / sqrt(2), m = u * (erfc(x) e^(x^2) / u) / 2, u = 1 / (1 + x / 2): the
// quotient is a polynomial of u to 1e-8 of itself on all of 0..1 (fitted here to its values
// at Chebyshev's points with weights that level the error).  What the square and the exponent of 2 lose
// in rounding, |v|^2 times as much in the tail, is carried on.
struct Tail {
    float m, t, x;
};
__device__ __forceinline__ Tail normal_tail(float v) {
    const float u = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.35355339f, 1.0f));
    float p = 0.0423526122f;
    p = fmaf(p, u, -0.230857749f);
    p = fmaf(p, u, 0.486179082f);
    p = fmaf(p, u, -0.446977725f);
    p = fmaf(p, u, 0.127089673f);
    p = fmaf(p, u, -0.0572325763f);
    p = fmaf(p, u, 0.093000611f);
    p = fmaf(p, u, 0.175376827f);
    p = fmaf(p, u, 0.246880587f);
    p = fmaf(p, u, 0.282093853f);
    p = fmaf(p, u, 0.282094795f);
    constexpr float c = -0.360673760f, c_rest = -4.81490747e-9f;  // of -log2(e) / 4
    const float x = fminf(fabsf(v), 40.0f);                        // from there on the tail is 0
    const float sq = x * x, of2 = sq * c, e = __builtin_amdgcn_exp2f(of2);
    const float rest = fmaf(fmaf(x, x, -sq), c, fmaf(sq, c_rest, fmaf(sq, c, -of2)));
    return {0.5f * u * p, fmaf(e, rest * 0.693147181f, e), x};
}
constexpr float kTanh = 1.59576912f, kCubic = 0.044715f;  // 2 sqrt(2 / pi): (1 + tanh(u)) / 2 = sigmoid(2 u)
constexpr float kDensity = 0.39894228f;                   // 1 / sqrt(2 pi)

__device__ __forceinline__ float activation(float v, uint32_t act) {
    switch (act) {
        case ZC_ACT_RELU: return v > 0.0f ? v : v != v ? v : 0.0f;
        case ZC_ACT_SILU: {
            const Sigmoid g = sigmoid_of(v);
            return fmaf(-g.x * g.s, g.t, fmaxf(v, 0.0f));
        }
        case ZC_ACT_GELU: {
            const Tail n = normal_tail(v);
            return fmaf(-n.x * (n.m * n.t), n.t, fmaxf(v, 0.0f));
        }
        case ZC_ACT_GELU_TANH: {
            const Sigmoid g = sigmoid_of(kTanh * fmaf(kCubic * v * v, v, v));
            return fmaf(-fminf(fabsf(v), 174.0f) * g.s, g.t, fmaxf(v, 0.0f));
        }
        case ZC_ACT_SIGMOID: {
            const Sigmoid g = sigmoid_of(v);
            return v >= 0.0f ? g.r : g.s * g.t;
        }
        default: return v;
    }
}

// d times the slope at v: left of 0 the slope is q, right of it 1 - q, where q is the tail less |v| times its density.
__device__ __forceinline__ float beside(float d, float v, float s, float t) { return v >= 0.0f ? d * fmaf(-s, t, 1.0f) : s * (d * t); }
__device__ __forceinline__ float sloped(float d, float v, uint32_t act) {
    switch (act) {
        case ZC_ACT_RELU: return v > 0.0f ? d : v != v ? v : 0.0f;
        case ZC_ACT_SILU: {
            const Sigmoid g = sigmoid_of(v);
            return beside(d, v, g.s * fmaf(-g.x, g.r, 1.0f), g.t);
        }
        case ZC_ACT_GELU: {
            const Tail n = normal_tail(v);
            return beside(d, v, n.t * fmaf(-n.x, kDensity, n.m), n.t);
        }
        case ZC_ACT_GELU_TANH: {
            // from 30 on the slope is 1 or 0 in 32 bits
            const float x = v != v ? v : fminf(fabsf(v), 30.0f), y = kCubic * x * x;
            const Sigmoid g = sigmoid_of(kTanh * fmaf(y, x, x));
            return beside(d, v, g.s * fmaf(-x * g.r, kTanh * fmaf(3.0f, y, 1.0f), 1.0f), g.t);
        }
        case ZC_ACT_SIGMOID: {
            const Sigmoid g = sigmoid_of(v);
            return g.s * (d * g.t) * g.r;
        }
        default: return d;
    }
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------

// Eight values of either type as they are stored.
struct Raw {
    u32v4 w[2];
    __device__ __forceinline__ void load(const void *p, uint32_t f32, uint64_t at, uint32_t n) {
        if (f32) {
            Eight<true> e;
            e.load(p, at, n, false);
            w[0] = e.w[0];
            w[1] = e.w[1];
        } else {
            Eight<false> e;
            e.load(p, at, n, false);
            w[0] = e.w[0];
        }
    }
    __device__ __forceinline__ void values(uint32_t f32, float (&v)[8]) const {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            v[i] = f32 ? __uint_as_float(w[i / 4][i & 3]) : (i & 1) ? bf_hi(w[0][i / 2]) : bf_lo(w[0][i / 2]);
    }
};
__device__ __forceinline__ void load8(const void *p, uint32_t f32, uint64_t at, uint32_t n, float (&v)[8]) {
    Raw r;
    r.load(p, f32, at, n);
    r.values(f32, v);
}
// The bias of columns c .. c + n - 1, and the residual of row r there.
__device__ __forceinline__ void load_bias(const Epilogue &e, uint32_t c, uint32_t n, float (&v)[8]) {
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = 0.0f;
    if (e.bias) load8(e.bias, e.bias_f32, c, n, v);
}
__device__ __forceinline__ void load_residual(const Epilogue &e, uint64_t r, uint32_t c, uint32_t n, Raw &w) {
    if (e.res) w.load(e.res, e.res_f32, r * e.res_stride + c, n);
}
// The sums of columns c .. c + n - 1 of row r become results in two steps: the pre-activation and its activation,
// and the residual sum.
__device__ __forceinline__ bool activates(const Epilogue &e) { return e.act != ZC_ACT_NONE || e.pre; }
__device__ __forceinline__ void activate8(const Epilogue &e, uint64_t r, uint32_t c, uint32_t n, float (&v)[8]) {
    if (e.pre) store_values<false>(e.pre + r * e.pre_stride + c, pack8(v), n);
    if (e.act != ZC_ACT_NONE)
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = activation(v[i], e.act);
}
__device__ __forceinline__ void store8(const Epilogue &e, uint64_t r, uint32_t c, uint32_t n, float (&v)[8], const Raw &res) {
    if (e.res) {
        float w[8];
        res.values(e.res_f32, w);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] = fmaf(e.scale, v[i], w[i]);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] *= e.scale;
    }
    if (e.out_f32)
        store_floats(static_cast<float *>(e.out) + r * e.out_stride + c, n, v);
    else
        store_values<false>(static_cast<uint16_t *>(e.out) + r * e.out_stride + c, pack8(v), n);
}
__device__ __forceinline__ void finish8(const Epilogue &e, uint64_t r, uint32_t c, uint32_t n, float (&v)[8]) {
    float bias[8];
    Raw res;
    load_bias(e, c, n, bias);
    load_residual(e, r, c, n, res);
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] += bias[i];
    if (activates(e)) activate8(e, r, c, n, v);
    store8(e, r, c, n, v, res);
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

constexpr uint32_t kPThreads = 256;
constexpr uint32_t kPBlock = 64;       // contraction of a stage
constexpr uint32_t kPBytes = 2 * kPBlock;  // of a row or column in a stage

// One operand of a tile of B rows (or columns) of the results.  A stage holds B x
// 64 values in places of 16 bytes, a wave's pieces of 64 places one after another:
//   along   row r of the tile is 128 bytes; chunk c (8 values of the contraction)
//           sits at place c ^ (r / 2 mod 8), so that sixteen lanes that read the
//           same chunk of sixteen rows meet sixteen different columns of banks
//   across  value k of the contraction is 2 B bytes; chunk c (8 results) sits at
//           place c ^ 4 (k mod 4), or c ^ 4 (k / 2 mod 2) where B is 64: a
//           transposing read takes 64 bytes of each of four k, which then lie in
//           four different quarters of the banks
template <uint32_t B, bool ACROSS>
struct Operand {
    static constexpr uint32_t kLoads = B / 32;         // pieces of a wave
    static constexpr uint32_t kTiles = B / 64;         // 32 x 32 tiles of a wave
    static constexpr uint32_t kReads = ACROSS ? 4 : 2;  // of a tile and half stage
    static constexpr uint32_t kRow = B / 8;            // across: chunks of a k

    const uint16_t *p;
    uint64_t ld;
    uint32_t first, last, k;  // the tile's first row, the last one there is; contraction
    uint32_t at[ACROSS ? kTiles : 1];

    // place `lane` of the wave's piece i: row (or k) and chunk
    __device__ __forceinline__ static uint32_t line(uint32_t wave, uint32_t i) {
        return ACROSS ? (wave * kLoads + i) * (kLanes / kRow) + lane_id() / kRow : wave * (B / 4) + 8 * i + lane_id() / 8;
    }
    __device__ __forceinline__ static uint32_t key(uint32_t k) { return B == 64 ? 4 * (k / 2 & 1) : 4 * (k & 3); }
    __device__ __forceinline__ static uint32_t chunk(uint32_t line) {
        return ACROSS ? (lane_id() % kRow) ^ key(line) : (lane_id() & 7) ^ (line / 2 & 7);
    }

    // byte offset of a lane's 16 bytes of a whole block from the block's start, rows past the last repeating it
    __device__ __forceinline__ uint32_t offset(uint32_t wave, uint32_t i) const {
        const uint32_t l = line(wave, i), c = chunk(l), room = last - first;
        return ACROSS ? l * (uint32_t)ld * 2 + min(16 * c, room / 8 * 16) : min(l, room) * (uint32_t)ld * 2 + 16 * c;
    }
    __device__ __forceinline__ const uint8_t *block(uint32_t kb) const {
        const uint64_t e = ACROSS ? (uint64_t)kb * kPBlock * ld + first : (uint64_t)first * ld + (uint64_t)kb * kPBlock;
        return reinterpret_cast<const uint8_t *>(p + e);
    }
    __device__ __forceinline__ uint64_t step() const { return ACROSS ? (uint64_t)kPBlock * ld * 2 : kPBytes; }

    // where a lane's 16 bytes of a whole block are, rows past the last repeating it: at any value, rows any way apart
    __device__ __forceinline__ const uint16_t *source(uint32_t kb, uint32_t wave, uint32_t i) const {
        const uint32_t l = line(wave, i), c = 8 * chunk(l), room = last - first;
        return p + (ACROSS ? ((uint64_t)kb * kPBlock + l) * ld + first + min(c, room / 8 * 8)
                           : (uint64_t)(first + min(l, room)) * ld + (uint64_t)kb * kPBlock + c);
    }
    // any block, any alignment: what lies past the contraction reads as 0
    __device__ __forceinline__ u32v4 load(uint32_t kb, uint32_t wave, uint32_t i) const {
        const uint32_t l = line(wave, i), c = chunk(l);
        const uint32_t kk = kb * kPBlock + (ACROSS ? l : 8 * c), r = first + (ACROSS ? 8 * c : l);
        Eight<false> w;
        w.clear();
        if (kk < k && r <= last) w.load(p, ACROSS ? kk * ld + r : r * ld + kk, ACROSS ? last + 1 - r : k - kk, false);
        return w.w[0];
    }

    // fragments: lane l holds row l mod 32 of a 32 x 32 tile and the contraction's 8 values 8 (l / 32) .. of 16
    __device__ __forceinline__ void place(uint32_t base, uint32_t within) {
        const uint32_t lane = lane_id();
        if (ACROSS) {
            const uint32_t j = lane % 16, k0 = 8 * (lane / 32) + j / 4;
#pragma unroll
            for (uint32_t i = 0; i < kTiles; ++i) {
                const uint32_t c = (within + 32 * i) / 8 + 2 * (lane / 16 & 1) + j % 4 / 2;
                at[ACROSS ? i : 0] = base + k0 * (2 * B) + 16 * (c ^ key(k0)) + 8 * (j & 1);
            }
        } else {
            at[0] = base + (within + lane % 32) * kPBytes;
        }
    }
    // read q of the tile i's fragment: along, the 16 values q of the half; across, 4 values of the contraction
    __device__ __forceinline__ void read(const uint8_t *stage, uint32_t half, uint32_t i, uint32_t q, bf16v8 (&f)[2]) const {
        if constexpr (ACROSS) {
            const uint32_t k = 32 * half + 16 * (q / 2) + 4 * (q & 1);
            const s16v4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16v4 *)(stage + at[i] + k * (2 * B)));
            const auto bits = __builtin_bit_cast(uint2, v);
            u32v4 w = __builtin_bit_cast(u32v4, f[q / 2]);
            w[2 * (q & 1)] = bits.x;
            w[2 * (q & 1) + 1] = bits.y;
            f[q / 2] = __builtin_bit_cast(bf16v8, w);
        } else {
            const uint32_t c = (4 * half + 2 * q + lane_id() / 32) ^ (lane_id() % 32 / 2 & 7u);
            f[q] = *reinterpret_cast<const bf16v8 *>(stage + at[0] + 32 * i * kPBytes + 16 * c);
        }
    }
};

__device__ __forceinline__ uint32_t up8(uint32_t n) { return (n + 7) / 8 * 8; }
// The id-th tile in bands of eight rows of tiles, column by column.
struct TilePlace {
    uint32_t row, col;
};
__device__ __forceinline__ TilePlace tile_place(uint32_t id, uint32_t mtiles, uint32_t ntiles) {
    const uint32_t band = id / (8 * ntiles), in_band = id % (8 * ntiles), band_rows = min(8u, mtiles - 8 * band);
    return {8 * band + in_band % band_rows, in_band / band_rows};
}

// BM x BN tile of four waves (2 x 2).  DIRECT: whole blocks go from memory straight
// into LDS, STAGES of them under way, in the order of the 8-bit products' tiles: the
// fragments of half a block are in registers while the other half's come out
// of LDS, and one barrier in the middle of a block frees its place and hands over
// the next.  Without DIRECT (operands at any element, rows far apart) blocks go
// through registers, two on their way while the one before them is multiplied, and so does the
// contraction's ragged end.  Rates, operands from memory: 8192^3 774 us (1420 TFLOP/s; the library
// reaches 1365), 8192 x 4096 x 7168 347 us (1390 TFLOP/s), both bound by the matrix
// instructions; 8192 x 256 x 7168 in two parts 34 us (121 MB, and 56 blocks a workgroup), 48 x 14336 x
// 4096 21.6 us (117 MB, 5.4 TB/s); without DIRECT 1024 x 4096 x 7168 105 us, rows at odd elements
// 125: a wave's loads, its reads of LDS and its products then follow each other with one wave a SIMD.
template <uint32_t BM, uint32_t BN, uint32_t STAGES, bool XA, bool XB, bool DIRECT>
__global__ __launch_bounds__(kPThreads, STAGES * (BM + BN) * kPBytes > 80 * 1024 ? 1 : 2) void product_kernel(ProductArgs p) {
    typedef Operand<BM, XA> OA;
    typedef Operand<BN, XB> OB;
    constexpr uint32_t MT = OA::kTiles, NT = OB::kTiles, LA = OA::kLoads, LB = OB::kLoads, LOADS = LA + LB;
    constexpr uint32_t kStage = (BM + BN) * kPBytes;
    constexpr uint32_t kRowBytes = BN / 2 * 4 + 16;  // of a wave's results on their way out
    constexpr uint32_t kRoom = STAGES * kStage > 4 * 32 * kRowBytes ? STAGES * kStage : 4 * 32 * kRowBytes;
    __shared__ alignas(1024) uint8_t sh[kRoom];
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);

    // Consecutive workgroups go to the eight XCDs in turn: an XCD gets one run of
    // tiles, in bands of eight rows of tiles, column by column, so that its CUs
    // share rows of both operands in its L2.
    const uint32_t mtiles = (p.m + BM - 1) / BM, ntiles = (p.n + BN - 1) / BN, total = mtiles * ntiles;
    // The tiles past p.whole are split: first the whole tiles, then part after part.
    uint32_t group = blockIdx.x, count = p.whole, part = 0;
    const bool split = group >= up8(p.whole);
    if (split) {
        count = total - p.whole;
        group -= up8(p.whole);
        part = group / up8(count);
        group -= part * up8(count);
    }
    const uint32_t xcd = group % 8, local = group / 8, per = count / 8, rest = count % 8;
    if (local >= per + (xcd < rest)) return;
    const uint32_t nth = xcd * per + min(xcd, rest) + local;
    const TilePlace place = tile_place(split ? p.whole + nth : nth, mtiles, ntiles);
    // (the same in every lane, which the loads into LDS need known)
    const auto same = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane(v); };
    const uint32_t m0 = same(place.row * BM), n0 = same(place.col * BN);
    const uint32_t kb0 = same(split ? (uint32_t)((uint64_t)p.blocks * part / p.splits) : 0u);
    const uint32_t kb1 = same(split ? (uint32_t)((uint64_t)p.blocks * (part + 1) / p.splits) : p.blocks);

    OA oa = {p.a, p.lda, m0, p.m - 1, p.k};
    OB ob = {p.b, p.ldb, n0, p.n - 1, p.k};
    const uint32_t wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * (BN / 2);
    oa.place(0, wm);
    ob.place(BM * kPBytes, wn);

    f32v16 acc[MT][NT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    bf16v8 fa[2][MT][2], fb[2][NT][2];  // [half of the block]
    // the q-th of a half's reads
    constexpr uint32_t kReads = MT * OA::kReads + NT * OB::kReads;
    const auto read_piece = [&](uint32_t at, uint32_t half, uint32_t q) {
        if (q < MT * OA::kReads)
            oa.read(sh + at, half, q / OA::kReads, q % OA::kReads, fa[half][q / OA::kReads % MT]);
        else
            ob.read(sh + at, half, (q - MT * OA::kReads) / OB::kReads % NT, (q - MT * OA::kReads) % OB::kReads,
                    fb[half][(q - MT * OA::kReads) / OB::kReads % NT]);
    };
    // B in the place of the left matrix: a lane then holds four consecutive columns of one row
    const auto multiply = [&](uint32_t half, uint32_t i, uint32_t j) {
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[half][j][h], fa[half][i][h], acc[i][j], 0, 0, 0);
    };

    const uint32_t whole = min(kb1, p.direct);
    if constexpr (DIRECT) if (kb0 < whole) {
        const uint32_t blocks = whole - kb0;
        const uint8_t *ga = oa.block(kb0), *gb = ob.block(kb0);
        uint32_t offa[LA], offb[LB];
#pragma unroll
        for (uint32_t i = 0; i < LA; ++i) offa[i] = oa.offset(wave, i);
#pragma unroll
        for (uint32_t i = 0; i < LB; ++i) offb[i] = ob.offset(wave, i);
        const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)&sh[0]);
        const uint32_t ldsa = lds0 + wave * LA * 1024, ldsb = lds0 + BM * kPBytes + wave * LB * 1024;
        const auto load_piece = [&](uint32_t t, uint32_t at, uint32_t i) {  // the wave's i-th load of block kb0 + t
            if (i < LA)
                lds_load16(ga + t * oa.step(), offa[i % LA], ldsa + at + i * 1024);
            else
                lds_load16(gb + t * ob.step(), offb[(i - LA) % LB], ldsb + at + (i - LA) * 1024);
        };
#pragma unroll
        for (uint32_t t = 0; t < STAGES; ++t)
            if (t < blocks)
#pragma unroll
                for (uint32_t i = 0; i < LOADS; ++i) load_piece(t, t * kStage, i);
        if (blocks >= STAGES)
            wait_and_meet<(int)((STAGES - 1) * LOADS)>();
        else
            wait_and_meet<0>();
#pragma unroll
        for (uint32_t q = 0; q < kReads; ++q) read_piece(0, 0, q);

        uint32_t at0 = 0, at1 = STAGES > 1 ? kStage : 0;  // where blocks t and t + 1 are
        const auto step = [&](uint32_t t, auto more) {
            constexpr bool MORE = decltype(more)::value;  // there is a block to load into this one's place
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {
                // block t + 1 has landed, and every wave holds the rest of block t
                if (half == 1) wait_and_meet<MORE ? (int)((STAGES - 2) * LOADS) : 0>();
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < NT; ++j) {
                        multiply(half, i, j);
                        constexpr uint32_t kSlots = MT * NT;
                        const uint32_t slot = i * NT + j;
                        if (MORE && half == 1)
#pragma unroll
                            for (uint32_t q = slot * LOADS / kSlots; q < (slot + 1) * LOADS / kSlots; ++q)
                                load_piece(t + STAGES, at0, q);
#pragma unroll
                        for (uint32_t q = slot * kReads / kSlots; q < (slot + 1) * kReads / kSlots; ++q)
                            read_piece(half ? at1 : at0, half ^ 1, q);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
            at0 = at1;
            at1 = at1 == (STAGES - 1) * kStage ? 0 : at1 + kStage;
        };
        uint32_t t = 0;
        for (; t + STAGES < blocks; ++t) step(t, std::true_type{});
        for (; t < blocks; ++t) step(t, std::false_type{});
        wait_and_meet<0>();
    }
    // a block in registers into place in LDS, and from there into the sums
    const auto lay_block = [&](uint32_t at, const u32v4 (&w)[LOADS]) {
#pragma unroll
        for (uint32_t i = 0; i < LOADS; ++i) {
            const uint32_t to = i < LA ? (wave * LA + i) * 1024 : BM * kPBytes + (wave * LB + i - LA) * 1024;
            *reinterpret_cast<u32v4 *>(sh + at + to + 16 * lane) = w[i];
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // (the loads under way are not waited for)
    };
    const auto take_block = [&](uint32_t at) {
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {
#pragma unroll
            for (uint32_t q = 0; q < kReads; ++q) read_piece(at, half, q);
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
                for (uint32_t j = 0; j < NT; ++j) multiply(half, i, j);
        }
    };
    if constexpr (!DIRECT) if (kb0 < whole) {
        // two places in turn: one is written while other waves may still read the other; two blocks on their way
        static_assert(STAGES == 2, "two places");
        const uint16_t *from[LOADS];
        u32v4 w[2][LOADS];
#pragma unroll
        for (uint32_t i = 0; i < LOADS; ++i) from[i] = i < LA ? oa.source(kb0, wave, i) : ob.source(kb0, wave, i - LA);
        const uint64_t last = whole - 1 - kb0;
        // (past the last whole block that one again: no branch around the loads, so that each is waited for by itself)
        const auto fetch_block = [&](uint64_t t, u32v4 (&to)[LOADS]) {
#pragma unroll
            for (uint32_t i = 0; i < LOADS; ++i)
                to[i] = *reinterpret_cast<const u32v4a2 *>(from[i] + min(t, last) * ((i < LA ? oa.step() : ob.step()) / 2));
        };
        fetch_block(0, w[0]);
        fetch_block(1, w[1]);
        for (uint32_t kb = kb0; kb < whole; kb += 2) {
            lay_block(0, w[0]);
            fetch_block(kb + 2 - kb0, w[0]);
            take_block(0);
            if (kb + 1 == whole) break;
            lay_block(kStage, w[1]);
            fetch_block(kb + 3 - kb0, w[1]);
            take_block(kStage);
        }
    }
    for (uint32_t kb = max(whole, kb0); kb < kb1; ++kb) {
        u32v4 w[LOADS];
#pragma unroll
        for (uint32_t i = 0; i < LOADS; ++i) w[i] = i < LA ? oa.load(kb, wave, i) : ob.load(kb, wave, i - LA);
        __syncthreads();  // every wave is done with the block before
        lay_block(0, w);
        take_block(0);
    }

    // Results through LDS, 32 rows of a wave at a time, so that a row's BN / 2 columns
    // leave as whole lines, eight a lane.  The residual of the next 32 rows is on its way
    // meanwhile: one row after another, each load waited for the stores before it
    // (8192 x 7168 x 4096 with a residual: 500 us instead of 381).
    __syncthreads();
    Epilogue e = p.e;
    if (split) {
        e = {};
        const uint64_t first = ((uint64_t)part * count + nth) * BM * BN - (uint64_t)m0 * BN - n0;
        e.out = reinterpret_cast<float *>(reinterpret_cast<uint64_t>(p.parts) + first * 4);
        e.out_stride = BN;
        e.out_f32 = 1;
        e.scale = 1.0f;
    }
    uint8_t *mine = sh + wave * 32 * kRowBytes;
    constexpr uint32_t eights = BN / 16, step = kLanes / eights, kTurns = 32 / step;
    const uint32_t c = n0 + wn + lane % eights * 8, n = c < p.n ? min(p.n - c, 8u) : 0u, r0 = m0 + wm + lane / eights;
    float bias[8];
    load_bias(e, c, n, bias);
    const bool acts = activates(e);
    f32v4 *const from = reinterpret_cast<f32v4 *>(mine + lane / eights * kRowBytes + lane % eights * 32);
    constexpr uint32_t kApart = step * kRowBytes / 16;
    const auto lay = [&](uint32_t i) {  // 32 rows into LDS
#pragma unroll
        for (uint32_t j = 0; j < NT; ++j)
#pragma unroll
            for (uint32_t q = 0; q < 16; q += 4)
                *reinterpret_cast<f32v4 *>(mine + lane % 32 * kRowBytes + (32 * j + 2 * q + 4 * (lane / 32)) * 4) =
                    f32v4{acc[i][j][q], acc[i][j][q + 1], acc[i][j][q + 2], acc[i][j][q + 3]};
    };
    // A whole tile without an activation: no branch stands between its loads and stores, so that the wait for the
    // next rows' residual is not one for the stores before it.  kind: no residual, BF16, floats.
    const auto finish = [&](auto f32, auto kind) {
        constexpr bool F32 = decltype(f32)::value;
        constexpr uint32_t K = decltype(kind)::value;
        Eight<K == 2> res[2][K ? kTurns : 1];
        const auto fetch = [&](uint32_t i) {
            if (K)
#pragma unroll
                for (uint32_t q = 0; q < kTurns; ++q)
                    res[i & 1][q % (K ? kTurns : 1)].load(e.res, (uint64_t)(r0 + 32 * i + q * step) * e.res_stride + c, 8, false);
        };
        fetch(0);
#pragma unroll
        for (uint32_t i = 0; i < MT; ++i) {
            lay(i);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (i + 1 < MT) fetch(i + 1);
#pragma unroll
            for (uint32_t q = 0; q < kTurns; ++q) {
                const f32v4 lo = from[q * kApart], hi = from[q * kApart + 1];
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
                for (uint32_t x = 0; x < 8; ++x)
                    v[x] = K ? fmaf(e.scale, v[x] + bias[x], res[i & 1][q % (K ? kTurns : 1)][x]) : (v[x] + bias[x]) * e.scale;
                const uint64_t at = (uint64_t)(r0 + 32 * i + q * step) * e.out_stride + c;
                if (F32)
                    store_floats(static_cast<float *>(e.out) + at, 8, v);
                else
                    store_values<false>(static_cast<uint16_t *>(e.out) + at, pack8(v), 8);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    };
    if (split || (!acts && m0 + BM <= p.m && n0 + BN <= p.n)) {  // (a part has room for the whole tile)
        typedef std::integral_constant<uint32_t, 0> None;
        typedef std::integral_constant<uint32_t, 1> Halves;
        typedef std::integral_constant<uint32_t, 2> Floats;
        if (e.out_f32)
            !e.res ? finish(std::true_type{}, None{}) : e.res_f32 ? finish(std::true_type{}, Floats{}) : finish(std::true_type{}, Halves{});
        else
            !e.res ? finish(std::false_type{}, None{}) : e.res_f32 ? finish(std::false_type{}, Floats{}) : finish(std::false_type{}, Halves{});
        return;
    }
    Raw next[kTurns];
    const auto fetch = [&](uint32_t i) {
#pragma unroll
        for (uint32_t q = 0; q < kTurns; ++q) {
            const uint32_t r = r0 + 32 * i + q * step;
            if (r < p.m && n) load_residual(e, r, c, n, next[q]);
        }
    };
    fetch(0);
#pragma unroll 1
    for (uint32_t i = 0; i < MT; ++i) {
        // (sums stay in registers only under indexes that the compiler knows)
#pragma unroll
        for (uint32_t known = 0; known < MT; ++known)
            if (known == i) lay(known);
        Raw res[kTurns];
#pragma unroll
        for (uint32_t q = 0; q < kTurns; ++q) res[q] = next[q];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (i + 1 < MT) fetch(i + 1);
        if (acts && !e.res) {
#pragma unroll 2
            for (uint32_t q = 0; q < kTurns; ++q) {
                const uint32_t r = r0 + 32 * i + q * step;
                const f32v4 lo = from[q * kApart], hi = from[q * kApart + 1];
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
                for (uint32_t x = 0; x < 8; ++x) v[x] += bias[x];
                if (r < p.m && n) {
                    activate8(e, r, c, n, v);
                    store8(e, r, c, n, v, Raw{});
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            continue;
        }
        if (acts)  // in its place in LDS: the code of the activations stands here once
#pragma unroll 1
            for (uint32_t q = 0; q < kTurns; ++q) {
                const uint32_t r = r0 + 32 * i + q * step;
                const f32v4 lo = from[q * kApart], hi = from[q * kApart + 1];
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
                for (uint32_t x = 0; x < 8; ++x) v[x] += bias[x];
                if (r < p.m && n) activate8(e, r, c, n, v);
                from[q * kApart] = f32v4{v[0], v[1], v[2], v[3]};
                from[q * kApart + 1] = f32v4{v[4], v[5], v[6], v[7]};
            }
#pragma unroll
        for (uint32_t q = 0; q < kTurns; ++q) {
            const uint32_t r = r0 + 32 * i + q * step;
            const f32v4 lo = from[q * kApart], hi = from[q * kApart + 1];
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (!acts)
#pragma unroll
                for (uint32_t x = 0; x < 8; ++x) v[x] += bias[x];
            if (r < p.m && n) store8(e, r, c, n, v, res[q]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// The parts of split tiles of 1 << row_bits rows and 1 << col_bits columns, added in order: bound by
// a launch and by the parts, 8192 x 256 in two parts 6.4 us (25 MB), eight tiles of 128 x 128 in eight 6.2.
__global__ __launch_bounds__(256) void product_join_kernel(ProductArgs p, uint32_t row_bits, uint32_t col_bits) {
    const uint32_t bits = row_bits + col_bits - 3;  // of eights of a tile
    const uint32_t mtiles = (p.m + (1u << row_bits) - 1) >> row_bits, ntiles = (p.n + (1u << col_bits) - 1) >> col_bits;
    const uint64_t all = (uint64_t)(mtiles * ntiles - p.whole) << bits;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (uint64_t)gridDim.x * 256) {
        const TilePlace place = tile_place(p.whole + (uint32_t)(i >> bits), mtiles, ntiles);
        const uint32_t in = (uint32_t)i & ((1u << bits) - 1);
        const uint32_t r = (place.row << row_bits) + (in >> (col_bits - 3));
        const uint32_t c = (place.col << col_bits) + (in & ((1u << (col_bits - 3)) - 1)) * 8;
        if (r >= p.m || c >= p.n) continue;
        const f32v4 *from = reinterpret_cast<const f32v4 *>(p.parts + i * 8);
        f32v4 lo = from[0], hi = from[1];
#pragma unroll 2
        for (uint32_t s = 1; s < p.splits; ++s) {
            lo += from[s * all * 2];
            hi += from[s * all * 2 + 1];
        }
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        finish8(p.e, r, c, min(p.n - c, 8u), v);
    }
}

// ---------------------------------------------------------------------------
// few rows: bound by reading the weights
// ---------------------------------------------------------------------------

// 16 bytes at any value.  A wave's 16-byte loads take three times as long where an address is not on 4 bytes (2 x 4096 x
// 10880 with rows at odd values 47.8 us, on 4 bytes 19.8): then the words they lie in are loaded, the first with the
// value before, and the last value by itself, and shifted into
// place (29.6 to 33.9 us; in tiles, whose waves have more loads than they can issue, this took 1.2 times as long as loads at any value).
template <bool ODD>
struct Loose {
    u32v4 w;
    uint32_t last;
    __device__ __forceinline__ static uint32_t shift(const uint16_t *p) { return (uint32_t)(uintptr_t)p & 2u; }
    __device__ __forceinline__ void load(const uint16_t *p) {
        w = *reinterpret_cast<const u32v4a4 *>(p - (ODD ? shift(p) / 2 : 0u));
        if (ODD) last = p[7];
    }
    __device__ __forceinline__ u32v4 value(uint32_t by) const {
        if (!ODD) return w;
        return u32v4{__builtin_amdgcn_alignbyte(w[1], w[0], by), __builtin_amdgcn_alignbyte(w[2], w[1], by),
                     __builtin_amdgcn_alignbyte(w[3], w[2], by), __builtin_amdgcn_alignbyte(last, w[3], by)};
    }
};

// 16 rows of B against 16 MT rows of A, both along the contraction.  The waves of a
// block take its blocks of 64 in turn, STEP at a time, straight from memory into
// the registers of the matrix instructions, and add their sums through LDS.  1 x
// 4096 x 14336, weights from memory: 22.9 us, 5.1 TB/s, what a large copy reaches.
template <uint32_t MT, uint32_t WAVES, uint32_t STEP, bool ODD>
__global__ __launch_bounds__(WAVES * 64) void product_rows_kernel(ProductArgs p) {
    __shared__ f32v4 part[WAVES][MT][kLanes];
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t ntiles = (p.n + 15) / 16, n0 = blockIdx.x % ntiles * 16, m0 = blockIdx.x / ntiles * 16 * MT;
    const uint32_t fr = lane % 16, fc = 8 * (lane / 16);
    const uint16_t *b = p.b + (uint64_t)min(n0 + fr, p.n - 1) * p.ldb;
    const uint16_t *a[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) a[i] = p.a + (uint64_t)min(m0 + 16 * i + fr, p.m - 1) * p.lda;
    f32v4 acc[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) acc[i] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t whole = p.k / kPBlock;
    // two turns' values in registers: one on its way while the other is multiplied
    struct Turn {
        Loose<ODD> b[STEP][2], a[STEP][MT][2];
    };
    const uint32_t byb = Loose<ODD>::shift(b);
    uint32_t bya[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) bya[i] = Loose<ODD>::shift(a[i]);
    Turn turns[2];
    const auto load = [&](Turn &t, uint32_t kb) {
#pragma unroll
        for (uint32_t u = 0; u < STEP; ++u)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                const uint64_t at = (uint64_t)(kb + u) * kPBlock + 32 * h + fc;
                t.b[u][h].load(b + at);
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i) t.a[u][i][h].load(a[i] + at);
            }
    };
    const auto take = [&](const Turn &t) {
#pragma unroll
        for (uint32_t u = 0; u < STEP; ++u)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8, t.b[u][h].value(byb)),
                                                                     __builtin_bit_cast(bf16v8, t.a[u][i][h].value(bya[i])), acc[i], 0, 0, 0);
    };
    uint32_t kb = wave * STEP;
    constexpr uint32_t kTurn = WAVES * STEP;
    if (kb + STEP <= whole) {
        load(turns[0], kb);
        for (;;) {
            kb += kTurn;
            if (kb + STEP > whole) {
                take(turns[0]);
                break;
            }
            load(turns[1], kb);
            take(turns[0]);
            kb += kTurn;
            if (kb + STEP > whole) {
                take(turns[1]);
                break;
            }
            load(turns[0], kb);
            take(turns[1]);
        }
    }
    // what is left of this wave's last turn, the contraction's ragged end in it
    for (uint32_t u = 0; u < STEP && kb + u < p.blocks; ++u)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t at = (kb + u) * kPBlock + 32 * h + fc, n = at < p.k ? p.k - at : 0u;
            Eight<false> wb, wa;
            wb.load(b, at, n, false);
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) {
                wa.load(a[i], at, n, false);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8, wb.w[0]),
                                                                 __builtin_bit_cast(bf16v8, wa.w[0]), acc[i], 0, 0, 0);
            }
        }
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    // a lane of the sums holds four consecutive columns of one row: two lanes' make eight
    if (lane >= 32) return;
    for (uint32_t i = wave; i < MT; i += WAVES) {
        const uint32_t from = lane % 16 + 32 * (lane / 16);
        f32v4 lo = part[0][i][from], hi = part[0][i][from + 16];
#pragma unroll
        for (uint32_t w = 1; w < WAVES; ++w) {
            lo += part[w][i][from];
            hi += part[w][i][from + 16];
        }
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const uint32_t r = m0 + 16 * i + lane % 16, c = n0 + 8 * (lane / 16);
        if (r < p.m && c < p.n) finish8(p.e, r, c, min(p.n - c, 8u), v);
    }
}

// ---------------------------------------------------------------------------
// the gradient of the pre-activation, and of the bias
// ---------------------------------------------------------------------------

struct SlopeArgs {
    const void *dout;
    const uint16_t *pre;
    uint16_t *dpre;
    float *parts;
    uint64_t dout_stride, pre_stride, dpre_stride;
    uint32_t rows, cols, row_step, act, dout_f32;
    float scale;
};
// A block takes 64 * 8 columns and, over its four waves, every fourth row of its run of rows, two rows of a wave
// on their way at once.  Bound by memory: 8192 x 4096 with
// SILU 50 us, 4 TB/s (64 runs of rows, a row of a wave at a time: 87).
constexpr uint32_t kSWaves = 4;
template <bool WIDE>
__global__ __launch_bounds__(kSWaves * kLanes) void slope_kernel(SlopeArgs a) {
    __shared__ float sums[kSWaves][kLanes * 8];
    const uint32_t lane = lane_id(), wave = threadIdx.x / kLanes;
    const uint32_t c = (blockIdx.x * kLanes + lane) * 8, n = c < a.cols ? min(a.cols - c, 8u) : 0u;
    const uint64_t r1 = min((uint64_t)a.rows, (uint64_t)(blockIdx.y + 1) * a.row_step);
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const auto fetch = [&](uint64_t r, Raw &d, Eight<false> &v) {
        if (r >= r1) return;
        d.load(a.dout, a.dout_f32, r * a.dout_stride + c, n);
        if (a.act != ZC_ACT_NONE) v.load(a.pre, r * a.pre_stride + c, n, true);
    };
    const auto work = [&](uint64_t r, const Raw &raw, const Eight<false> &v) {
        if (r >= r1) return;
        float d[8];
        raw.values(a.dout_f32, d);
        if (a.act != ZC_ACT_NONE)
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) d[i] = sloped(d[i], v[i], a.act);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            d[i] *= a.scale;
            acc[i] += d[i];
        }
        if (a.dpre) store_values<WIDE>(a.dpre + r * a.dpre_stride + c, pack8(d), n);
    };
    for (uint64_t r = (uint64_t)blockIdx.y * a.row_step + wave; r < r1; r += 2 * kSWaves) {
        Raw d0, d1;
        Eight<false> v0, v1;
        fetch(r, d0, v0);
        fetch(r + kSWaves, d1, v1);
        work(r, d0, v0);
        work(r + kSWaves, d1, v1);
    }
    if (!a.parts) return;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) sums[wave][lane * 8 + i] = acc[i];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kLanes * 8; i += kSWaves * kLanes) {
        const uint32_t col = blockIdx.x * kLanes * 8 + i;
        float s = sums[0][i];
#pragma unroll
        for (uint32_t w = 1; w < kSWaves; ++w) s += sums[w][i];
        if (col < a.cols) a.parts[(uint64_t)blockIdx.y * a.cols + col] = s;
    }
}
// The parts of a column's sum, added in order: 64 columns a block, in 16 runs of parts.  256 parts
// of 4096 columns 7.3 us, a launch and the latency of 16 loads in a row.
constexpr uint32_t kRuns = 16;
__global__ __launch_bounds__(kLanes * kRuns) void column_sums_kernel(const float *parts, uint32_t count, uint32_t cols,
                                                                     float *out) {
    __shared__ float run[kRuns][kLanes];
    const uint32_t c = blockIdx.x * kLanes + lane_id(), w = threadIdx.x / kLanes;
    float v = 0.0f;
    if (c < cols)
        for (uint32_t i = count * w / kRuns; i < count * (w + 1) / kRuns; ++i) v += parts[(uint64_t)i * cols + c];
    run[w][lane_id()] = v;
    __syncthreads();
    if (w || c >= cols) return;
#pragma unroll
    for (uint32_t i = 1; i < kRuns; ++i) v += run[i][lane_id()];
    out[c] = v;
}

// ---------------------------------------------------------------------------
// which kernel
// ---------------------------------------------------------------------------

enum Tile { kT128, kT128Deep, kT256x128, kT256, kT128x64, kT64, kTAny, kTAny64 };
struct ProductChoice {
    uint32_t rows_mt;  // > 0: product_rows_kernel with so many tiles of 16 rows
    Tile tile;
    uint32_t tm, tn, splits;
    uint64_t tiles, whole;  // the first so many tiles are not split

    uint64_t groups() const { return splits > 1 ? ceil_div(whole, 8) * 8 + splits * (ceil_div(tiles - whole, 8) * 8) : ceil_div(tiles, 8) * 8; }
    uint64_t part_bytes() const { return splits > 1 ? (tiles - whole) * tm * tn * 4 * splits : 0; }
};

// Up to 32 rows: product_rows_kernel, if the model beneath it puts no tile before it.  2 x 4096 x 10880 takes 20.9 us
// there and 25.1 in tiles in eight parts, 2 x 162 x 10880 16.1 and 10.5, with rows at odd values 25.6 and 15.9.  Of 240
// products of 1 to 32 rows, 162 to 8192 columns and contractions of 512 to 13312 the choice is within 5 % of the
// faster in 218 and within 20 % in 236; at worst it takes 1.4 times as long (24 x 8192 x 2560 at odd values).
// The shape and split with the least time by this model: the workgroups of one turn of
// the CUs cost `start` us, and each block of 64 of their contraction `alone` us a turn or
// `shared` us a workgroup of the busiest CU, whichever is more; the parts of a split cost a
// launch and their bytes.  All tiles are split, or none, or those that overhang the last whole
// turn of one tile a CU (1021 x 4099 x 7173, 264 tiles: 174 us whole, 161 with all in two
// parts, 133 with the last eight in four).  The figures are fitted, for the order of the choices and not for
// their times, to every shape and split timed at 17 to 8192 rows, 256 to 8192 columns and
// contractions of 512 to 14336, operands from memory, in all three directions: of 484
// products the choice is within 5 % of the fastest in 424 and within 20 % in 470; at worst it takes
// 1.8 times as long, at 17 x 1024 x 2048 (16 us with eight parts where no split takes 9).  With
// operands off the wide path, of 324 products 311 and 324.
struct TileRate {
    Tile tile;
    uint32_t tm, tn, at_once;
    double start, alone, shared;
};
constexpr TileRate kDirectTiles[] = {
    {kT128, 128, 128, 512, 0.0, 1.64, 1.07},      {kT128Deep, 128, 128, 256, 3.35, 0.96, 0.107},
    {kT256x128, 256, 128, 256, 9.7, 1.314, 0.26}, {kT256, 256, 256, 256, 11.06, 2.124, 1.744},
    {kT128x64, 128, 64, 256, 3.21, 0.18, 0.774},  {kT64, 64, 64, 512, 0.0, 0.24, 0.551}};
constexpr TileRate kAnyTiles[] = {{kTAny, 128, 128, 512, 1.52, 0.0, 0.801}, {kTAny64, 64, 64, 1024, 0.0, 0.01, 0.395}};
// of product_rows_kernel: a block of the contraction, a row beside it (us), bytes of the weights a us
struct RowsRate {
    double block, row, bytes;
};
constexpr RowsRate kDirectRows = {0.1, 0.008, 3.2e6}, kAnyRows = {0.1, 0.006, 4.2e6};
constexpr uint32_t kMostSplits = 8;
constexpr uint64_t kMostGroups = 0xFFFFFFFFull / kPThreads;  // of one launch
constexpr double kJoinStart = 4.27, kJoinBytes = 0.895e6, kAnyJoinStart = 2.94, kAnyJoinBytes = 2.9e6;  // us; bytes a us

static uint32_t log2_of(uint32_t n) { return 31 - (uint32_t)__builtin_clz(n); }

static ProductChoice product_choice(uint64_t m, uint64_t n, uint64_t k, bool along, bool direct, uint32_t most_splits) {
    ProductChoice c = {};
    const double blocks = (double)ceil_div(k, kPBlock);
    double best = 0.0;
    if (along && m <= 32 && ceil_div(n, 16) < (1u << 22)) {
        const RowsRate &r = direct ? kDirectRows : kAnyRows;
        const double alone = blocks * (r.block + r.row * (double)m), bytes = (double)(n * k * 2) / r.bytes;
        c.rows_mt = m <= 16 ? 1 : 2;
        c.splits = 1;
        best = 1.0 + (alone > bytes ? alone : bytes);
    }
    const auto offer = [&](const TileRate &t, uint32_t splits, uint64_t tiles, uint64_t whole) {
        const ProductChoice o = {0, t.tile, t.tm, t.tn, splits, tiles, whole};
        if (o.part_bytes() > ZC_MATMUL_WORKSPACE_MAX || o.groups() > kMostGroups) return;
        const uint64_t parts = (tiles - whole) * splits, turns = ceil_div(whole, t.at_once), beside = turns * t.at_once - whole;
        const double more = (double)ceil_div(parts > beside ? parts - beside : 0, t.at_once);
        const double alone = (double)turns + more / splits;
        const double busiest = (double)ceil_div(whole, 256) + (double)ceil_div(parts, 256) / splits;
        double us = t.start * ((double)turns + more) + blocks * (t.alone * alone > t.shared * busiest ? t.alone * alone : t.shared * busiest);
        if (splits > 1)
            us += (direct ? kJoinStart : kAnyJoinStart) + (double)o.part_bytes() / (direct ? kJoinBytes : kAnyJoinBytes);
        if (best == 0.0 || us < best) {
            best = us;
            c = o;
        }
    };
    const auto offer_tile = [&](const TileRate &t) {
        const uint64_t tiles = ceil_div(m, t.tm) * ceil_div(n, t.tn), turns = tiles / 256 * 256;
        offer(t, 1, tiles, tiles);
        for (uint32_t s = 2; s <= most_splits && blocks >= 2 * s; s *= 2) {
            offer(t, s, tiles, 0);
            if (turns && turns < tiles) offer(t, s, tiles, turns);
        }
    };
    if (direct)
        for (const TileRate &t : kDirectTiles) offer_tile(t);
    else
        for (const TileRate &t : kAnyTiles) offer_tile(t);
    return c;
}

template <bool XA, bool XB>
static void launch_tiles(const ProductArgs &p, Tile tile, dim3 grid, Launches &on) {
    const dim3 block(kPThreads);
    switch (tile) {
        case kT256: return on.launch((product_kernel<256, 256, 2, XA, XB, true>), grid, block, p);
        case kT256x128: return on.launch((product_kernel<256, 128, 3, XA, XB, true>), grid, block, p);
        case kT128Deep: return on.launch((product_kernel<128, 128, 3, XA, XB, true>), grid, block, p);
        case kT128: return on.launch((product_kernel<128, 128, 2, XA, XB, true>), grid, block, p);
        case kT128x64: return on.launch((product_kernel<128, 64, 6, XA, XB, true>), grid, block, p);
        case kT64: return on.launch((product_kernel<64, 64, 4, XA, XB, true>), grid, block, p);
        case kTAny64: return on.launch((product_kernel<64, 64, 2, XA, XB, false>), grid, block, p);
        default: return on.launch((product_kernel<128, 128, 2, XA, XB, false>), grid, block, p);
    }
}

// Straight loads into LDS take 16 bytes at a time from 32-bit offsets.
static bool direct_ok(const void *p, uint64_t ld) { return aligned(p, 16) && ld % 8 == 0 && ld <= (1u << 22); }

static zc_status launch_product(ProductArgs p, uint64_t m, uint64_t n, uint64_t k, bool xa, bool xb, void *ws,
                                uint64_t ws_bytes, void *stream) {
    p.m = (uint32_t)m;
    p.n = (uint32_t)n;
    p.k = (uint32_t)k;
    p.blocks = (uint32_t)ceil_div(k, kPBlock);
    const bool direct = direct_ok(p.a, p.lda) && direct_ok(p.b, p.ldb);
    const bool odd = !aligned(p.a, 4) || !aligned(p.b, 4) || p.lda % 2 || p.ldb % 2;
    // a whole block may be loaded unless its last chunks pass the end of the operand
    p.direct = p.k / kPBlock;
    if (k % kPBlock == 0 && p.direct && ((xa && m % 8) || (xb && n % 8))) --p.direct;
    if ((xa && p.lda < 8) || (xb && p.ldb < 8)) p.direct = 0;
    const bool room = ws && ws_bytes >= zc_matmul_workspace_bytes(m, n, k);
    const ProductChoice c = product_choice(m, n, k, !xa && !xb, direct, room ? kMostSplits : 1);
    const uint64_t groups = c.rows_mt ? ceil_div(m, 16 * c.rows_mt) * ceil_div(n, 16) : c.groups();
    if (!groups) return ZC_ERR_INVALID_ARG;  // more tiles than a launch takes
    Launches on(stream);
    if (c.rows_mt) {
        const dim3 grid((uint32_t)groups);
        // (8 waves, 2, or turns of 2, 6 or 8 blocks took 1 to 1.2 times as long, loads marked for single use 1.3)
        if (c.rows_mt == 1)
            on.launch((odd ? product_rows_kernel<1, 4, 4, true> : product_rows_kernel<1, 4, 4, false>), grid, dim3(256), p);
        else
            on.launch((odd ? product_rows_kernel<2, 4, 4, true> : product_rows_kernel<2, 4, 4, false>), grid, dim3(256), p);
        return on.status();
    }
    p.whole = (uint32_t)c.whole;
    p.splits = c.splits;
    p.parts = static_cast<float *>(ws);
    const dim3 grid((uint32_t)groups);
    if (!xa && !xb) launch_tiles<false, false>(p, c.tile, grid, on);
    if (!xa && xb) launch_tiles<false, true>(p, c.tile, grid, on);
    if (xa && xb) launch_tiles<true, true>(p, c.tile, grid, on);
    if (c.splits > 1) {
        const uint64_t units = (c.tiles - c.whole) * c.tm * c.tn / 8 / 256;
        on.launch(product_join_kernel, dim3((uint32_t)(units < 4096 ? units : 4096)), dim3(256), p, log2_of(c.tm), log2_of(c.tn));
    }
    return on.status();
}

static bool real_type(uint32_t t) { return t == ZC_F32 || t == ZC_BF16; }
static bool typed_aligned(const void *p, uint32_t type) { return aligned(p, type == ZC_F32 ? 4 : 2); }
static bool row_ok(uint64_t stride, uint64_t cols) { return stride >= cols && stride <= kMaxStride; }
static bool finite_float(float v) { return v - v == 0.0f; }

// A gradient: add + product.
static zc_status gradient(ProductArgs p, uint64_t m, uint64_t n, uint64_t k, bool xa, const void *d_add,
                          uint32_t add_type, uint64_t add_stride, void *d_out, uint32_t out_type, uint64_t out_stride,
                          void *ws, uint64_t ws_bytes, void *stream) {
    if (!real_type(out_type) || !row_ok(out_stride, n) || (d_add && (!real_type(add_type) || !row_ok(add_stride, n))))
        return ZC_ERR_INVALID_ARG;
    if (!m || !n) return ZC_OK;
    if (!d_out || (k && (!p.a || !p.b))) return ZC_ERR_INVALID_ARG;
    if (!aligned(p.a, 2) || !aligned(p.b, 2) || !typed_aligned(d_out, out_type) ||
        (d_add && !typed_aligned(d_add, add_type)) || !aligned(ws, 16))
        return ZC_ERR_MISALIGNED;
    p.e.res = d_add;
    p.e.res_f32 = add_type == ZC_F32;
    p.e.res_stride = add_stride;
    p.e.out = d_out;
    p.e.out_f32 = out_type == ZC_F32;
    p.e.out_stride = out_stride;
    p.e.scale = 1.0f;
    return launch_product(p, m, n, k, xa, true, ws, ws_bytes, stream);
}

constexpr uint32_t kSlopeRuns = 256;  // runs of rows whose column sums are parts, at most

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_matmul_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t contraction) {
    if (rows > kMaxRows || cols > kMaxRows || contraction > kMaxRows || !rows || !cols) return 0;
    uint64_t most = 0;
    for (int along = 0; along < 2; ++along)
        for (int direct = 0; direct < 2; ++direct) {
            const ProductChoice c = product_choice(rows, cols, contraction, along != 0, direct != 0, kMostSplits);
            if (c.part_bytes() > most) most = c.part_bytes();
        }
    return most;
}

extern "C" zc_status zc_matmul(const void *d_a, uint64_t m, uint64_t a_stride, const void *d_w, uint64_t n, uint64_t k,
                               uint64_t w_stride, const zc_epilogue *epilogue, void *d_out, uint32_t out_type,
                               uint64_t out_stride, void *d_workspace, uint64_t workspace_bytes, void *stream) {
    if (m > kMaxRows || n > kMaxCols || k > kMaxCols || !row_ok(a_stride, k) || !row_ok(w_stride, k) ||
        !real_type(out_type) || !row_ok(out_stride, n))
        return ZC_ERR_INVALID_ARG;
    ProductArgs p = {};
    p.e.scale = 1.0f;
    if (epilogue) {
        const zc_epilogue &e = *epilogue;
        if (e.activation > ZC_ACT_SIGMOID || !finite_float(e.scale) || (e.d_bias && !real_type(e.bias_type)) ||
            (e.d_residual && (!real_type(e.residual_type) || !row_ok(e.residual_stride, n))) ||
            (e.d_pre && !row_ok(e.pre_stride, n)))
            return ZC_ERR_INVALID_ARG;
        p.e.bias = e.d_bias;
        p.e.bias_f32 = e.bias_type == ZC_F32;
        p.e.res = e.d_residual;
        p.e.res_f32 = e.residual_type == ZC_F32;
        p.e.res_stride = e.residual_stride;
        p.e.pre = static_cast<uint16_t *>(e.d_pre);
        p.e.pre_stride = e.pre_stride;
        p.e.act = e.activation;
        p.e.scale = e.scale;
    }
    if (!m || !n) return ZC_OK;
    if (!d_out || (k && (!d_a || !d_w))) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_a, 2) || !aligned(d_w, 2) || !typed_aligned(d_out, out_type) || !aligned(d_workspace, 16) ||
        (p.e.bias && !typed_aligned(p.e.bias, epilogue->bias_type)) ||
        (p.e.res && !typed_aligned(p.e.res, epilogue->residual_type)) || !aligned(p.e.pre, 2))
        return ZC_ERR_MISALIGNED;
    p.a = static_cast<const uint16_t *>(d_a);
    p.b = static_cast<const uint16_t *>(d_w);
    p.lda = a_stride;
    p.ldb = w_stride;
    p.e.out = d_out;
    p.e.out_f32 = out_type == ZC_F32;
    p.e.out_stride = out_stride;
    return launch_product(p, m, n, k, false, false, d_workspace, workspace_bytes, stream);
}

extern "C" uint64_t zc_activation_backward_workspace_bytes(uint64_t rows, uint64_t cols) {
    if (rows > kMaxRows || cols > kMaxCols || !rows || !cols) return 0;
    return ceil_div(kSlopeRuns * cols * 4, 256) * 256;
}

extern "C" zc_status zc_activation_backward(const void *d_dout, uint32_t dout_type, uint64_t rows, uint64_t cols,
                                            uint64_t dout_stride, const void *d_pre, uint64_t pre_stride,
                                            uint32_t activation, float scale, void *d_dpre, uint64_t dpre_stride,
                                            float *d_dbias, void *d_workspace, uint64_t workspace_bytes,
                                            void *stream) {
    const bool sloped = activation != ZC_ACT_NONE;
    if (!real_type(dout_type) || rows > kMaxRows || cols > kMaxCols || activation > ZC_ACT_SIGMOID ||
        !finite_float(scale) || !row_ok(dout_stride, cols) || (sloped && !row_ok(pre_stride, cols)) ||
        (d_dpre && !row_ok(dpre_stride, cols)))
        return ZC_ERR_INVALID_ARG;
    if (!cols || (!rows && !d_dbias) || (!d_dpre && !d_dbias)) return ZC_OK;
    if (rows && (!d_dout || (sloped && !d_pre) || (d_dbias && !d_workspace))) return ZC_ERR_INVALID_ARG;
    if (!typed_aligned(d_dout, dout_type) || (sloped && !aligned(d_pre, 2)) || !aligned(d_dpre, 2) || !aligned(d_dbias, 4) ||
        !aligned(d_workspace, 16))
        return ZC_ERR_MISALIGNED;
    if (rows && d_dbias && workspace_bytes < zc_activation_backward_workspace_bytes(rows, cols)) return ZC_ERR_CAPACITY;
    SlopeArgs a = {};
    a.dout = d_dout;
    a.pre = static_cast<const uint16_t *>(d_pre);
    a.dpre = static_cast<uint16_t *>(d_dpre);
    a.parts = d_dbias ? static_cast<float *>(d_workspace) : nullptr;
    a.dout_stride = dout_stride;
    a.pre_stride = pre_stride;
    a.dpre_stride = dpre_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.row_step = (uint32_t)ceil_div(ceil_div(rows, kSlopeRuns), kSWaves) * kSWaves;
    a.act = activation;
    a.dout_f32 = dout_type == ZC_F32;
    a.scale = scale;
    const uint32_t runs = rows ? (uint32_t)ceil_div(rows, a.row_step) : 0;
    Launches on(stream);
    const bool wide = cols % 8 == 0 && aligned(d_dpre, 16) && dpre_stride % 8 == 0;
    if (rows)
        on.launch(wide ? slope_kernel<true> : slope_kernel<false>, dim3((uint32_t)ceil_div(cols, kLanes * 8), runs),
                  dim3(kSWaves * kLanes), a);
    if (d_dbias)
        on.launch(column_sums_kernel, dim3((uint32_t)ceil_div(cols, kLanes)), dim3(kLanes * kRuns), a.parts, runs, a.cols,
                  d_dbias);
    return on.status();
}

extern "C" zc_status zc_matmul_dgrad(const void *d_dpre, uint64_t m, uint64_t n, uint64_t dpre_stride, const void *d_w,
                                     uint64_t k, uint64_t w_stride, const void *d_add, uint32_t add_type,
                                     uint64_t add_stride, void *d_dx, uint32_t dx_type, uint64_t dx_stride,
                                     void *d_workspace, uint64_t workspace_bytes, void *stream) {
    if (m > kMaxRows || n > kMaxCols || k > kMaxCols || !row_ok(dpre_stride, n) || !row_ok(w_stride, k))
        return ZC_ERR_INVALID_ARG;
    ProductArgs p = {};
    p.a = static_cast<const uint16_t *>(d_dpre);
    p.b = static_cast<const uint16_t *>(d_w);
    p.lda = dpre_stride;
    p.ldb = w_stride;
    return gradient(p, m, k, n, false, d_add, add_type, add_stride, d_dx, dx_type, dx_stride, d_workspace,
                    workspace_bytes, stream);
}

extern "C" zc_status zc_matmul_wgrad(const void *d_dpre, uint64_t m, uint64_t n, uint64_t dpre_stride, const void *d_a,
                                     uint64_t k, uint64_t a_stride, const void *d_add, uint32_t add_type,
                                     uint64_t add_stride, void *d_dw, uint32_t dw_type, uint64_t dw_stride,
                                     void *d_workspace, uint64_t workspace_bytes, void *stream) {
    if (m > kMaxRows || n > kMaxCols || k > kMaxCols || !row_ok(dpre_stride, n) || !row_ok(a_stride, k))
        return ZC_ERR_INVALID_ARG;
    ProductArgs p = {};
    p.a = static_cast<const uint16_t *>(d_dpre);
    p.b = static_cast<const uint16_t *>(d_a);
    p.lda = dpre_stride;
    p.ldb = a_stride;
    return gradient(p, n, k, m, true, d_add, add_type, add_stride, d_dw, dw_type, dw_stride, d_workspace,
                    workspace_bytes, stream);
}
