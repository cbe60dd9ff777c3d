// Grouped products of 8-bit floating point with a power-of-two scale for each
// block of 128, MI355X / gfx950:
//   forward   out[r, c] = sum over k of A[r, k] B_g[c, k], rows r of group g
//   gradient  out[g, i, j] = sum over the rows r of group g of A[i, r] B[j, r]
// The scaled matrix instructions apply the scales: 2^(a - 127) 2^(b - 127) for
// every lane's 32 values, in the 32-bit sum, at no cost of their own.
#include <type_traits>

#include "zc_lds.h"
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
    uint64_t split_stride;               // elements of one part of a split contraction; gridDim.y parts
};

constexpr uint32_t kMThreads = 256;

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

__device__ __forceinline__ i32v8 join(const u32v4 (&h)[2]) {
    return __builtin_bit_cast(i32v8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int FA, int FB>
__device__ __forceinline__ f32v16 mfma(const i32v8 &a, const i32v8 &b, const f32v16 &c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, FA, FB, 0, (int)sa, 0, (int)sb);
}

// ---------------------------------------------------------------------------
// tiles of four waves, loads straight into LDS
// ---------------------------------------------------------------------------

typedef uint32_t u32v2a2 __attribute__((ext_vector_type(2), aligned(2)));

// A stage is one block of 128 along the contraction: 128 bytes of every row, a
// whole cache line each.  (Stages of 64 bytes, four deep, asked the L2 for twice
// as many half lines and took 1.3 times as long.)  As many as fit 160 KiB of LDS.
template <uint32_t BM, uint32_t BN, uint32_t STAGES>
struct TileShared {
    uint8_t stage[STAGES][(BM + BN) * kBlock];
    uint32_t scale[2][4][2][kLanes];  // four blocks' scale bytes of the rows that a wave loads, of A and of B
    uint32_t touched[4][kLanes];  // what the touches of later blocks bring, never read
};

// BM x BN tile of four waves (2 x 2).  The fragments of half a block are in
// registers while the other half's come out of LDS.  In the middle of a block
// every wave holds the rest of it, and one barrier then frees its buffer for the
// block STAGES after it and hands over the next one.  Between two matrix
// instructions stand a read and a load, so that neither stops them for long.
// T: uint16_t for BF16 results, uint32_t for floats.
//
// Bound by the matrix instructions and the clock that they leave: 65536 x 4096 x
// 7168 in 32 equal groups takes 1450 us, 2650 TFLOP/s, 8192 x 8192 x 8192 392 us,
// 2800; the instructions alone, from registers, reach 3700 at the same power,
// and a 256 x 256 tile spends 1.1 us a block when few are at work (its
// instructions 0.85 at 2.4 GHz) and 1.4 when all are.  About 10 us of a tile are
// its start and its end.  256 x 256 since a row's bytes then serve 256 columns:
// 128 x 128 moves twice the bytes from the L2, at 64 bytes a clock and CU, and
// takes 1.5 times as long.
template <uint32_t BM, uint32_t BN, uint32_t STAGES, bool WGRAD, int FA, int FB, bool FULL, typename T>
__global__ __launch_bounds__(kMThreads, (sizeof(TileShared<BM, BN, STAGES>) > 80 * 1024 ? 1 : 2)) void tile_kernel(MatArgs p) {
    constexpr uint32_t MT = BM / 64, NT = BN / 64;         // 32 x 32 tiles of a wave
    constexpr uint32_t LA = BM / 32, LB = BN / 32;         // 16-byte loads of a wave and block, 8 rows each
    constexpr uint32_t LOADS = LA + LB;
    __shared__ alignas(1024) TileShared<BM, BN, STAGES> sh;
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t ntiles = (p.n + BN - 1) / BN;

    // Consecutive workgroups go to the eight XCDs in turn.  The tiles are walked
    // in bands of eight rows of tiles, column by column: 32 consecutive ones, as many
    // as an XCD has CUs, are 8 x 4 tiles that share rows of A and B in its L2
    // (bands of 4 or 16 took 1.05 and 1.1 times as long).  Forward, an XCD gets one
    // run of tiles, away from the others' rows (runs of 32 in turn: 1.05 times as
    // long); the weight gradient's tiles take longer in groups of many rows, which
    // runs of 32 in turn spread over the XCDs (one run each: 2.1 times as long on
    // groups between 290 and 3500 rows).
    uint32_t nt = 0;
    const auto pick = [&](uint32_t mtiles) -> uint32_t {
        const uint32_t total = mtiles * ntiles, xcd = blockIdx.x % 8, local = blockIdx.x / 8;
        const uint32_t per = total / 8, rest = total % 8;
        const uint32_t id = WGRAD ? (local / 32 * 8 + xcd) * 32 + local % 32 : xcd * per + min(xcd, rest) + local;
        if (id >= total || (!WGRAD && local >= per + (xcd < rest))) return ~0u;
        const uint32_t band = id / (8 * ntiles), in_band = id % (8 * ntiles);
        const uint32_t band_rows = min(8u, mtiles - 8 * band);
        nt = in_band / band_rows;
        return 8 * band + in_band % band_rows;
    };

    uint32_t mt, m0, m1, kb0, kb1;
    const uint8_t *b = p.b, *bs = p.bs;
    uint64_t out0 = 0;
    if (WGRAD) {
        const uint32_t per_group = (p.m + BM - 1) / BM;
        mt = pick(per_group * p.groups);
        if (mt == ~0u) return;
        const Span sp = find_group(p.offsets, p.groups, p.rows, mt / per_group);
        m0 = (mt % per_group) * BM;
        m1 = p.m;
        kb0 = sp.blocks0;
        kb1 = kb0 + (sp.end - sp.begin + kBlock - 1) / kBlock;
        out0 = (uint64_t)sp.group * p.out_group;
    } else {
        const Span sp = find_tile(p.offsets, p.groups, p.rows, BM, [&](uint32_t total) { return mt = pick(total); });
        if (!sp.found) return;
        m0 = sp.begin + sp.tile * BM;
        m1 = sp.end;
        kb0 = (uint32_t)((uint64_t)p.blocks * blockIdx.y / gridDim.y);
        kb1 = (uint32_t)((uint64_t)p.blocks * (blockIdx.y + 1) / gridDim.y);
        b += sp.group * p.b_group;
        bs += sp.group * p.bs_group;
        out0 = blockIdx.y * p.split_stride;
    }
    const uint32_t n0 = nt * BN;
    const uint32_t blocks = kb1 - kb0;

    f32v16 acc[MT][NT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const uint32_t wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * (BN / 2);
    if (blocks) {
        // where the lane's loads start: row lane / 8 of 8, and the 16-byte chunk that its place in LDS holds.  Chunk c of
        // row r sits at c ^ (r / 2 mod 8): sixteen lanes read 256 bytes at a time, and the same chunk of sixteen rows then
        // lies in sixteen different columns of banks (with r mod 8 every read took twice its four cycles).  Rows past
        // the end repeat the last one (their results are not stored)
        const uint32_t chunk = 16 * ((lane & 7u) ^ (lane / 16));
        const uint8_t *ga = p.a + (uint64_t)m0 * p.lda + (uint64_t)kb0 * kBlock;
        const uint8_t *gb = b + (uint64_t)n0 * p.ldb + (uint64_t)kb0 * kBlock;
        uint32_t offa[LA], offb[LB];
#pragma unroll
        for (uint32_t i = 0; i < LA; ++i)
            offa[i] = min(wave * (BM / 4) + 8 * i + lane / 8, m1 - 1 - m0) * (uint32_t)p.lda + (chunk ^ (64 * (i & 1)));
#pragma unroll
        for (uint32_t i = 0; i < LB; ++i)
            offb[i] = min(wave * (BN / 4) + 8 * i + lane / 8, p.n - 1 - n0) * (uint32_t)p.ldb + (chunk ^ (64 * (i & 1)));
        const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)&sh.stage[0][0]);
        const uint32_t ldsa = lds0 + wave * (BM / 4) * kBlock;
        const uint32_t ldsb = lds0 + BM * kBlock + wave * (BN / 4) * kBlock;
        constexpr uint32_t kStageStep = (BM + BN) * kBlock;

        // scales: four blocks of a row are a dword; rows of the wave: BM / 4 of A, BN / 4 of B, one a lane (the
        // lanes past them repeat the last, in places of their own: a condition would be a branch in the loop)
        const uint8_t *sa0 = p.as + (uint64_t)m0 * p.ldas;
        const uint8_t *sb0 = bs + (uint64_t)(n0 >> p.b_shift) * p.ldbs;
        const uint32_t sra = wave * (BM / 4) + min(lane, BM / 4 - 1), srb = wave * (BN / 4) + min(lane, BN / 4 - 1);
        const uint32_t soffa = min(sra, m1 - 1 - m0) * (uint32_t)p.ldas;
        const uint32_t soffb = ((min(n0 + srb, p.n - 1) >> p.b_shift) - (n0 >> p.b_shift)) * (uint32_t)p.ldbs;
        const uint32_t ldss = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)&sh.scale[0][0]);
        const auto load_scales = [&](uint32_t c) {  // blocks 4c .. 4c + 3
            const uint32_t at = ldss + ((c & 1) * 4 + wave) * 2 * kLanes * 4;
            lds_load4(sa0 + 4 * c, soffa, at);
            lds_load4(sb0 + 4 * c, soffb, at + kLanes * 4);
        };
        // A touch brings one line per row of a later block into the L2: a quarter of A's rows and an eighth of B's, since
        // the four and eight tiles beside this one that share them touch the others.  Three blocks ahead: 3 % of the
        // time where the operands come from HBM (65536 x 4096 x 7168, 32 groups), nothing where they do not.
        const uint32_t part = wave < 2 ? (nt & 3) * (BM / 4) + wave * (BM / 8) : (mt & 7) * (BN / 8) + (wave - 2) * (BN / 16);
        const uint32_t touch_row = part + min(lane, (wave < 2 ? BM / 8 : BN / 16) - 1);
        const uint32_t touch_off = wave < 2 ? min(touch_row, m1 - 1 - m0) * (uint32_t)p.lda
                                            : min(touch_row, p.n - 1 - n0) * (uint32_t)p.ldb;
        const uint8_t *const touch_base = wave < 2 ? ga : gb;
        const uint32_t ldst = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)&sh.touched[wave][0]);
        const auto touch = [&](uint32_t t) { lds_load4(touch_base + (uint64_t)min(t, blocks - 1) * kBlock, touch_off, ldst); };
        const auto load_piece = [&](uint32_t t, uint32_t at, uint32_t i) {  // the wave's i-th load of block kb0 + t
            if (i < LA)
                lds_load16(ga + (uint64_t)t * kBlock, offa[i % LA], ldsa + at + i * 1024);
            else
                lds_load16(gb + (uint64_t)t * kBlock, offb[(i - LA) % LB], ldsb + at + (i - LA) * 1024);
        };

        // fragments: lane l holds row l mod 32, of the half block's four chunks l / 32 and l / 32 + 2 (the order along the
        // contraction does not matter as long as A and B agree)
        const uint32_t fr = lane % 32, fc = lane / 32, sw = fr / 2 & 7u;
        const uint32_t ra0 = (wm + fr) * kBlock, rb0 = (BM + wn + fr) * kBlock;
        u32v4 fa[2][MT][2], fb[2][NT][2];  // [half of the block]
        uint32_t ea[MT], eb[NT];
        const uint8_t *const stages = &sh.stage[0][0];
        const auto read_a = [&](uint32_t at, uint32_t half, uint32_t i, uint32_t h) -> u32v4 {
            return *reinterpret_cast<const u32v4 *>(
                stages + (at + ra0 + 32 * i * kBlock + 16 * ((4 * half + 2 * h + fc) ^ sw)));
        };
        const auto read_b = [&](uint32_t at, uint32_t half, uint32_t j, uint32_t h) -> u32v4 {
            return *reinterpret_cast<const u32v4 *>(
                stages + (at + rb0 + 32 * j * kBlock + 16 * ((4 * half + 2 * h + fc) ^ sw)));
        };
        // the q-th of the 2 (MT + NT) reads of a half
        constexpr uint32_t kReads = 2 * (MT + NT);
        const auto read_piece = [&](uint32_t at, uint32_t half, uint32_t q) {
            if (q < 2 * MT)
                fa[half][q / 2 % MT][q & 1] = read_a(at, half, q / 2 % MT, q & 1);
            else
                fb[half][(q / 2 - MT) % NT][q & 1] = read_b(at, half, (q / 2 - MT) % NT, q & 1);
        };
        uint32_t wa4[MT], wb4[NT];  // four blocks' scales of the lane's rows
        const auto read_scales = [&](uint32_t kb) {
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) {
                const uint32_t r = wm + 32 * i + fr;
                wa4[i] = sh.scale[kb / 4 & 1][r / (BM / 4)][0][r % (BM / 4)];
            }
#pragma unroll
            for (uint32_t j = 0; j < NT; ++j) {
                const uint32_t r = wn + 32 * j + fr;
                wb4[j] = sh.scale[kb / 4 & 1][r / (BN / 4)][1][r % (BN / 4)];
            }
        };
        const auto take_scales = [&](uint32_t kb) {  // block kb's in the low byte
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) ea[i] = wa4[i] >> (8 * (kb & 3));
#pragma unroll
            for (uint32_t j = 0; j < NT; ++j) eb[j] = wb4[j] >> (8 * (kb & 3));
        };

        const uint32_t chunk0 = kb0 / 4, chunk_last = (kb1 - 1) / 4;
        load_scales(chunk0);
        if (chunk0 < chunk_last) load_scales(chunk0 + 1);
#pragma unroll
        for (uint32_t t = 0; t < STAGES; ++t)
            if (t < blocks)
#pragma unroll
                for (uint32_t i = 0; i < LOADS; ++i) load_piece(t, t * kStageStep, i);
        if (blocks >= STAGES)
            wait_and_meet<(int)((STAGES - 1) * LOADS)>();
        else
            wait_and_meet<0>();
        touch(STAGES);
        read_scales(kb0);
        take_scales(kb0);
#pragma unroll
        for (uint32_t q = 0; q < kReads; ++q) read_piece(0, 0, q);

        uint32_t at0 = 0, at1 = kStageStep;  // where blocks t and t + 1 are
        // one block; MORE: there is a block to load into its place
        const auto step = [&](uint32_t t, auto more) {
            constexpr bool MORE = decltype(more)::value;
            // younger than block t + 1 are at least the loads of the STAGES - 2 blocks after it and one touch
            constexpr int kYounger = MORE ? 1 + (int)((STAGES - 2) * LOADS) : 0;
            const uint32_t kb = kb0 + t;
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {
                if (half == 1) {
                    // block t + 1 has landed, and every wave holds the rest of block t
                    wait_and_meet<kYounger>();
                    // the next four blocks' scales, again with every block (the same bytes): a branch here would
                    // let the compiler move the matrix instructions behind it, away from the loads they hide
                    if (MORE) load_scales(min(kb / 4 + 1, chunk_last));
                }
                bf16v8 wb[FULL ? NT : 1][4];
                if (FULL)
#pragma unroll
                    for (uint32_t j = 0; j < NT; ++j) widen<FB>(join(fb[half][j]), eb[j] & 0xFFu, wb[j % (FULL ? NT : 1)]);
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i) {
                    bf16v8 wa[4];
                    if (FULL) widen<FA>(join(fa[half][i]), ea[i] & 0xFFu, wa);
#pragma unroll
                    for (uint32_t j = 0; j < NT; ++j) {
                        if (FULL) {
#pragma unroll
                            for (uint32_t q = 0; q < 4; ++q)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j % (FULL ? NT : 1)][q], wa[q],
                                                                                   acc[i][j], 0, 0, 0);
                        } else {
                            // B in the place of the left matrix: a lane then holds four consecutive columns of one row
                            acc[i][j] = mfma<FB, FA>(join(fb[half][j]), join(fa[half][i]), acc[i][j], eb[j], ea[i]);
                        }
                        // between the matrix instructions: the reads of the other half, and the loads of block t + STAGES
                        constexpr uint32_t kSlots = MT * NT;
                        const uint32_t slot = i * NT + j;
                        if (MORE && half == 1)
#pragma unroll
                            for (uint32_t q = slot * LOADS / kSlots; q < (slot + 1) * LOADS / kSlots; ++q)
                                load_piece(t + STAGES, at0, q);
#pragma unroll
                        for (uint32_t q = slot * kReads / kSlots; q < (slot + 1) * kReads / kSlots; ++q)
                            read_piece(half ? at1 : at0, half ^ 1, q);
                        if (half == 1 && slot + 1 == kSlots) {
                            read_scales(kb + 1);
                            touch(t + STAGES + 1);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            take_scales(kb + 1);
            at0 = at1;
            at1 = at1 == (STAGES - 1) * kStageStep ? 0 : at1 + kStageStep;
        };
        uint32_t t = 0;
        for (; t + STAGES < blocks; ++t) step(t, std::true_type{});
        for (; t < blocks; ++t) step(t, std::false_type{});
    }

    // Results through LDS, 64 (or 32) rows of a wave at a time, so that a row's BN / 2
    // columns leave as whole lines.
    wait_and_meet<0>();
    uint8_t *const room = reinterpret_cast<uint8_t *>(&sh);
    constexpr uint32_t es = sizeof(T), row_bytes = BN / 2 * es + 16, chunks = BN / 2 * es / 16, per = 16 / es;
    constexpr uint32_t tiles = sizeof(sh) >= 4 * 64 * row_bytes ? 2 : 1, rounds = MT / tiles, rows = 32 * tiles;
    static_assert(sizeof(sh) >= 4 * rows * row_bytes, "room for a round of every wave");
    uint8_t *mine = room + wave * rows * row_bytes;
    T *out = static_cast<T *>(p.out) + out0;
    typedef std::conditional_t<es == 2, u32v4a2, u32v4a4> Line;  // 16 bytes at any element
#pragma unroll
    for (uint32_t round = 0; round < rounds; ++round) {
#pragma unroll
        for (uint32_t i = 0; i < tiles; ++i)
#pragma unroll
            for (uint32_t j = 0; j < NT; ++j)
#pragma unroll
                for (uint32_t e = 0; e < 16; e += 4) {
                    const f32v16 &v = acc[round * tiles + i][j];
                    uint8_t *w = mine + (32 * i + lane % 32) * row_bytes + (32 * j + 2 * e + 4 * (lane / 32)) * es;
                    if (es == 2)
                        *reinterpret_cast<u32v2 *>(w) = u32v2{bf_pack(v[e], v[e + 1]), bf_pack(v[e + 2], v[e + 3])};
                    else
                        *reinterpret_cast<u32v4 *>(w) = u32v4{__float_as_uint(v[e]), __float_as_uint(v[e + 1]),
                                                              __float_as_uint(v[e + 2]), __float_as_uint(v[e + 3])};
                }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        // a row's chunks go to consecutive lanes
        constexpr uint32_t step = kLanes / chunks;
        static_assert(kLanes % chunks == 0, "whole rows a step");
        const uint32_t cc = lane % chunks, c = n0 + wn + cc * per;
        uint32_t r = m0 + wm + round * rows + lane / chunks;
        const uint8_t *from = mine + (lane / chunks) * row_bytes + cc * 16;
        T *o = out + (uint64_t)r * p.ldo + c;
        const bool whole = c + per <= p.n;
#pragma unroll 4
        for (uint32_t q = 0; q < rows / step; ++q, r += step, from += step * row_bytes, o += step * p.ldo) {
            const u32v4 v = *reinterpret_cast<const u32v4 *>(from);
            if (r < m1 && c < p.n) {
                if (whole) {
                    *reinterpret_cast<Line *>(o) = v;
                } else {
                    for (uint32_t k = 0; k < per && c + k < p.n; ++k)
                        o[k] = (T)(v[k * es / 4] >> (8 * es * k % 32));
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Four results of a row, of which n exist.
template <typename T>
__device__ __forceinline__ void store4(T *o, float a, float b, float c, float d, uint32_t n) {
    if constexpr (sizeof(T) == 2) {
        const u32v2 w = {bf_pack(a, b), bf_pack(c, d)};
        if (n >= 4) {
            *reinterpret_cast<u32v2a2 *>(o) = w;
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 3; ++j)
                if (j < n) o[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    } else {
        const u32v4 w = {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
        if (n >= 4) {
            *reinterpret_cast<u32v4a4 *>(o) = w;
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 3; ++j)
                if (j < n) o[j] = w[j];
        }
    }
}

// The parts of a split contraction, added in order.
template <typename T>
__global__ __launch_bounds__(256) void add_parts_kernel(const float *parts, uint32_t splits, uint64_t stride, T *out,
                                                        uint32_t m, uint32_t n, uint64_t ldo, const int32_t *offsets,
                                                        uint32_t groups) {
    // rows of no group have no parts and are left as they are
    const uint32_t lo = offsets ? clamp_row(offsets[0], m) : 0u;
    uint32_t hi = m;
    if (offsets) {
        uint32_t high = lo;
        for (uint32_t g = lane_id(); g <= groups; g += kLanes) high = max(high, clamp_row(offsets[g], m));
        hi = last_lane(scan_max(high));
    }
    const uint32_t per_row = (n + 3) / 4;
    const uint64_t all = (uint64_t)(hi - lo) * per_row;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (uint64_t)gridDim.x * 256) {
        const uint64_t r = lo + i / per_row;
        const uint32_t c = (uint32_t)(i % per_row) * 4;
        const float *src = parts + r * n + c;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t k = min(n - c, 4u);
        if (k == 4 && n % 4 == 0) {
            for (uint32_t s = 0; s < splits; ++s) {
                const u32v4 w = *reinterpret_cast<const u32v4 *>(src + s * stride);
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) v[j] += __uint_as_float(w[j]);
            }
        } else {
            for (uint32_t s = 0; s < splits; ++s)
                for (uint32_t j = 0; j < k; ++j) v[j] += src[s * stride + j];
        }
        store4(out + r * ldo + c, v[0], v[1], v[2], v[3], k);
    }
}

// ---------------------------------------------------------------------------
// few rows: bound by reading the weights
// ---------------------------------------------------------------------------

typedef float f32v4 __attribute__((ext_vector_type(4)));

// 16 rows of B against 16 MT rows of A.  The waves of a block take the blocks of
// the contraction in turn, STEP at a time, straight from memory into the
// registers of the matrix instructions (a row's 64 bytes by four lanes), and add
// their sums through LDS.  Values are widened to BF16 with their scale, so the
// products are exact; the conversions take a fraction of the time of the loads.
template <uint32_t MT, uint32_t WAVES, uint32_t STEP, int FA, int FB, typename T>
__global__ __launch_bounds__(WAVES * 64) void rows_kernel(MatArgs p) {
    __shared__ f32v4 part[WAVES][MT][kLanes];
    const uint32_t lane = lane_id(), wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t ntiles = (p.n + 15) / 16, nt = blockIdx.x % ntiles, mt = blockIdx.x / ntiles;
    const Span sp = find_tile(p.offsets, p.groups, p.rows, 16 * MT, [&](uint32_t) { return mt; });
    if (!sp.found) return;
    const uint32_t m0 = sp.begin + sp.tile * 16 * MT, m1 = sp.end, n0 = nt * 16;
    const uint32_t fr = lane % 16, fc = 16 * (lane / 16);
    const uint8_t *b = p.b + sp.group * p.b_group + (uint64_t)min(n0 + fr, p.n - 1) * p.ldb + fc;
    const uint8_t *bs = p.bs + sp.group * p.bs_group + (uint64_t)(n0 >> p.b_shift) * p.ldbs;
    const uint8_t *a[MT], *as[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
        const uint64_t r = min(m0 + 16 * i + fr, m1 - 1);
        a[i] = p.a + r * p.lda + fc;
        as[i] = p.as + r * p.ldas;
    }
    f32v4 acc[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) acc[i] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t kb = wave * STEP; kb < p.blocks; kb += WAVES * STEP) {
        // STEP blocks: their scales are bytes of one dword
        const uint32_t sb = *reinterpret_cast<const uint32_t *>(bs + (kb & ~3u)) >> (8 * (kb & 3));
        u32v4 fb[STEP][2], fa[STEP][MT][2];
        uint32_t sa[MT];
#pragma unroll
        for (uint32_t u = 0; u < STEP; ++u) {
            const uint64_t at = (uint64_t)min(kb + u, p.blocks - 1) * kBlock;
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                fb[u][h] = *reinterpret_cast<const u32v4 *>(b + at + 64 * h);
#pragma unroll
                for (uint32_t i = 0; i < MT; ++i) fa[u][i][h] = *reinterpret_cast<const u32v4 *>(a[i] + at + 64 * h);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < MT; ++i) sa[i] = *reinterpret_cast<const uint32_t *>(as[i] + (kb & ~3u)) >> (8 * (kb & 3));
#pragma unroll
        for (uint32_t u = 0; u < STEP; ++u) {
            if (kb + u >= p.blocks) break;
            bf16v8 wb[4];
            widen<FB>(join(fb[u]), (sb >> (8 * u)) & 0xFFu, wb);
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) {
                bf16v8 wa[4];
                widen<FA>(join(fa[u][i]), (sa[i] >> (8 * u)) & 0xFFu, wa);
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], wa[q], acc[i], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (uint32_t i = wave; i < MT; i += WAVES) {
        f32v4 v = part[0][i][lane];
#pragma unroll
        for (uint32_t w = 1; w < WAVES; ++w) v += part[w][i][lane];
        // a lane holds four consecutive columns of one row
        const uint32_t r = m0 + 16 * i + fr, c = n0 + 4 * (lane / 16);
        if (r < m1) {
            store4(static_cast<T *>(p.out) + (uint64_t)r * p.ldo + c, v[0], v[1], v[2], v[3], c < p.n ? p.n - c : 0u);
        }
    }
}

// ---------------------------------------------------------------------------
// which kernel
// ---------------------------------------------------------------------------

// kTile128: two workgroups on a CU, two stages each; kTile128Deep: one, three stages.
enum Shape { kTile128, kTile128Deep, kTile256x128, kTile256 };

template <bool WGRAD, int FA, int FB, typename T>
static void launch_tile(const MatArgs &p, bool full, Shape shape, dim3 grid, Launches &on) {
    const dim3 block(kMThreads);
    if (full)
        on.launch((tile_kernel<128, 128, 2, WGRAD, FA, FB, true, T>), grid, block, p);
    else if (shape == kTile256)
        on.launch((tile_kernel<256, 256, 2, WGRAD, FA, FB, false, T>), grid, block, p);
    else if (!WGRAD && shape == kTile256x128)
        on.launch((tile_kernel<256, 128, 3, WGRAD, FA, FB, false, T>), grid, block, p);
    else if (!WGRAD && shape == kTile128Deep)
        on.launch((tile_kernel<128, 128, 3, WGRAD, FA, FB, false, T>), grid, block, p);
    else
        on.launch((tile_kernel<128, 128, 2, WGRAD, FA, FB, false, T>), grid, block, p);
}

template <int FA, int FB, typename T>
static void launch_rows(const MatArgs &p, uint32_t mt, dim3 grid, Launches &on) {
    if (mt == 1)
        on.launch((rows_kernel<1, 8, 4, FA, FB, T>), grid, dim3(512), p);
    else
        on.launch((rows_kernel<2, 8, 4, FA, FB, T>), grid, dim3(512), p);
}

// Upper bound of the tiles of `tile` rows over all groups.
static uint64_t row_tiles(uint64_t rows, uint64_t groups, uint64_t tile) {
    return rows / tile + (rows < groups ? rows : groups);
}

struct Choice {
    uint32_t rows_mt;  // > 0: rows_kernel with this many 16-row tiles
    Shape shape;
    uint32_t splits;
};

// Few rows a group: rows_kernel.  At n = 4096, k = 7168 it takes 6.9 us for 1 row
// (tiles 12.2), 8.8 for 16 (13.7), 12.7 for 32 (14.9), 19.6 for 64 (16.0); with 8
// groups of 1 row 34 (57), of 16 rows 53 (58), with 32 groups of 16 rows 236 (200).
// Else the shape with the least time by this model: a round of workgroups over the
// 256 CUs takes, for each block of the contraction, 1.2 us with tiles of 256 x 256,
// 0.85 with 256 x 128, 0.55 with 128 x 128 alone on a CU, and 1.1 with two of those
// on it, and 4 to 9 us for its start and end.  With few tiles of 128 x 128 the
// contraction is split, at the cost of writing and adding the parts (4 us and
// their bytes).  Groups are taken to have equally many rows.
//
// The model orders the shapes; its times are rough (512 x 4096 x 7168: 67, 45, 29
// and 40 us measured, 76, 54, 35 and 66 by the model; 4096 x 4096 x 7168: 92, 117,
// 137 and 122, and 76, 107, 139 and 131).  Every shape was timed at 17 to 2048 rows (powers
// of two, and 17 and 33), n = 512, 2048, 4096, 8192 and k = 512, 2048, 7168, 16384,
// one group, weights from memory, calls back to back: of those 128 products the
// choice is within 5 % of the fastest shape in 97 and within 20 % in 114.  The
// others, up to 1.7 times the fastest: 33 to 128 rows with k = 2048 or n = 512,
// where rows_kernel takes 7 to 9 us and a split 11 to 13 (its second launch), and
// 17 rows with k = 16384, where a split takes 15 to 17 and rows_kernel 20 to 21.
static Choice choose(uint64_t m, uint64_t n, uint64_t k, uint64_t groups, bool full) {
    Choice c = {0, kTile128, 1};
    const uint64_t used = m < groups ? m : groups, per_group = used ? ceil_div(m, used) : 0;
    const bool launchable = row_tiles(m, groups, 16) * ceil_div(n, 16) < (1u << 22);
    if (launchable && (per_group <= 12 || (used == 1 && per_group <= 32))) {
        c.rows_mt = per_group <= 16 ? 1 : 2;
        return c;
    }
    const double blocks = (double)ceil_div(k, kBlock);
    const auto tiles = [&](uint64_t tm, uint64_t tn) { return used * ceil_div(per_group, tm) * ceil_div(n, tn); };
    const auto time = [](uint64_t t, uint64_t at_once, double us) { return (double)ceil_div(t, at_once) * us; };
    const uint64_t t128 = tiles(128, 128);
    double best = time(t128, 512, 1.1 * blocks + 4.0);
    const auto offer = [&](Shape shape, uint32_t splits, double us) {
        if (us < best) {
            best = us;
            c.shape = shape;
            c.splits = splits;
        }
    };
    if (!full) {
        offer(kTile256, 1, time(tiles(256, 256), 256, 1.2 * blocks + 9.0));
        offer(kTile256x128, 1, time(tiles(256, 128), 256, 0.85 * blocks + 6.0));
        offer(kTile128Deep, 1, time(t128, 256, 0.55 * blocks + 4.0));
    }
    for (uint32_t s = 2; s <= 8; s *= 2) {
        const uint64_t bytes = m * n * 4 * s;
        if (bytes > ZC_FP8_MATMUL_WORKSPACE_MAX || blocks < 4 * s) break;
        const double add = 4.0 + 2.0 * (double)bytes / 4.0e6;
        if (full)
            offer(kTile128, s, time(t128 * s, 512, 1.1 * blocks / s + 4.0) + add);
        else
            offer(kTile128Deep, s, time(t128 * s, 256, 0.55 * blocks / s + 4.0) + add);
    }
    return c;
}

template <int FA, int FB>
static void launch_forward(MatArgs p, bool bf16, bool full, const Choice &c, float *ws, dim3 grid, Launches &on) {
    if (c.rows_mt) {
        if (bf16)
            launch_rows<FA, FB, uint16_t>(p, c.rows_mt, grid, on);
        else
            launch_rows<FA, FB, uint32_t>(p, c.rows_mt, grid, on);
        return;
    }
    if (c.splits == 1) {
        if (bf16)
            launch_tile<false, FA, FB, uint16_t>(p, full, c.shape, grid, on);
        else
            launch_tile<false, FA, FB, uint32_t>(p, full, c.shape, grid, on);
        return;
    }
    void *out = p.out;
    const uint64_t ldo = p.ldo;
    p.out = ws;
    p.ldo = p.n;
    p.split_stride = (uint64_t)p.rows * p.n;
    grid.y = c.splits;
    launch_tile<false, FA, FB, uint32_t>(p, full, c.shape, grid, on);
    const uint64_t units = ceil_div((uint64_t)p.rows * ceil_div(p.n, 4), 256);
    const dim3 add((uint32_t)(units < 4096 ? units : 4096));
    if (bf16)
        on.launch(add_parts_kernel<uint16_t>, add, dim3(256), ws, c.splits, p.split_stride, static_cast<uint16_t *>(out),
                  p.rows, p.n, ldo, p.offsets, p.groups);
    else
        on.launch(add_parts_kernel<uint32_t>, add, dim3(256), ws, c.splits, p.split_stride, static_cast<uint32_t *>(out),
                  p.rows, p.n, ldo, p.offsets, p.groups);
}

static zc_status launch_forward(const MatArgs &p, uint32_t ta, uint32_t tb, bool bf16, bool full, Choice c, float *ws,
                                Launches &on) {
    if (!ws) c.splits = 1;
    const uint64_t tm = c.rows_mt ? 16 * c.rows_mt : c.shape == kTile128 || c.shape == kTile128Deep ? 128 : 256;
    const uint64_t tn = c.rows_mt ? 16 : c.shape == kTile256 ? 256 : 128;
    const uint64_t tiles = row_tiles(p.rows, p.groups, tm) * ceil_div(p.n, tn);
    const uint32_t threads = c.rows_mt ? 512 : kMThreads;
    if (tiles > 0xFFFFFFFFull / threads - 256) return ZC_ERR_INVALID_ARG;
    const dim3 grid((uint32_t)(c.rows_mt ? tiles : ceil_div(tiles, 8) * 8));
    const int fa = ta == ZC_FP8_E5M2, fb = tb == ZC_FP8_E5M2;
    if (!fa && !fb) launch_forward<0, 0>(p, bf16, full, c, ws, grid, on);
    if (!fa && fb) launch_forward<0, 1>(p, bf16, full, c, ws, grid, on);
    if (fa && !fb) launch_forward<1, 0>(p, bf16, full, c, ws, grid, on);
    if (fa && fb) launch_forward<1, 1>(p, bf16, full, c, ws, grid, on);
    return on.status();
}

template <int FA, int FB>
static void launch_wgrad(const MatArgs &p, bool bf16, bool full, Shape shape, dim3 grid, Launches &on) {
    if (bf16)
        launch_tile<true, FA, FB, uint16_t>(p, full, shape, grid, on);
    else
        launch_tile<true, FA, FB, uint32_t>(p, full, shape, grid, on);
}

static zc_status launch_wgrad(const MatArgs &p, uint32_t ta, uint32_t tb, bool bf16, bool full, Launches &on) {
    const uint64_t t256 = ceil_div(p.m, 256) * ceil_div(p.n, 256) * p.groups;
    const Shape shape = !full && t256 >= 192 ? kTile256 : kTile128;
    const uint64_t tiles = shape == kTile256 ? t256 : ceil_div(p.m, 128) * ceil_div(p.n, 128) * p.groups;
    if (tiles > 0xFFFF00u) return ZC_ERR_INVALID_ARG;
    const dim3 grid((uint32_t)ceil_div(tiles, 256) * 256);
    const int fa = ta == ZC_FP8_E5M2, fb = tb == ZC_FP8_E5M2;
    if (!fa && !fb) launch_wgrad<0, 0>(p, bf16, full, shape, grid, on);
    if (!fa && fb) launch_wgrad<0, 1>(p, bf16, full, shape, grid, on);
    if (fa && !fb) launch_wgrad<1, 0>(p, bf16, full, shape, grid, on);
    if (fa && fb) launch_wgrad<1, 1>(p, bf16, full, shape, grid, on);
    return on.status();
}

// A tile's rows are reached by 32-bit offsets from its first: 256 rows of at most 2^24 bytes.
constexpr uint64_t kMaxContraction = 1ull << 24;

static bool types_ok(uint32_t ta, uint32_t tb, uint32_t to, uint32_t sum) {
    return is_fp8(ta) && is_fp8(tb) && (to == ZC_F32 || to == ZC_BF16) && sum <= ZC_FP8_SUM_FULL;
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_fp8_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, uint32_t groups) {
    if (m > kMaxRows || n > kMaxCols || k > kMaxContraction || groups == 0 || groups > ZC_MAX_EXPERTS || !m || !n) return 0;
    uint64_t most = 0;
    for (int full = 0; full < 2; ++full) {
        const Choice c = choose(m, n, k, groups, full != 0);
        if (c.splits > 1 && m * n * 4 * c.splits > most) most = m * n * 4 * c.splits;
    }
    return most;
}

extern "C" zc_status zc_fp8_matmul(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t m,
                                   const void *d_b, const uint8_t *d_b_scales, uint32_t b_type, uint64_t n,
                                   uint64_t k, uint32_t groups, const int32_t *d_offsets, void *d_out,
                                   uint32_t out_type, uint64_t out_stride, uint32_t sum_mode,
                                   void *d_workspace, uint64_t workspace_bytes, void *stream) {
    if (!types_ok(a_type, b_type, out_type, sum_mode) || m > kMaxRows || n > kMaxCols || k > kMaxContraction || groups == 0 ||
        groups > ZC_MAX_EXPERTS || (!d_offsets && groups != 1) || out_stride < n || out_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!m || !n) return ZC_OK;
    if (!d_out || (k && (!d_a || !d_a_scales || !d_b || !d_b_scales))) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_a, 16) || !aligned(d_a_scales, 4) || !aligned(d_b, 16) || !aligned(d_b_scales, 4) ||
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
    const bool full = sum_mode == ZC_FP8_SUM_FULL;
    const Choice c = choose(m, n, k, groups, full);
    const bool room = d_workspace && workspace_bytes >= zc_fp8_matmul_workspace_bytes(m, n, k, groups);
    Launches on(stream);
    return launch_forward(p, a_type, b_type, out_type == ZC_BF16, full, c,
                          room ? static_cast<float *>(d_workspace) : nullptr, on);
}

extern "C" zc_status zc_fp8_matmul_wgrad(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t n,
                                         const void *d_b, const uint8_t *d_b_scales, uint32_t b_type, uint64_t k,
                                         uint64_t padded_rows, uint64_t rows, uint32_t groups,
                                         const int32_t *d_offsets, void *d_out, uint32_t out_type,
                                         uint32_t sum_mode, void *stream) {
    if (!types_ok(a_type, b_type, out_type, sum_mode) || rows > kMaxRows || n > kMaxCols || k > kMaxCols || groups == 0 ||
        groups > ZC_MAX_EXPERTS || (!d_offsets && groups != 1) || padded_rows % kBlock ||
        padded_rows > kMaxContraction)
        return ZC_ERR_INVALID_ARG;
    if (padded_rows < zc_fp8_padded_rows(rows, groups)) return ZC_ERR_CAPACITY;
    if (!n || !k) return ZC_OK;
    if (!d_out || (rows && (!d_a || !d_a_scales || !d_b || !d_b_scales))) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_a, 16) || !aligned(d_a_scales, 4) || !aligned(d_b, 16) || !aligned(d_b_scales, 4) ||
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
    Launches on(stream);
    return launch_wgrad(p, a_type, b_type, out_type == ZC_BF16, sum_mode == ZC_FP8_SUM_FULL, on);
}
