// The token exchange around the experts, MI355X / gfx950: the order of the token
// copies by expert (a stable counting sort), the payload in that order, the
// weighted sum of a token's copies, and its gradients.
#include "zc_moe_device.h"

namespace zc {
namespace moe {

// ---------------------------------------------------------------------------
// plan: stable counting sort of tokens * top_k expert ids
// ---------------------------------------------------------------------------

constexpr uint32_t kPlanThreads = 256;
constexpr uint32_t kPlanWaves = kPlanThreads / kLanes;
constexpr uint32_t kPlanChunk = 1024;      // a block ranks this many copies, or a multiple
constexpr uint32_t kPlanMaxChunks = 256;   // every block reads every chunk's counts: keeps their number bounded
constexpr uint32_t kBins = ZC_MAX_EXPERTS + 1;  // one bin more for dropped copies

struct PlanArgs {
    const int32_t *ids;
    uint32_t *hist;  // [chunks][experts + 1]
    int32_t *offsets, *position, *source;
    uint32_t copies, experts, chunks, per_chunk;
};

__device__ __forceinline__ uint32_t bin_of(const PlanArgs &a, uint32_t i) {
    const int32_t id = a.ids[i];
    return id >= 0 && (uint32_t)id < a.experts ? (uint32_t)id : a.experts;
}

// Copies of every expert in one chunk.
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanArgs a) {
    __shared__ uint32_t bins[kBins];
    for (uint32_t e = threadIdx.x; e <= a.experts; e += kPlanThreads) bins[e] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * a.per_chunk, i1 = min(i0 + a.per_chunk, a.copies);
#pragma unroll 4
    for (uint32_t i = i0 + threadIdx.x; i < i1; i += kPlanThreads) atomicAdd(&bins[bin_of(a, i)], 1u);
    __syncthreads();
    uint32_t *row = a.hist + (uint64_t)blockIdx.x * (a.experts + 1);
    for (uint32_t e = threadIdx.x; e <= a.experts; e += kPlanThreads) row[e] = bins[e];
}

// Ranks a chunk's copies.  A copy's row is the copies of lower experts (a scan
// of the totals), the same expert's copies of earlier chunks, of earlier waves
// of the chunk, and of earlier lanes of its wave: integer counts only, so the
// order is that of the copies.  Bound by the latency of those steps: 65,536
// copies to 256 experts take 9.8 us, and their counts 4.8 before them (both with
// chunks of 2048, whose counts were read one after another: 24 us).  A single chunk
// needs no counts of others.
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanArgs a) {
    __shared__ uint32_t total[kBins + 3];              // copies of an expert in all chunks
    __shared__ uint32_t base[kPlanWaves + 1][kBins + 3];  // a wave's next row of every expert; below: counts of wave w at w + 1
    __shared__ uint32_t part[kPlanWaves];
    const uint32_t tid = threadIdx.x, lane = lane_id(), wave = tid / kLanes, nb = a.experts + 1;
    for (uint32_t e = tid; e < nb; e += kPlanThreads)
#pragma unroll
        for (uint32_t w = 0; w <= kPlanWaves; ++w) base[w][e] = 0;
    __syncthreads();
    const uint32_t per_wave = a.per_chunk / kPlanWaves;
    const uint32_t i0 = min(blockIdx.x * a.per_chunk + wave * per_wave, a.copies), i1 = min(i0 + per_wave, a.copies);
#pragma unroll 4
    for (uint32_t i = i0 + lane; i < i1; i += kLanes) atomicAdd(&base[wave + 1][bin_of(a, i)], 1u);
    if (a.chunks > 1) {
        for (uint32_t e = tid; e < nb; e += kPlanThreads) {
            uint32_t all = 0, before = 0;
#pragma unroll 16
            for (uint32_t c = 0; c < a.chunks; ++c) {
                const uint32_t v = a.hist[(uint64_t)c * nb + e];
                before += c < blockIdx.x ? v : 0u;
                all += v;
            }
            total[e] = all;
            base[0][e] = before;
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (uint32_t e = tid; e < nb; e += kPlanThreads) {
            uint32_t all = 0;
#pragma unroll
            for (uint32_t w = 1; w <= kPlanWaves; ++w) all += base[w][e];
            total[e] = all;
        }
        __syncthreads();
    }
    // copies of lower experts: each thread takes consecutive bins
    const uint32_t per = (nb + kPlanThreads - 1) / kPlanThreads, e0 = tid * per, e1 = min(e0 + per, nb);
    uint32_t mine = 0;
    for (uint32_t e = e0; e < e1; ++e) mine += total[e];
    const uint32_t incl = scan_sum(mine);
    if (lane == kLanes - 1) part[wave] = incl;
    __syncthreads();
    uint32_t run = incl - mine;
    for (uint32_t w = 0; w < wave; ++w) run += part[w];
    for (uint32_t e = e0; e < e1; ++e) {
        uint32_t next = base[0][e] + run;
        if (blockIdx.x == 0) a.offsets[e] = (int32_t)run;  // bin `experts` (dropped copies) ends the last expert's rows
        run += total[e];
        base[0][e] = next;
#pragma unroll
        for (uint32_t w = 1; w < kPlanWaves; ++w) base[w][e] = next += base[w][e];
    }
    __syncthreads();
    uint32_t *next = base[wave];
    const uint32_t bits = 32 - __builtin_clz(a.experts + 1);  // of the largest bin, the one for lanes past the end
    for (uint32_t j = i0; j < i1; j += kLanes) {
        const uint32_t i = j + lane;
        const bool in = i < i1;
        const uint32_t b = in ? bin_of(a, i) : a.experts + 1;
        // lanes of the same bin, one bit of the bin's number at a time
        uint64_t same = ~0ull;
        for (uint32_t bit = 0; bit < bits; ++bit) {
            const uint64_t on = __ballot((b >> bit) & 1u);
            same &= ((b >> bit) & 1u) ? on : ~on;
        }
        const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
        uint32_t p = 0;
        if (in) p = next[b] + rank;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // every lane has read before the counts move on
        if (in && rank == 0) next[b] += (uint32_t)__popcll(same);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (in) {
            const bool dropped = b == a.experts;
            a.position[i] = dropped ? -1 : (int32_t)p;
            if (a.source) a.source[p] = dropped ? -1 : (int32_t)i;
        }
    }
}

// Copies of a chunk: kPlanChunk, or the multiple of it that leaves at most
// kPlanMaxChunks chunks.
static uint32_t per_chunk_of(uint64_t copies) {
    return (uint32_t)(ceil_div(copies, (uint64_t)kPlanChunk * kPlanMaxChunks) * kPlanChunk);
}

__global__ void plan_empty_kernel(int32_t *offsets, uint32_t n) {
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

// ---------------------------------------------------------------------------
// rows of BF16, eight values an access
// ---------------------------------------------------------------------------

constexpr uint32_t kRowThreads = 256;
constexpr uint32_t kRowStep = kRowThreads * 8;
constexpr uint32_t kCopies = 8;  // copies of a token whose rows are on their way at once

__device__ __forceinline__ float value_of(const u32v4 &w, uint32_t i) { return (i & 1) ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]); }

// A row that is read several times (by several blocks, or again for further
// copies) is not marked for single use, as load_values does.
template <bool WIDE>
__device__ __forceinline__ u32v4 load_again(const uint16_t *p, uint32_t n) {
    if (n >= 8) return WIDE ? *reinterpret_cast<const u32v4 *>(p) : *reinterpret_cast<const u32v4a2 *>(p);
    return load_values<WIDE>(p, n);
}
// The copies' rows are written without the mark (with it the gradients of 8192 x
// 8 rows took 1.3 times as long).
template <bool WIDE>
__device__ __forceinline__ void store_row(uint16_t *p, const u32v4 &w, uint32_t n) {
    if (WIDE) {
        if (n >= 8) *reinterpret_cast<u32v4 *>(p) = w;
    } else {
        store_values<false>(p, w, n);
    }
}
__device__ __forceinline__ u32v4 pack_values(const float (&v)[8]) {
    return u32v4{bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7])};
}

struct RowArgs {
    const uint16_t *x;   // dispatch: tokens; combine: the experts' rows
    const uint16_t *dy;  // combine's backward
    const int32_t *position;
    const float *weights;
    uint16_t *out;
    float *dweights;
    uint64_t xs, dys, os;
    uint32_t tokens, top_k, rows, hidden;
};

// The row of copy k of token t, -1 if it has none (uniform).
__device__ __forceinline__ int32_t row_of(const RowArgs &a, uint64_t t, uint32_t k) {
    if (k >= a.top_k) return -1;
    const int32_t p = __builtin_amdgcn_readfirstlane(a.position[t * a.top_k + k]);
    return p >= 0 && (uint32_t)p < a.rows ? p : -1;
}

// The row is read once and written to each of its places.  Block (t, y): the
// y-th 2048 values of the row and every gridDim.y-th after it.  Bound by memory:
// 8192 x 8 rows of 7168 take 205 us, 5.2 TB/s.
template <bool WIDE>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowArgs a) {
    for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const uint16_t *src = a.x + t * a.xs;
        for (uint32_t h = blockIdx.y * kRowStep + threadIdx.x * 8; h < a.hidden; h += gridDim.y * kRowStep) {
            const u32v4 w = load_again<WIDE>(src + h, a.hidden - h);
            for (uint32_t k = 0; k < a.top_k; ++k) {
                const int32_t p = row_of(a, t, k);
                if (p >= 0) store_row<WIDE>(a.out + (uint64_t)p * a.os + h, w, a.hidden - h);
            }
        }
    }
}

// The sums stay in 32 bits, k ascending; eight copies' rows are on their way at
// once, each marked for single use (8192 x 8 rows of 7168: 246 -> 214 us, 4.9 TB/s).
// Blocks as in dispatch_kernel.
template <bool WIDE>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowArgs a) {
    for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        for (uint32_t h = blockIdx.y * kRowStep + threadIdx.x * 8; h < a.hidden; h += gridDim.y * kRowStep) {
            const uint32_t n = a.hidden - h;
            float sum[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) sum[i] = 0.0f;
            for (uint32_t k0 = 0; k0 < a.top_k; k0 += kCopies) {
                u32v4 z[kCopies];
                int32_t p[kCopies];
                float w[kCopies];
#pragma unroll
                for (uint32_t j = 0; j < kCopies; ++j) p[j] = row_of(a, t, k0 + j);
#pragma unroll
                for (uint32_t j = 0; j < kCopies; ++j) {
                    w[j] = p[j] >= 0 && a.weights ? a.weights[t * a.top_k + k0 + j] : 1.0f;
                    if (p[j] >= 0) z[j] = load_values<WIDE>(a.x + (uint64_t)p[j] * a.xs + h, n);
                }
#pragma unroll
                for (uint32_t j = 0; j < kCopies; ++j)
                    if (p[j] >= 0)
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i) sum[i] = fmaf(w[j], value_of(z[j], i), sum[i]);
            }
            store_row<WIDE>(a.out + t * a.os + h, pack_values(sum), n);
        }
    }
}

// One block a token: dz = w dy and the products <dy, z>, each copy's summed over
// the block in an order fixed by the sizes.  Bound by memory: 8192 x 8 rows of
// 7168 take 414 us, 5.1 TB/s.
template <bool WIDE>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowArgs a) {
    __shared__ float part[kRowThreads / kLanes][kCopies];
    const uint32_t lane = lane_id(), wave = threadIdx.x / kLanes;
    for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        for (uint32_t k0 = 0; k0 < a.top_k; k0 += kCopies) {
            int32_t p[kCopies];
            float w[kCopies], dot[kCopies];
#pragma unroll
            for (uint32_t j = 0; j < kCopies; ++j) p[j] = row_of(a, t, k0 + j);
#pragma unroll
            for (uint32_t j = 0; j < kCopies; ++j) {
                w[j] = p[j] >= 0 && a.weights && a.out ? a.weights[t * a.top_k + k0 + j] : 1.0f;
                dot[j] = 0.0f;
            }
            for (uint32_t h = threadIdx.x * 8; h < a.hidden; h += kRowStep) {
                const uint32_t n = a.hidden - h;
                const u32v4 dy = load_again<WIDE>(a.dy + t * a.dys + h, n);
                u32v4 z[kCopies];
                if (a.dweights)
#pragma unroll
                    for (uint32_t j = 0; j < kCopies; ++j)
                        if (p[j] >= 0) z[j] = load_values<WIDE>(a.x + (uint64_t)p[j] * a.xs + h, n);
                if (a.out)
#pragma unroll
                    for (uint32_t j = 0; j < kCopies; ++j)
                        if (p[j] >= 0) {
                            float dz[8];
#pragma unroll
                            for (uint32_t i = 0; i < 8; ++i) dz[i] = w[j] * value_of(dy, i);
                            store_row<WIDE>(a.out + (uint64_t)p[j] * a.os + h, pack_values(dz), n);
                        }
                if (a.dweights)  // values past the end are zeros on both sides
#pragma unroll
                    for (uint32_t j = 0; j < kCopies; ++j)
                        if (p[j] >= 0)
#pragma unroll
                            for (uint32_t i = 0; i < 8; ++i) dot[j] = fmaf(value_of(dy, i), value_of(z[j], i), dot[j]);
            }
            if (!a.dweights) continue;
#pragma unroll
            for (uint32_t j = 0; j < kCopies; ++j) {
                const float d = wave_sum_f(dot[j]);
                if (lane == 0) part[wave][j] = d;
            }
            __syncthreads();
            if (threadIdx.x < kCopies && k0 + threadIdx.x < a.top_k) {
                float s = 0.0f;
#pragma unroll
                for (uint32_t v = 0; v < kRowThreads / kLanes; ++v) s += part[v][threadIdx.x];
                a.dweights[t * a.top_k + k0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

static bool sizes_ok(uint64_t tokens, uint32_t top_k) {
    return top_k >= 1 && top_k <= ZC_MAX_TOP_K && tokens <= kMaxRows && tokens * top_k <= kMaxRows;
}
static bool wide(const void *p, uint64_t stride) { return aligned(p, 16) && stride % 8 == 0; }
static uint32_t token_blocks(uint32_t tokens) { return tokens < (1u << 20) ? tokens : (1u << 20); }
// Blocks of a row of `hidden` values: one for each 2048, so that a few tokens
// spread over the device too, at most 16.
static dim3 row_grid(uint32_t tokens, uint32_t hidden) {
    const uint64_t pieces = ceil_div(hidden, kRowStep);
    return dim3(token_blocks(tokens), (uint32_t)(pieces < 16 ? pieces : 16));
}

}  // namespace moe
}  // namespace zc

using namespace zc::moe;

extern "C" uint64_t zc_dispatch_workspace_bytes(uint64_t tokens, uint32_t top_k, uint32_t experts) {
    if (!sizes_ok(tokens, top_k) || experts == 0 || experts > ZC_MAX_EXPERTS) return 0;
    if (!tokens) return 256;
    const uint64_t chunks = ceil_div(tokens * top_k, per_chunk_of(tokens * top_k));
    return ceil_div(chunks * (experts + 1) * 4, 256) * 256;
}

extern "C" zc_status zc_dispatch_plan(const int32_t *d_ids, uint64_t tokens, uint32_t top_k, uint32_t experts,
                                      void *d_workspace, uint64_t workspace_bytes, int32_t *d_offsets,
                                      int32_t *d_position, int32_t *d_source, void *stream) {
    if (!sizes_ok(tokens, top_k) || experts == 0 || experts > ZC_MAX_EXPERTS || !d_offsets ||
        (tokens && (!d_ids || !d_position || !d_workspace)))
        return ZC_ERR_INVALID_ARG;
    if (!aligned(d_ids, 4) || !aligned(d_offsets, 4) || !aligned(d_position, 4) || !aligned(d_source, 4) ||
        !aligned(d_workspace, 16))
        return ZC_ERR_MISALIGNED;
    if (tokens && workspace_bytes < zc_dispatch_workspace_bytes(tokens, top_k, experts)) return ZC_ERR_CAPACITY;
    Launches on(stream);
    if (!tokens) {
        on.launch(plan_empty_kernel, dim3(1), dim3(256), d_offsets, experts + 1);
        return on.status();
    }
    PlanArgs a = {d_ids, static_cast<uint32_t *>(d_workspace), d_offsets, d_position, d_source,
                  (uint32_t)(tokens * top_k), experts, 0, per_chunk_of(tokens * top_k)};
    a.chunks = (uint32_t)ceil_div(a.copies, a.per_chunk);
    if (a.chunks > 1) on.launch(plan_count_kernel, dim3(a.chunks), dim3(kPlanThreads), a);
    on.launch(plan_place_kernel, dim3(a.chunks), dim3(kPlanThreads), a);
    return on.status();
}

extern "C" zc_status zc_dispatch(const void *d_x, uint64_t tokens, uint64_t hidden, uint64_t x_stride,
                                 const int32_t *d_position, uint32_t top_k, void *d_out, uint64_t rows,
                                 uint64_t out_stride, void *stream) {
    if (!sizes_ok(tokens, top_k) || rows > kMaxRows || hidden > kMaxCols || x_stride < hidden ||
        x_stride > kMaxStride || out_stride < hidden || out_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!tokens || !hidden || !rows) return ZC_OK;
    if (!d_x || !d_position || !d_out) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_x, 2) || !aligned(d_position, 4) || !aligned(d_out, 2)) return ZC_ERR_MISALIGNED;
    RowArgs a = {};
    a.x = static_cast<const uint16_t *>(d_x);
    a.position = d_position;
    a.out = static_cast<uint16_t *>(d_out);
    a.xs = x_stride;
    a.os = out_stride;
    a.tokens = (uint32_t)tokens;
    a.top_k = top_k;
    a.rows = (uint32_t)rows;
    a.hidden = (uint32_t)hidden;
    Launches on(stream);
    const dim3 block(kRowThreads);
    if (hidden % 8 == 0 && wide(d_x, x_stride) && wide(d_out, out_stride))
        on.launch(dispatch_kernel<true>, row_grid(a.tokens, a.hidden), block, a);
    else
        on.launch(dispatch_kernel<false>, row_grid(a.tokens, a.hidden), block, a);
    return on.status();
}

extern "C" zc_status zc_combine(const void *d_z, uint64_t rows, uint64_t hidden, uint64_t z_stride,
                                const int32_t *d_position, const float *d_weights, uint64_t tokens, uint32_t top_k,
                                void *d_y, uint64_t y_stride, void *stream) {
    if (!sizes_ok(tokens, top_k) || rows > kMaxRows || hidden > kMaxCols || z_stride < hidden ||
        z_stride > kMaxStride || y_stride < hidden || y_stride > kMaxStride)
        return ZC_ERR_INVALID_ARG;
    if (!tokens || !hidden) return ZC_OK;
    if ((rows && !d_z) || !d_position || !d_y) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_z, 2) || !aligned(d_position, 4) || !aligned(d_weights, 4) || !aligned(d_y, 2))
        return ZC_ERR_MISALIGNED;
    RowArgs a = {};
    a.x = static_cast<const uint16_t *>(d_z);
    a.position = d_position;
    a.weights = d_weights;
    a.out = static_cast<uint16_t *>(d_y);
    a.xs = z_stride;
    a.os = y_stride;
    a.tokens = (uint32_t)tokens;
    a.top_k = top_k;
    a.rows = (uint32_t)rows;
    a.hidden = (uint32_t)hidden;
    Launches on(stream);
    const dim3 block(kRowThreads);
    if (hidden % 8 == 0 && wide(d_z, z_stride) && wide(d_y, y_stride))
        on.launch(combine_kernel<true>, row_grid(a.tokens, a.hidden), block, a);
    else
        on.launch(combine_kernel<false>, row_grid(a.tokens, a.hidden), block, a);
    return on.status();
}

extern "C" zc_status zc_combine_backward(const void *d_dy, uint64_t dy_stride, const void *d_z, uint64_t rows,
                                         uint64_t hidden, uint64_t z_stride, const int32_t *d_position,
                                         const float *d_weights, uint64_t tokens, uint32_t top_k, void *d_dz,
                                         uint64_t dz_stride, float *d_dweights, void *stream) {
    if (!sizes_ok(tokens, top_k) || rows > kMaxRows || hidden > kMaxCols || dy_stride < hidden ||
        dy_stride > kMaxStride || (d_dweights && (z_stride < hidden || z_stride > kMaxStride)) ||
        (d_dz && (dz_stride < hidden || dz_stride > kMaxStride)))
        return ZC_ERR_INVALID_ARG;
    if (!tokens || (!d_dz && !d_dweights)) return ZC_OK;
    if ((hidden && !d_dy) || !d_position || (d_dweights && rows && hidden && !d_z)) return ZC_ERR_INVALID_ARG;
    if (!aligned(d_dy, 2) || !aligned(d_z, 2) || !aligned(d_position, 4) || !aligned(d_weights, 4) ||
        !aligned(d_dz, 2) || !aligned(d_dweights, 4))
        return ZC_ERR_MISALIGNED;
    RowArgs a = {};
    a.x = static_cast<const uint16_t *>(d_z);
    a.dy = static_cast<const uint16_t *>(d_dy);
    a.position = d_position;
    a.weights = d_weights;
    a.out = static_cast<uint16_t *>(d_dz);
    a.dweights = d_dweights;
    a.xs = z_stride;
    a.dys = dy_stride;
    a.os = dz_stride;
    a.tokens = (uint32_t)tokens;
    a.top_k = top_k;
    a.rows = (uint32_t)rows;
    a.hidden = (uint32_t)hidden;
    Launches on(stream);
    const dim3 grid(token_blocks(a.tokens)), block(kRowThreads);
    if (hidden % 8 == 0 && wide(d_dy, dy_stride) && (!d_dweights || wide(d_z, z_stride)) &&
        (!d_dz || wide(d_dz, dz_stride)))
        on.launch(combine_backward_kernel<true>, grid, block, a);
    else
        on.launch(combine_backward_kernel<false>, grid, block, a);
    return on.status();
}
