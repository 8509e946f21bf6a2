// attend.cu -- attention of one new token per request over the paged entries
// of an MLA or SWA layer, for sm_103a.
//
// Mathematics. The query's heads share one entry k_t per token, whose first V
// values are also the value: x_ht = c q_h . k_t, out_h = sum_t p_ht k_t[:V]
// with p the softmax of x over t. One pass over the cache keeps, per head, a
// reference m and the sums l = sum 2^(x - m), O = sum 2^(x - m) k[:V] (x in
// units of log 2); parts of a cache are joined by scaling them to one m.
//
// Every token's entry is read from HBM once and used for two products per
// head, so with H heads a byte of a 16-bit cache carries about 2 H operations
// (576 values, 512 of them the value): 60 at 32 heads, 121 at 64. The copy
// rate allows 270 per byte at the dense tensor rate, so the call is bound by
// HBM, and the tensor cores have to run beside the loads. CUDA cores cannot
// (6.3 ms for 32 requests of 8192 tokens; the copy rate's floor is 45 us).
//
// Split. The cache is cut into tiles of up to 64 tokens of one page; all
// requests' tiles in a row are shared out evenly over the CTAs (one per SM),
// whatever the lengths, so a CTA works through a run of segments (request,
// tiles). A request inside one CTA is finished there; one that spans several
// leaves its (m, l, O) per CTA in the workspace and a second kernel joins
// them. (Caches of a few tiles each are not split.) Above 64 heads, groups of
// heads take CTAs of their own, side by side.
//
// A CTA: a loader brings the tile's entries to shared memory (panels of 64
// values, 128-byte swizzle), one warp issues the products on the tensor cores,
// eight warps do the softmax.
//   S [64 heads x 64 tokens]   = Q . K^T    (A = Q, B = the tile, both with
//                                            the summed axis contiguous)
//   O^T [V values x heads]    += V^T . P^T  (A = the same tile read along its
//                                            values, B = P)
// The second product is taken transposed so that its 128 rows are values, of
// which there are always enough, and its columns the heads, of which there may
// be few: O^T takes V/128 x heads columns of tensor memory, and no row of the
// tensor cores idles however few heads there are. P goes through shared memory
// as bf16 or f16 (the entries' type; f16 for an fp8 cache): the only rounding
// below 32 bits on the way, at most half a step of p (2^-8 bf16, 2^-11 f16)
// per token. l is summed from p before it is rounded. The reference m only
// moves when a logit exceeds it by 8, so O is rarely rescaled; p is at most 2^8
// then, or, as f16, 2^15: there it is lifted by 2^7, so that the many small
// weights of a long cache stay above f16's smallest values.
//
// Entries of 16 bits come by TMA: a tensor map over (values, page rows,
// blocks) needs no address arithmetic, and rows past a page's end read as
// zero. fp8 entries are loaded to registers, widened to f16 (exact) and stored
// to the same panels; q is brought to f16 with a power of two per head.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "follow.cuh"
#include "lmc_internal.h"
#include "tensor.cuh"

namespace {

using namespace lmc;

constexpr int kMaxEntry = 576;
constexpr int kMaxValue = 512;
constexpr int kTile = 64;             // tokens per tile
constexpr int kMaxHeads = 64;         // heads per CTA
constexpr int kPanel = kTile * 128;   // bytes of 64 values of a tile's rows
constexpr int kMaxStages = 4;
constexpr int kMaxCols = 160;         // CTAs along the cache's length (an SM each)
constexpr int kSoftWarps = 8;
constexpr int kScoreWarp = 8;          // issues S = Q K^T
constexpr int kValueWarp = 9;          // issues O^T += V^T P^T
constexpr int kAheadWarp = 10;         // sends tiles to come on to L2
constexpr int kLoaderWarp = 11;        // 16-bit entries: one warp
constexpr int kFirstFp8Loader = 12;    // fp8: eight, two whole warpgroups
constexpr int kFp8Loaders = 8;        // warps, eight of a tile's rows each
// Tiles sent on to L2 before their copy is issued. Measured at 32 x 8192 tokens
// and at 256 windows of 4096: none 66.8 / 177 us, one 62.4 / 165, two 63.5 /
// 166, three 67.5 / 177, five 81 / 224 (they are gone again when they are
// wanted).
constexpr int kAhead = 1;
constexpr int kNap = 300;             // ns between looks at the loaders' progress (100: the same, 800: 63.8 / 169 us)
constexpr int kEarlyPanels = 5;       // of an fp8 tile, widened before its stage is free (3: 1 us more, 6: 6, 7: 11 of 122)
// Registers per thread of an fp8 CTA's warpgroups: 2 x 80 + 56 + 2 x 128 of the
// 5 x 96 it starts with (fewer for the softmax or the loaders spill).
constexpr int kSoftRegisters = 80, kIssueRegisters = 56, kLoadRegisters = 128;
template <bool kFp8>
constexpr int kThreads = (kFp8 ? kFirstFp8Loader + kFp8Loaders : kLoaderWarp + 1) * 32;
constexpr float kLag = 8.0f;          // how far (log2) a logit may exceed the reference
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kSmemLimit = 227 * 1024;

// Shared memory that is not a tile: barriers and per-head numbers.
struct Control {
    uint64_t q_full, q_free;
    uint64_t q_raw;              // fp8: queries as they came
    uint64_t kv_full[kMaxStages], kv_free[kMaxStages];
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, pv_done, o_free;
    uint64_t valid[2 * kMaxStages];  // a tile's rows that are attended
    uint64_t zero[2 * kMaxStages];   // and those to be cleared before they are values
    uint32_t tmem;
    uint32_t gave_up;            // a wait ran out: nothing waits any more
    uint64_t ended[2];           // all of an issuing warp's products, after that
    uint32_t tiles, segments;    // that the loaders asked for
    int32_t loading;             // the tile whose load was issued last
    float factor[kMaxHeads];     // rescaling of a head's O
    float half[2][kMaxHeads];    // a head's maximum or sum in each half of the tokens
    alignas(16) float inverse[kMaxHeads];  // 1 / l
    float q_scale[kMaxHeads];    // fp8: what q was divided by
};

struct AttendPlan {
    CUtensorMap cache;  // 16-bit entries
    CUtensorMap query;
    const uint8_t *pool;  // fp8: the layer's block 0
    int64_t block_stride;
    int64_t num_blocks;
    const int32_t *table;
    int64_t row_stride;
    const int32_t *lengths;
    const uint16_t *q;
    int64_t q_request_stride, q_head_stride;
    uint16_t *out;
    int64_t out_request_stride, out_head_stride;
    float *lse;  // caller's, or NULL
    int64_t lse_request_stride;
    float *weights;  // caller's, or NULL
    int64_t weights_request_stride;
    // workspace
    int4 *segment;   // [2 cols]: (request, tiles here, all its tiles, 0) a CTA left unfinished, or (-1, ..)
    float2 *part_ml; // [2 cols][H]
    float *part_o;   // [2 cols][H][V]
    float *lse2;     // [R][H], log2
    float *logits;   // [R][H][logit_stride], log2, or NULL
    int64_t logit_stride;
    uint32_t *status;
    int32_t R, H, E, V;
    int32_t max_length;        // the caller's, and what the table holds
    int32_t window;            // 0: none
    int32_t block_size;        // N
    int32_t token_bytes;
    int32_t pages_per_tile;    // > 1 where several pages fit a tile
    int32_t span;              // tokens of a page, or of a tile's pages
    int32_t tiles_per_span;
    uint32_t span_inverse, tiles_inverse;  // see quotient()
    int32_t cols;              // CTAs along the length
    uint32_t cols_inverse;
    int32_t whole;             // > 0: a CTA has as many requests to itself; nothing is joined
    int32_t brief;             // the stream's next kernel, another call's, may be brought in at once
    int32_t head_groups, group_heads;  // heads of a CTA
    int32_t padded_heads;      // rounded up to 16
    int32_t panels;            // of an entry in shared memory
    int32_t value_tiles;       // of 128 values
    int32_t stages;
    int32_t cache_copies, query_copies;  // TMA copies for all panels of a box
    int32_t q_bf16;            // q's and out's type
    float scale;               // of fp8 entries
    float log2_scale;          // softmax_scale * scale * log2(e)
};

// ---- requests and tiles ----------------------------------------------------

struct Range {
    int lo, L;  // tokens [lo, L)
    bool ok;    // a length that can be served
};

__device__ __forceinline__ Range range_for(const AttendPlan &P, int length) {
    Range g;
    g.L = length;
    g.ok = g.L >= 0 && g.L <= P.max_length;
    g.lo = P.window > 0 ? max(0, g.L - P.window) : 0;
    return g;
}

// n / d for 0 <= n < 2^31 by m = floor(2^32 / d) (2^32 - 1 for d = 1): the
// product's upper half is the quotient or one less.
__device__ __forceinline__ int quotient(int n, int d, uint32_t m) {
    const int q = (int)__umulhi((uint32_t)n, m);
    return q + (n - q * d >= d ? 1 : 0);
}

__device__ __forceinline__ int tile_of(const AttendPlan &P, int t) {
    const int s = quotient(t, P.span, P.span_inverse);
    return s * P.tiles_per_span + (t - s * P.span) / kTile;
}

__device__ __forceinline__ Range range_of(const AttendPlan &P, int r) { return range_for(P, __ldca(P.lengths + r)); }

__device__ __forceinline__ int tiles_of(const AttendPlan &P, const Range &g) {
    return !g.ok || g.L == 0 ? 0 : tile_of(P, g.L - 1) + 1 - tile_of(P, g.lo);
}

// A CTA's run of segments. Each warp walks it on its own: 32 requests at a
// time, a lane each. (All requests' tiles together number less than 2^31.)
struct Walk {
    int pos, end;     // the CTA's tiles still to come, of all requests' in a row
    int length;       // this lane's request's,
    int start, stop;  // and its tiles
    int r0;           // the first of the 32 requests at hand

    // the current segment
    int r, first, count;  // request, its first tile here (of the request's), tiles
    int tiles;            // the request's
    bool begins, ends;    // the request begins / ends in this CTA
    Range range;

    __device__ __forceinline__ void load(const AttendPlan &P, int base) {
        const int lane = threadIdx.x & 31;
        length = r0 + lane < P.R ? __ldca(P.lengths + r0 + lane) : 0;
        const int n = tiles_of(P, range_for(P, length));
        int sum = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o)
                sum += x;
        }
        stop = base + sum;
        start = stop - n;
    }

    template <bool kFp8>
    __device__ __forceinline__ void init(const AttendPlan &P, int col) {
        r0 = 0;
        load(P, 0);
        if (P.whole > 0) {  // requests [a, b), none of them shared
            const int a = col * P.whole, b = min(a + P.whole, P.R);
            if (b <= 32) {
                pos = __shfl_sync(0xffffffffu, start, a);
                end = __shfl_sync(0xffffffffu, stop, b - 1);
                return;
            }
            int before = 0, here = 0;
            // (by __ldca a register of the fp8 kernel spills, 120.4 -> 121.0 us for
            // 4 x 131072 tokens; by a plain load the other takes 64.5 instead of
            // 63.2 for 32 x 8192)
            for (int i = threadIdx.x & 31; i < b; i += 32)
                (i < a ? before : here) += tiles_of(P, kFp8 ? range_for(P, P.lengths[i]) : range_of(P, i));
            pos = __reduce_add_sync(0xffffffffu, before);
            end = pos + __reduce_add_sync(0xffffffffu, here);
            return;
        }
        int total = 0;
        for (int i = 32 + (threadIdx.x & 31); i < P.R; i += 32)
            total += tiles_of(P, range_of(P, i));
        total = __reduce_add_sync(0xffffffffu, total) + __shfl_sync(0xffffffffu, stop, 31);
        // equal shares, so only the last CTAs may have none (in 64 bits: a
        // share times a CTA's number may pass the total)
        const int64_t each = quotient(total + P.cols - 1, P.cols, P.cols_inverse);
        pos = (int)min(col * each, (int64_t)total);
        end = (int)min(pos + each, (int64_t)total);
    }

    __device__ __forceinline__ bool next(const AttendPlan &P) {
        if (pos >= end)
            return false;
        uint32_t here;
        while ((here = __ballot_sync(0xffffffffu, start <= pos && pos < stop)) == 0) {
            r0 += 32;
            if (r0 >= P.R)
                return false;  // the lengths changed under the call
            load(P, __shfl_sync(0xffffffffu, stop, 31));
        }
        const int k = __ffs(here) - 1;
        const int s = __shfl_sync(0xffffffffu, start, k), e = __shfl_sync(0xffffffffu, stop, k);
        r = r0 + k;
        range = range_for(P, __shfl_sync(0xffffffffu, length, k));
        begins = s == pos;
        ends = e <= end;
        first = pos - s + tile_of(P, range.lo);
        count = min(e, end) - pos;
        tiles = e - s;
        pos += count;
        return true;
    }
};

// A tile's tokens: [t0, t0 + rows) of one page, or of pages_per_tile pages.
struct Tile {
    int t0, rows, page, row0;
};

__device__ __forceinline__ Tile tile_at(const AttendPlan &P, int tile) {
    Tile T;
    const int s = quotient(tile, P.tiles_per_span, P.tiles_inverse);
    T.row0 = (tile - s * P.tiles_per_span) * kTile;
    T.t0 = s * P.span + T.row0;
    T.rows = min(kTile, P.span - T.row0);
    T.page = s * P.pages_per_tile;
    return T;
}

__device__ __forceinline__ uint64_t bits(int lo, int hi) {  // [lo, hi) of 64
    lo = max(lo, 0);
    hi = min(hi, 64);
    if (hi <= lo)
        return 0;
    return (hi - lo == 64 ? ~0ull : ((1ull << (hi - lo)) - 1)) << lo;
}

// ---- barriers, tensor cores ------------------------------------------------

// Waits for a phase. When the limit runs out the CTA gives up as a whole: no
// later wait waits, every warp runs its loops to their end (so that the
// barriers among threads stay matched) and the status word says so.
__device__ __forceinline__ void bar_wait(Control &C, uint64_t *bar, uint32_t parity, uint32_t *status) {
    if (bar_try(bar, parity))
        return;
    for (uint32_t k = 0; k < kWaitLimit; k++) {
        if (bar_try(bar, parity))
            return;
        if ((k & 255u) == 255u && *(volatile uint32_t *)&C.gave_up)
            return;
    }
    *(volatile uint32_t *)&C.gave_up = 1;
    atomicOr(status, LMC_ST_TIMEOUT);
}

// Whether the CTA has given up, the same for the whole warp. Copies are only
// asked for where it has not: an earlier one of the same barrier may still run.
__device__ __forceinline__ bool gone(Control &C) {
    return __any_sync(0xffffffffu, *(volatile uint32_t *)&C.gave_up != 0);
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// o[k] for a k known at run time, without an indexed (local memory) array.
__device__ __forceinline__ uint32_t at16(const uint32_t (&o)[16], int k) {
    uint32_t x = o[0];
#pragma unroll
    for (int i = 1; i < 16; i++)
        x = k == i ? o[i] : x;
    return x;
}

// ---- the CTA's roles ---------------------------------------------------------

struct Memory {
    uint8_t *q, *kv, *p;
    int stage_bytes;
};

// The page a warp resolved last: the tiles of a page follow one another, and
// the block table's latency would be paid for each.
struct LastPage {
    int r = -1, page = -1, block = -1;
};

// The block ids of a tile's pages, one per lane, and which rows they and the
// range leave: a bad page's status bit is raised here.
__device__ __forceinline__ int resolve(const AttendPlan &P, const Walk &W, const Tile &T, uint64_t &valid, uint32_t &bad,
                                       LastPage &last) {
    const int lane = threadIdx.x & 31;
    valid = bits(W.range.lo - T.t0, min(T.rows, W.range.L - T.t0));
    if (P.pages_per_tile == 1) {
        if (W.r != last.r || T.page != last.page) {
            int block = P.table[W.r * P.row_stride + T.page];
            if (block < 0 || block >= P.num_blocks) {
                bad |= block == -1 ? LMC_ST_NO_BLOCK : LMC_ST_BLOCK_OOR;
                block = -1;
            }
            last.r = W.r;
            last.page = T.page;
            last.block = block;
        }
        if (last.block < 0)
            valid = 0;
        return last.block;
    }
    int block = -1;
    const int64_t p0 = ((int64_t)T.page + lane) * P.block_size;  // the page's tokens
    if (lane < P.pages_per_tile && p0 < W.range.L && p0 + P.block_size > W.range.lo) {
        block = P.table[W.r * P.row_stride + T.page + lane];
        if (block < 0 || block >= P.num_blocks) {
            bad |= block == -1 ? LMC_ST_NO_BLOCK : LMC_ST_BLOCK_OOR;
            block = -1;
        }
    }
    const uint32_t pages = __ballot_sync(0xffffffffu, block >= 0);
    uint64_t have = 0;
    for (int k = 0; k < P.pages_per_tile; k++)
        if (pages >> k & 1)
            have |= bits(k * P.block_size, (k + 1) * P.block_size);
    valid &= have;
    return block;
}

// One warp: queries and 16-bit entries by TMA.
__device__ __forceinline__ void load_by_tma(const AttendPlan &P, Control &C, const Memory &M, Walk &W, int group) {
    const int lane = threadIdx.x & 31;
    uint32_t bad = 0, n = 0, segments = 0;
    LastPage last;
    auto end = [&] {
        if (bad)
            atomicOr(P.status, bad);
        if (lane == 0) {
            C.tiles = n;
            C.segments = segments;
        }
    };
    while (W.next(P)) {
        const int row_panels = (P.E + 63) / 64;
        for (int j = 0; j < W.count; j++, n++) {
            const int st = (int)uniform(n % P.stages);
            const Tile T = tile_at(P, W.first + j);
            uint64_t valid;
            const int block = resolve(P, W, T, valid, bad, last);
            // pages there are: one held by every lane, or one per lane
            const uint32_t pages = __ballot_sync(0xffffffffu, block >= 0) & (P.pages_per_tile == 1 ? 1u : ~0u);
            const int row0 = (int)uniform(T.row0);
            uint8_t *to = M.kv + (size_t)st * M.stage_bytes;
            const uint32_t bytes =
                uniform(__popc(pages) * row_panels * (P.pages_per_tile == 1 ? kTile : P.block_size) * 128);
            if (lane == 0) {
                // rows behind a page's end are filled with zeros, others hold what lies there
                C.valid[n % (2 * kMaxStages)] = valid;
                C.zero[n % (2 * kMaxStages)] =
                    ~valid & (P.pages_per_tile == 1 && pages != 0 ? bits(0, T.rows) : ~0ull);
            }
            const int block0 = (int)uniform(block);
            if (n >= (uint32_t)P.stages)
                bar_wait(C, &C.kv_free[st], (n / P.stages - 1) & 1, P.status);
            if (gone(C))
                return end();
            if (P.pages_per_tile == 1) {
                if (elect()) {
                    bar_expect(&C.kv_full[st], bytes);
                    if (block0 >= 0)
                        for (int i = 0; i < P.cache_copies; i++)
                            tma_box(&P.cache, to + i * kPanel, i * 64, row0, block0, &C.kv_full[st]);
                }
            } else {
                if (elect())
                    bar_expect(&C.kv_full[st], bytes);
                for (int k = 0; k < P.pages_per_tile; k++) {
                    const int b = (int)__shfl_sync(0xffffffffu, block, k);
                    if (b >= 0 && elect())
                        for (int i = 0; i < P.cache_copies; i++)
                            tma_box(&P.cache, to + i * kPanel + k * P.block_size * 128, i * 64, 0, b, &C.kv_full[st]);
                }
            }
            __syncwarp();
            if (lane == 0)
                *(volatile int32_t *)&C.loading = (int)n;
            if (j == 0) {  // the queries second: their place is free later than the first tile's
                const int r = (int)uniform(W.r);
                if (segments > 0)
                    bar_wait(C, &C.q_free, (segments - 1) & 1, P.status);
                if (gone(C)) {
                    n++;
                    return end();
                }
                if (elect()) {
                    bar_expect(&C.q_full, (uint32_t)(row_panels * P.padded_heads * 128));
                    for (int i = 0; i < P.query_copies; i++)
                        tma_box(&P.query, M.q + i * P.padded_heads * 128, i * 64, group * P.group_heads, r, &C.q_full);
                }
                __syncwarp();
                segments++;
            }
        }
    }
    end();
}

// Queries to f16 where they lie in shared memory, each head's times a power of
// two that brings its largest value to [2^14, 2^15): exact for values within
// 2^27 of it. Eight warps, four rows at a time each, eight lanes to a row.
// (Read from global memory instead, at this point all CTAs ask for the same
// few lines: 24,000 cycles a segment.)
__device__ __forceinline__ void query_to_f16(const AttendPlan &P, Control &C, const Memory &M, int warp) {
    const int lane = threadIdx.x & 31, piece = lane & 7, pieces = P.E / 8;
#pragma unroll 1
    for (int h = warp * 4 + lane / 8; h < P.padded_heads; h += 4 * kFp8Loaders) {
        // padded_heads is a multiple of 16, so a warp's lanes are here together
        uint8_t *const row = M.q + h * 128;
        const int panel = P.padded_heads * 128, x = h & 7;
        float top = 0.0f;
#pragma unroll 3
        for (int c = piece; c < pieces; c += 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + (c >> 3) * panel + ((piece ^ x) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; k++)
                top = fmaxf(top, fmaxf(fabsf(from_q(w[k] & 0xffff, P.q_bf16)), fabsf(from_q(w[k] >> 16, P.q_bf16))));
        }
        for (int o = 4; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^e with e = 14 - floor(log2(top)), at least -113. 2^126 and its
        // inverse are the last that normal floats hold: every bf16 is a multiple
        // of 2^-133, so times that f16 holds it as it is. Beside an infinity
        // (e = -114) all finite values stay finite: what is lost of them does
        // not show in logits that are infinite. 1 where all are zero
        const int exponent = (int)(__float_as_uint(top) >> 23) - 127;
        const int e = top == 0.0f ? 0 : min(126, 14 - exponent);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        if (piece == 0)
            C.q_scale[h] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 3
        for (int c = piece; c < pieces; c += 8) {
            uint4 *const at = reinterpret_cast<uint4 *>(row + (c >> 3) * panel + ((piece ^ x) << 4));
            const uint4 v = *at;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; k++)
                o[k] = pack<false>(from_q(w[k] & 0xffff, P.q_bf16) * up, from_q(w[k] >> 16, P.q_bf16) * up);
            *at = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Eight warps: queries and fp8 entries, widened to f16 on the way. A warp
// holds eight of a tile's rows, four lanes to a row: a lane takes 16 codes of
// each panel, so a panel's codes are read as 64-byte pieces and its two
// 16-byte halves are stored without bank conflicts, at offsets that do not
// change from tile to tile. Half of a tile is widened in registers before its
// stage is free, while the next one's codes come from L2 into the registers
// that this frees; the other half goes through registers only after that (all
// of it widened early takes 72 registers more, and the softmax pays for them).
__device__ __forceinline__ void load_fp8(const AttendPlan &P, Control &C, const Memory &M, Walk &W, int group) {
    constexpr int kPanels = kMaxEntry / 64;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kFirstFp8Loader;
    const int row = warp * 8 + lane / 4, piece = lane & 3;
    const int chunks = P.E / 16;  // of an entry
    const uint32_t at0 = row * 128 + (((2 * piece) ^ (row & 7)) << 4), at1 = row * 128 + (((2 * piece + 1) ^ (row & 7)) << 4);
    uint32_t bad = 0, n = 0, segments = 0;
    constexpr int kEarly = kEarlyPanels;
    uint4 codes[kPanels];
    uint32_t wide[kEarly][8];
    uint64_t valid = 0, next_valid = 0;
    const uint8_t *src = nullptr;  // the next tile's codes
    LastPage last;
    const int my_page = P.pages_per_tile == 1 ? 0 : row / P.block_size;
    const int my_row = row - my_page * P.block_size;

    Tile T;
    auto find = [&](int j) {
        if (j > 0 && T.row0 + 2 * kTile <= P.span && T.t0 + 2 * kTile <= W.range.L && last.block >= 0) {
            // most often: a whole tile behind another of the same page
            T.row0 += kTile;
            T.t0 += kTile;
            src += kTile * P.token_bytes;
            next_valid = ~0ull;
        } else {
            T = tile_at(P, W.first + j);
            const int block = resolve(P, W, T, next_valid, bad, last);
            const int64_t b = __shfl_sync(0xffffffffu, block, my_page & 31);
            src = P.pool + b * P.block_stride + (int64_t)(T.row0 + my_row) * P.token_bytes + piece * 16;
        }
        if (warp == 0 && lane == 0)
            *(volatile int32_t *)&C.loading = (int)n + (j > 0);
    };
    auto load = [&](int i) {
        codes[i] = make_uint4(0, 0, 0, 0);
        if ((next_valid >> row & 1) && i * 4 + piece < chunks)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(codes[i].x), "=r"(codes[i].y), "=r"(codes[i].z), "=r"(codes[i].w)
                         : "l"(src + i * 64));
    };
    auto widen = [&](uint32_t(&o)[8], const uint4 &c) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 8; k++)
            asm volatile("cvt.rn.f16x2.e4m3x2 %0, %1;"
                         : "=r"(o[k])
                         : "h"((unsigned short)(w[k >> 1] >> (16 * (k & 1)))));
    };
    auto put = [&](uint8_t *to, int i, const uint32_t(&o)[8]) {
        if (i * 4 + piece < chunks) {
            *reinterpret_cast<uint4 *>(to + i * kPanel + at0) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(to + i * kPanel + at1) = make_uint4(o[4], o[5], o[6], o[7]);
        }
    };

    auto end = [&] {
        if (bad)
            atomicOr(P.status, bad);
        if (warp == 0 && lane == 0)
            C.segments = segments;
    };
    while (W.next(P)) {
        // a turn stores tile j and loads tile j + 1
#pragma unroll 1
        for (int j = -1; j < W.count; j++) {
            const bool store = j >= 0, more = j + 1 < W.count;
            valid = next_valid;
            if (store)
#pragma unroll
                for (int i = 0; i < kEarly; i++)
                    widen(wide[i], codes[i]);
            if (more) {
                find(j + 1);
#pragma unroll
                for (int i = 0; i < kEarly; i++)
                    load(i);
            }
            if (store) {
                const int st = n % P.stages;
                if (n >= (uint32_t)P.stages)
                    bar_wait(C, &C.kv_free[st], (n / P.stages - 1) & 1, P.status);
                uint8_t *to = M.kv + (size_t)st * M.stage_bytes;
#pragma unroll
                for (int i = 0; i < kEarly; i++)
                    put(to, i, wide[i]);
#pragma unroll
                for (int i = kEarly; i < kPanels; i++) {
                    widen(wide[i - kEarly], codes[i]);
                    put(to, i, wide[i - kEarly]);
                }
                if (warp == 0 && lane == 0) {
                    C.valid[n % (2 * kMaxStages)] = valid;
                    C.zero[n % (2 * kMaxStages)] = 0;  // the rows left out hold zeros
                }
                fence_async();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&C.kv_full[st]);
                n++;
            }
            if (more)  // behind the arrival, which the fence would hold up until they are there
#pragma unroll
                for (int i = kEarly; i < kPanels; i++)
                    load(i);
            if (!store) {  // the queries, while the first tile is on its way
                const int r = (int)uniform(W.r);
                if (segments > 0)
                    bar_wait(C, &C.q_free, (segments - 1) & 1, P.status);
                if (gone(C))
                    return end();
                if (warp == 0 && elect()) {
                    bar_expect(&C.q_raw, (uint32_t)((P.E + 63) / 64 * P.padded_heads * 128));
                    for (int i = 0; i < P.query_copies; i++)
                        tma_box(&P.query, M.q + i * P.padded_heads * 128, i * 64, group * P.group_heads, r, &C.q_raw);
                }
                __syncwarp();
                bar_wait(C, &C.q_raw, segments & 1, P.status);
                segments++;
                query_to_f16(P, C, M, warp);
                fence_async();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&C.q_full);
            }
        }
    }
    end();
}

// A CTA that gave up, all its roles ended: what it left running ends (or the
// limit runs out) before its memory goes to another. The two warps that issue
// products commit all of theirs once more; the third waits for the copies.
__device__ __forceinline__ void outlast(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitLimit && !bar_try(bar, parity); i++) {
    }
}

template <bool kFp8>
__device__ void wind_up(const AttendPlan &P, Control &C, int warp) {
    if (warp == kScoreWarp || warp == kValueWarp) {
        uint64_t *const done = &C.ended[warp - kScoreWarp];
        if (elect())
            commit(done);
        __syncwarp();
        outlast(done, 0);
    } else if (warp == kAheadWarp) {
        if (!kFp8)
            for (uint32_t k = C.tiles > (uint32_t)P.stages ? C.tiles - P.stages : 0; k < C.tiles; k++)
                outlast(&C.kv_full[k % P.stages], (k / P.stages) & 1);
        if (C.segments > 0)
            outlast(kFp8 ? &C.q_raw : &C.q_full, (C.segments - 1) & 1);
    }
}

// One warp: sends tiles on to L2, kAhead of them before they are loaded (the
// two stages hold too little to cover the latency of HBM), over the ends of
// requests too. A page's rows are one run of bytes. It goes by the loaders'
// progress, but nothing waits for it.
__device__ __forceinline__ void send_ahead(const AttendPlan &P, Control &C, Walk &W) {
    uint32_t unused = 0;  // bad pages are raised when they are loaded
    uint64_t valid;
    LastPage last;
    int n = 0;
    while (W.next(P))
        for (int j = 0; j < W.count; j++, n++) {
            if (n < P.stages)
                continue;  // loaded at once
            for (uint32_t k = 0; k < kWaitLimit; k++) {
                if ((int)uniform(*(volatile uint32_t *)&C.loading) >= n - kAhead)
                    break;
                if (uniform(*(volatile uint32_t *)&C.gave_up))
                    return;
                __nanosleep(kNap);
            }
            const Tile T = tile_at(P, W.first + j);
            const int block = resolve(P, W, T, valid, unused, last);
            const int rows = P.pages_per_tile == 1 ? T.rows : P.block_size;
            const bool mine = (threadIdx.x & 31) < P.pages_per_tile;
            if (mine && block >= 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 P.pool + (int64_t)block * P.block_stride + (int64_t)T.row0 * P.token_bytes),
                             "r"(rows * P.token_bytes)
                             : "memory");
            __syncwarp();
        }
}

// One warp: S = Q K^T of each tile, as soon as it is there. (The two products
// are issued by two warps, so that neither waits behind the other's barriers.)
template <bool kBf16>
__device__ __forceinline__ void multiply_scores(const AttendPlan &P, Control &C, const Memory &M, Walk &W) {
    const uint32_t tmem = uniform(C.tmem);
    const uint32_t qk = instruction(kBf16, false, 64, kTile);
    // descriptors hold addresses in units of 16 bytes: steps are added to them
    const uint64_t q0 = matrix(smem_addr(M.q), 16, 1024);
    const uint32_t q_panel = P.padded_heads * 128 >> 4;
    const int steps = P.E / 16, panels = steps / 4;
    uint32_t n = 0, segments = 0;
    while (W.next(P)) {
        bar_wait(C, &C.q_full, segments & 1, P.status);
        for (int j = 0; j < W.count; j++, n++) {
            const int st = (int)uniform(n % P.stages);
            const uint32_t d = tmem + uniform(n & 1) * 64;
            const uint64_t k0 = matrix(smem_addr(M.kv) + st * M.stage_bytes, 16, 1024);
            if (n >= 2)
                bar_wait(C, &C.s_free[n & 1], (n / 2 - 1) & 1, P.status);
            bar_wait(C, &C.kv_full[st], (n / P.stages) & 1, P.status);
            __syncwarp();
            fence_after();
            if (elect()) {
                for (int i = 0; i < panels; i++)
#pragma unroll
                    for (int s = 0; s < 4; s++)
                        mma(d, q0 + i * q_panel + s * (32 >> 4), k0 + i * (kPanel >> 4) + s * (32 >> 4), qk, i + s > 0);
                for (int s = 4 * panels; s < steps; s++)
                    mma(d, q0 + panels * q_panel + (s & 3) * (32 >> 4), k0 + panels * (kPanel >> 4) + (s & 3) * (32 >> 4),
                        qk, s > 0);
                commit(&C.s_full[n & 1]);
                if (j == W.count - 1)
                    commit(&C.q_free);
            }
            __syncwarp();
        }
        segments++;
    }
}

// One warp: O^T += V^T P^T of each tile, once its P is written.
template <bool kBf16>
__device__ __forceinline__ void multiply_values(const AttendPlan &P, Control &C, const Memory &M, Walk &W) {
    const uint32_t o = uniform(C.tmem) + 128;
    const uint32_t pv = instruction(kBf16, true, 128, P.padded_heads);
    const uint64_t p0 = matrix(smem_addr(M.p), 16, 1024);
    uint32_t n = 0, segments = 0;
    while (W.next(P)) {
        for (int j = 0; j < W.count; j++, n++) {
            const int st = (int)uniform(n % P.stages);
            const uint64_t v0 = matrix(smem_addr(M.kv) + st * M.stage_bytes, kPanel, 1024);
            if (j == 0 && segments > 0)
                bar_wait(C, &C.o_free, (segments - 1) & 1, P.status);
            bar_wait(C, &C.p_full, n & 1, P.status);
            __syncwarp();
            fence_after();
            if (elect()) {
#pragma unroll
                for (int t = 0; t < kMaxValue / 128; t++)
                    if (t < P.value_tiles) {
#pragma unroll
                        for (int s = 0; s < kTile / 16; s++)
                            mma(o + t * P.padded_heads, v0 + t * (2 * kPanel >> 4) + s * (2048 >> 4), p0 + s * (32 >> 4),
                                pv, j > 0 || s > 0);
                    }
                commit(&C.kv_free[st]);
                commit(&C.pv_done);
            }
            __syncwarp();
        }
        segments++;
    }
}

// One value of up to 16 heads, times each head's factor: without a test per
// head where there are 16 (a test per store costs three times the store).
template <typename T, typename F>
__device__ __forceinline__ void write_heads(const uint32_t (&o)[16], const float *factor, int heads, T *to, int64_t stride,
                                            F convert) {
    if (heads >= 16) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(factor + k);
            to[0] = convert(__uint_as_float(o[k]) * f.x);
            to[stride] = convert(__uint_as_float(o[k + 1]) * f.y);
            to[2 * stride] = convert(__uint_as_float(o[k + 2]) * f.z);
            to[3 * stride] = convert(__uint_as_float(o[k + 3]) * f.w);
            to += 4 * stride;
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < heads; k++, to += stride)
            *to = convert(__uint_as_float(at16(o, k)) * factor[k]);
    }
}

// A tile's logits (log2) to the workspace, for the token weights: pairs of
// tokens where the whole tile is attended and its first token lies on an even
// place, else one by one. c0: the thread's first token of the tile.
__device__ __forceinline__ void keep_logits(const AttendPlan &P, const Walk &W, const Tile &T, const float *s, int head0,
                                            int heads, int ra, int c0) {
    const int at = T.t0 - (W.range.lo & ~1);
    const uint64_t inside = bits(W.range.lo - T.t0, min(T.rows, W.range.L - T.t0));
    float *a = P.logits + ((int64_t)W.r * P.H + head0 + ra) * P.logit_stride + at + c0, *b = a + 8 * P.logit_stride;
    if (inside == ~0ull && (at & 1) == 0) {
        if (ra < heads)
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<float2 *>(a + 8 * i) = make_float2(s[4 * i], s[4 * i + 1]);
        if (ra + 8 < heads)
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<float2 *>(b + 8 * i) = make_float2(s[4 * i + 2], s[4 * i + 3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int c = 8 * (i >> 2) + (i & 1);
        if ((inside >> (c + c0) & 1) && ((i & 2) ? ra + 8 : ra) < heads)
            ((i & 2) ? b : a)[c] = s[i];
    }
}

// Eight warps: the softmax, P, and the results. Warps w and w + 4 share heads
// 16 w .. 16 w + 15 of S (the lanes of tensor memory that both may read): w
// takes the tile's first 32 tokens, w + 4 the last. Of O^T they hold values
// 32 w .. 32 w + 31 of each 128, w of the even 128s and w + 4 of the odd.
template <bool kBf16, bool kFp8>
__device__ __forceinline__ void soften(const AttendPlan &P, Control &C, const Memory &M, Walk &W, int col, int group) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
    const uint32_t lanes = C.tmem + ((uint32_t)(quarter * 32) << 16);
    const int ra = quarter * 16 + lane / 4, rb = ra + 8;  // this thread's heads
    const int c0 = 32 * half + 2 * (lane & 3);            // and its first token
    const bool active = quarter * 16 < P.padded_heads;
    const int head0 = group * P.group_heads;
    const int heads = min(P.group_heads, P.H - head0);
    constexpr float kLift = kBf16 ? 0.0f : 7.0f;  // log2 of p's factor
    uint32_t n = 0;
    int4 left[2] = {make_int4(-1, 0, 0, 0), make_int4(-1, 0, 0, 0)};  // what the CTA leaves unfinished
    uint8_t *const pa = M.p + ra * 128 + 4 * (lane & 3), *const pb = M.p + rb * 128 + 4 * (lane & 3);

    // the rows of requests without tokens, while the first tile is on its way
    for (int r = col; r < P.R; r += P.cols) {
        const Range g = range_of(P, r);
        if (!g.ok || g.L != 0)
            continue;
        for (int h = head0 + (threadIdx.x >> 5); h < head0 + heads; h += kSoftWarps) {
            for (int v = lane; v < P.V; v += 32)
                P.out[r * P.out_request_stride + h * P.out_head_stride + v] = 0;
            if (lane == 0 && P.lse != nullptr)
                P.lse[r * P.lse_request_stride + h] = -INFINITY;
        }
    }

    for (uint32_t segments = 0; W.next(P); segments++) {
        float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;
        float ca = P.log2_scale, cb = P.log2_scale;
#pragma unroll 1
        for (int j = 0; j < W.count; j++, n++) {
            const int st = n % P.stages;
            bar_wait(C, &C.kv_full[st], (n / P.stages) & 1, P.status);
            if (kFp8 && j == 0) {
                bar_wait(C, &C.q_full, segments & 1, P.status);
                if (active) {
                    ca = P.log2_scale * C.q_scale[ra];
                    cb = P.log2_scale * C.q_scale[rb];
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&C.q_free);
            }
            const uint64_t valid = C.valid[n % (2 * kMaxStages)], zero = C.zero[n % (2 * kMaxStages)];
            bar_wait(C, &C.s_full[n & 1], (n >> 1) & 1, P.status);
            fence_after();
            uint32_t raw[16];
            float *s = reinterpret_cast<float *>(raw);
            float xa = -INFINITY, xb = -INFINITY;
            if (active) {
                load_s(raw, lanes + (n & 1) * 64 + half * 32);
                wait_ld();
            }
            fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(&C.s_free[n & 1]);
            if (active) {
#pragma unroll
                for (int i = 0; i < 16; i++)
                    s[i] *= (i & 2) ? cb : ca;
                if (valid != ~0ull) {
                    const uint64_t mine = valid >> c0;
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        if (!(mine >> (8 * (i >> 2) + (i & 1)) & 1))
                            s[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    xa = fmaxf(xa, fmaxf(s[i], s[i + 1]));
                    xb = fmaxf(xb, fmaxf(s[i + 2], s[i + 3]));
                }
                if (P.logits != nullptr)
                    keep_logits(P, W, tile_at(P, W.first + j), s, head0, heads, ra, c0);
            }
            // Does any logit exceed its head's reference by too much? (Each
            // thread asks for its own; the heads' maxima are only made then.)
            if (soft_any(xa > ma + kLag || xb > mb + kLag)) {
                xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
                xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
                xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
                xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
                if (active && (lane & 3) == 0) {
                    C.half[half][ra] = xa;
                    C.half[half][rb] = xb;
                }
                soft_sync();
                if (active) {
                    xa = fmaxf(xa, C.half[half ^ 1][ra]);
                    xb = fmaxf(xb, C.half[half ^ 1][rb]);
                }
                float fa = 1.0f, fb = 1.0f;
                if (xa > ma + kLag) {
                    fa = exp2_fast(ma - xa);
                    ma = xa;
                }
                if (xb > mb + kLag) {
                    fb = exp2_fast(mb - xb);
                    mb = xb;
                }
                la *= fa;
                lb *= fb;
                if (j > 0) {
                    if (active && half == 0 && (lane & 3) == 0) {
                        C.factor[ra] = fa;
                        C.factor[rb] = fb;
                    }
                    soft_sync();
                    bar_wait(C, &C.pv_done, (n - 1) & 1, P.status);
                    fence_after();
#pragma unroll 1
                    for (int t = half; t < P.value_tiles; t += 2)
#pragma unroll 1
                        for (int c = 0; c < P.padded_heads; c += 16) {
                            uint32_t o[16];
                            const uint32_t at = lanes + 128 + t * P.padded_heads + c;
                            load_o(o, at);
                            wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; k++)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * C.factor[c + k]);
                            store_o(o, at);
                        }
                    wait_st();
                    fence_before();
                }
                soft_sync();  // the maxima and factors may be written again
            }
            // P and the cleared rows go where the last tile's product read
            if (n > 0)
                bar_wait(C, &C.pv_done, (n - 1) & 1, P.status);
            if (active) {
                const float na = ma == -INFINITY ? 0.0f : ma - kLift, nb = mb == -INFINITY ? 0.0f : mb - kLift;
                const int x = ra & 7;  // rb & 7 is the same
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float p0 = exp2_fast(s[4 * i] - na), p1 = exp2_fast(s[4 * i + 1] - na);
                    const float p2 = exp2_fast(s[4 * i + 2] - nb), p3 = exp2_fast(s[4 * i + 3] - nb);
                    la += p0 + p1;
                    lb += p2 + p3;
                    *reinterpret_cast<uint32_t *>(pa + (((i + 4 * half) ^ x) << 4)) = pack<kBf16>(p0, p1);
                    *reinterpret_cast<uint32_t *>(pb + (((i + 4 * half) ^ x) << 4)) = pack<kBf16>(p2, p3);
                }
            }
            if (!kFp8 && zero != 0) {
                // tokens that are not attended take part with p = 0: their
                // values must not be infinite or NaN
                // (eight lanes to a row's panel: whole rows' stores would all
                // fall into the same banks)
                uint8_t *kv = M.kv + (size_t)st * M.stage_bytes + (threadIdx.x & 7) * 16;
                for (int row = threadIdx.x >> 3; row < kTile; row += kSoftWarps * 4)
                    if (zero >> row & 1)
                        for (int i = 0; i < 2 * P.value_tiles; i++)
                            *reinterpret_cast<uint4 *>(kv + i * kPanel + row * 128) = make_uint4(0, 0, 0, 0);
            }
            fence_async();
            __syncwarp();
            if (lane == 0)
                bar_arrive(&C.p_full);
        }

        // the segment's end: each head's sum over its threads
        la += __shfl_xor_sync(0xffffffffu, la, 1);
        lb += __shfl_xor_sync(0xffffffffu, lb, 1);
        la += __shfl_xor_sync(0xffffffffu, la, 2);
        lb += __shfl_xor_sync(0xffffffffu, lb, 2);
        if (active && half == 1 && (lane & 3) == 0) {
            C.half[1][ra] = la;
            C.half[1][rb] = lb;
        }
        soft_sync();
        const bool whole = W.begins && W.ends;
        const int slot = 2 * col + (W.begins ? 1 : 0);
        if (active && half == 0 && (lane & 3) == 0) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int row = k ? rb : ra;
                const float m0 = k ? mb : ma, m = m0 == -INFINITY ? 0.0f : m0 - kLift;
                const float l = (k ? lb : la) + C.half[1][row];
                C.inverse[row] = whole ? (l == 0.0f ? 0.0f : P.scale / l) : P.scale;
                if (row >= heads)
                    continue;
                const int h = head0 + row;
                if (whole) {
                    const float lse = l == 0.0f ? -INFINITY : m + log2f(l);
                    P.lse2[(int64_t)W.r * P.H + h] = lse;
                    if (P.lse != nullptr)
                        P.lse[W.r * P.lse_request_stride + h] = lse * 0.693147180559945309f;
                } else {
                    P.part_ml[(int64_t)slot * P.H + h] = make_float2(m, l);
                }
            }
        }
        if (!whole)
            left[slot & 1] = make_int4(W.r, W.count, W.tiles, 0);
        soft_sync();
        bar_wait(C, &C.pv_done, (n - 1) & 1, P.status);
        fence_after();
#pragma unroll 1
        for (int t = half; t < P.value_tiles; t += 2) {
            const int v = t * 128 + quarter * 32 + lane;
            uint32_t o[kFp8 ? 1 : 2][16];  // (an fp8 cache leaves the softmax few registers)
            constexpr int kTake = kFp8 ? 1 : 2;
#pragma unroll 1
            for (int c0 = 0; c0 < P.padded_heads; c0 += 16 * kTake) {
                load_o(o[0], lanes + 128 + t * P.padded_heads + c0);
                if (kTake > 1 && c0 + 16 < P.padded_heads)
                    load_o(o[kTake - 1], lanes + 128 + t * P.padded_heads + c0 + 16);
                wait_ld();
#pragma unroll
                for (int i = 0; i < kTake; i++) {
                    const int c = c0 + 16 * i;
                    if (v >= P.V) {
                        // not a value: nothing to write
                    } else if (whole) {
                        uint16_t *to = P.out + W.r * P.out_request_stride + (head0 + c) * P.out_head_stride + v;
                        write_heads(o[i], C.inverse + c, heads - c, to, P.out_head_stride,
                                    [&](float x) { return to_out(x, P.q_bf16); });
                    } else {
                        float *to = P.part_o + ((int64_t)slot * P.H + head0 + c) * P.V + v;
                        write_heads(o[i], C.inverse + c, heads - c, to, (int64_t)P.V, [](float x) { return x; });
                    }
                    __syncwarp();  // together again for the next read of tensor memory
                }
            }
        }
        fence_before();
        soft_sync();  // the inverses may be written again
        if (lane == 0)
            bar_arrive(&C.o_free);
    }
    if (threadIdx.x == 0 && group == 0) {
        P.segment[2 * col] = left[0];
        P.segment[2 * col + 1] = left[1];
    }
}

template <bool kBf16, bool kFp8>
__global__ void __launch_bounds__(kThreads<kFp8>, 1) lmc_attend_kernel(const __grid_constant__ AttendPlan P) {
    extern __shared__ __align__(1024) uint8_t attend_mem[];
    __shared__ Control C;
    const int warp = threadIdx.x >> 5;
    const int group = blockIdx.x % P.head_groups, col = blockIdx.x / P.head_groups;
    Memory M;
    M.q = attend_mem;
    M.stage_bytes = P.panels * kPanel;
    M.kv = M.q + (size_t)((P.E + 63) / 64) * P.padded_heads * 128;
    M.p = M.kv + (size_t)P.stages * M.stage_bytes;
    if (threadIdx.x == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.query) : "memory");
        if (!kFp8)
            asm volatile("prefetch.tensormap [%0];" ::"l"(&P.cache) : "memory");
    }
    if (threadIdx.x == 0) {
        bar_init(&C.q_full, kFp8 ? kFp8Loaders : 1);
        bar_init(&C.q_raw, 1);
        bar_init(&C.q_free, kFp8 ? 1 + kSoftWarps : 1);  // the products', and the readers of q_scale
        for (int i = 0; i < P.stages; i++) {
            bar_init(&C.kv_full[i], kFp8 ? kFp8Loaders : 1);
            bar_init(&C.kv_free[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(&C.s_full[i], 1);
            bar_init(&C.s_free[i], kSoftWarps);
        }
        bar_init(&C.p_full, kSoftWarps);
        bar_init(&C.pv_done, 1);
        bar_init(&C.o_free, kSoftWarps);
        bar_init(&C.ended[0], 1);
        bar_init(&C.ended[1], 1);
        C.gave_up = 0;
        C.loading = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    // Tensor memory is asked for after the wait: a kernel before this one that
    // has yet to ask for its own would wait for this one, which waits for it.
    // (And the next one may only start when this one's is had.)
    wait_for_launch();
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&C.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (P.brief)
        let_next_start();

    if (warp < kSoftWarps) {
        if (kFp8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSoftRegisters));
        Walk W;
        W.init<kFp8>(P, col);
        soften<kBf16, kFp8>(P, C, M, W, col, group);
    } else if (kFp8 && warp >= kFirstFp8Loader) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLoadRegisters));
        Walk W;
        W.init<kFp8>(P, col);
        load_fp8(P, C, M, W, group);
    } else {
        if (kFp8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegisters));
        Walk W;
        W.init<kFp8>(P, col);
        if (warp == kScoreWarp)
            multiply_scores<kBf16>(P, C, M, W);
        else if (warp == kValueWarp)
            multiply_values<kBf16>(P, C, M, W);
        else if (warp == kAheadWarp)
            send_ahead(P, C, W);
        else if (!kFp8)
            load_by_tma(P, C, M, W, group);
    }
    // lengths that cannot be served
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < P.R; r += blockDim.x)
            if (!range_of(P, r).ok)
                atomicOr(P.status, LMC_ST_BAD_JOB);
    fence_before();
    __syncthreads();
    fence_after();
    if (C.gave_up) {
        wind_up<kFp8>(P, C, warp);
        __syncthreads();
    }
    if (warp == kScoreWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(C.tmem));
}

// ---- joining -------------------------------------------------------------------

// Warps of a joining block: a head each, or all of them one head: four take a
// quarter of its values each, four times, for every fourth part.
template <int kSlices>
constexpr int kJoinWarps = kSlices == 1 ? 4 : 16;
constexpr int kJoinNotes = kMaxCols / 32;  // per lane

// Block (x, y): joins heads of the x-th request that spans several CTAs (each
// begins in a CTA of its own, so there are at most as many as requests and
// CTAs). A warp joins a head, or (kSlices = 4) a quarter of its values and of
// its parts. What bounds it is latency, so it makes three trips to memory: all
// CTAs' notes, the parts' factors, the parts. (Looking for the request in a
// loop over the notes and reading its length again took 14.5 us for 152
// requests of 32 heads, four warps to a head in every case 12 us; with few
// heads to join, one warp to a head leaves the device idle.)
template <int kSlices>
__global__ void __launch_bounds__(kJoinWarps<kSlices> * 32) lmc_attend_join_kernel(const __grid_constant__ AttendPlan P) {
    constexpr int kTake = kMaxValue / 128 / kSlices;  // float4s per lane
    constexpr int kShare = kSlices == 1 ? 1 : 4;      // a warp takes every kShare-th part
    __shared__ float factors[kJoinWarps<kSlices>][kMaxCols];
    __shared__ float4 shares[kShare][kShare == 1 ? 1 : kMaxValue / 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = kSlices == 1 ? blockIdx.y * kJoinWarps<1> + warp : blockIdx.y;
    const int v0 = 4 * lane + (kSlices == 1 ? 0 : 128 * (warp & 3)), share = kSlices == 1 ? 0 : warp >> 2;
    wait_for_launch();
    let_next_start();
    if (h >= P.H)
        return;
    int4 begun[kJoinNotes];
    int2 gone_on[kJoinNotes];
#pragma unroll
    for (int i = 0; i < kJoinNotes; i++) {
        const int c = 32 * i + lane;
        begun[i] = make_int4(-1, 0, 0, 0);
        gone_on[i] = make_int2(-1, 0);
        if (c < P.cols) {
            begun[i] = P.segment[2 * c + 1];
            gone_on[i] = *reinterpret_cast<const int2 *>(P.segment + 2 * c);
        }
    }
    int col = -1, seen = 0, r = -1, rest = 0;
#pragma unroll
    for (int i = 0; i < kJoinNotes; i++) {
        const uint32_t here = __ballot_sync(0xffffffffu, begun[i].x >= 0);
        const int rank = seen + __popc(here & ((1u << lane) - 1u));
        const uint32_t mine = __ballot_sync(0xffffffffu, begun[i].x >= 0 && rank == (int)blockIdx.x);
        if (mine != 0) {
            const int k = __ffs(mine) - 1;
            col = 32 * i + k;
            r = __shfl_sync(0xffffffffu, begun[i].x, k);
            rest = __shfl_sync(0xffffffffu, begun[i].z - begun[i].y, k);
        }
        seen += __popc(here);
    }
    if (col < 0)
        return;
    // parts: slot 2 col + 1, then 2 (col + 1), ...; all CTAs but the last have
    // as many tiles as the next one
    int next_r = -1, each = 0;
#pragma unroll
    for (int i = 0; i < kJoinNotes; i++)
        if (32 * i + lane == col + 1) {
            next_r = gone_on[i].x;
            each = gone_on[i].y;
        }
    next_r = __shfl_sync(0xffffffffu, next_r, (col + 1) & 31);
    each = __shfl_sync(0xffffffffu, each, (col + 1) & 31);
    const int parts = rest > 0 && next_r == r ? min(P.cols - col, 1 + (rest + each - 1) / max(1, each)) : 1;
    const float2 *ml = P.part_ml + (int64_t)2 * col * P.H + h;
    float2 x[kJoinNotes];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kJoinNotes; i++) {
        const int k = 32 * i + lane;
        x[i] = k < parts ? ml[(int64_t)(2 * k + (k == 0)) * P.H] : make_float2(0.0f, 0.0f);
        if (x[i].y != 0.0f)
            top = fmaxf(top, x[i].x);
    }
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinNotes; i++) {
        const float f = x[i].y == 0.0f ? 0.0f : exp2_fast(x[i].x - top);
        factors[warp][32 * i + lane] = f;
        sum += x[i].y == 0.0f ? 0.0f : x[i].y * f;
    }
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (lane == 0 && (kSlices == 1 || warp == 0)) {
        const float lse = sum == 0.0f ? -INFINITY : top + log2f(sum);
        P.lse2[(int64_t)r * P.H + h] = lse;
        if (P.lse != nullptr)
            P.lse[r * P.lse_request_stride + h] = lse * 0.693147180559945309f;
    }
    float4 acc[kTake] = {};
    const float *part = P.part_o + ((int64_t)2 * col * P.H + h) * P.V + v0;
    const int64_t step = (int64_t)P.H * P.V;
#pragma unroll(kSlices == 1 ? 2 : 10)
    for (int i = share; i < parts; i += kShare) {
        const float f = factors[warp][i];
#pragma unroll
        for (int k = 0; k < kTake; k++)
            if (v0 + 128 * k < P.V) {
                const float4 y = __ldcs(reinterpret_cast<const float4 *>(part + (2 * i + (i == 0)) * step + 128 * k));
                acc[k].x += y.x * f;
                acc[k].y += y.y * f;
                acc[k].z += y.z * f;
                acc[k].w += y.w * f;
            }
    }
    if constexpr (kShare > 1) {
        shares[share][v0 / 4] = acc[0];
        __syncthreads();
        if (share > 0)
            return;
        for (int k = 1; k < kShare; k++) {
            const float4 y = shares[k][v0 / 4];
            acc[0].x += y.x;
            acc[0].y += y.y;
            acc[0].z += y.z;
            acc[0].w += y.w;
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *to = P.out + r * P.out_request_stride + h * P.out_head_stride + v0;
#pragma unroll
    for (int k = 0; k < kTake; k++, to += 128)
        if (v0 + 128 * k < P.V) {
            to[0] = to_out(acc[k].x * inv, P.q_bf16);
            to[1] = to_out(acc[k].y * inv, P.q_bf16);
            to[2] = to_out(acc[k].z * inv, P.q_bf16);
            to[3] = to_out(acc[k].w * inv, P.q_bf16);
        }
}

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 256;  // of a block's turn: four per thread
constexpr int kWeightParts = 4;     // the heads are dealt out to as many threads
// Blocks per SM, about. (256 requests of 100 tokens in a batch that could hold
// 131072: one block for every 256 tokens that there might be 161 us, 64 an SM 34,
// 32 an SM 30, 8 an SM 26; 64 ragged requests of up to 32768, whose blocks then
// take turns at 32 and 8: 106.8, 106.8, 109.3 and 120.)
constexpr int kWeightPerSm = 64;

// Each token's sum over the heads of 2^(logit - lse). A thread has four tokens
// and a quarter of the heads, so all of its loads are in flight at once; the
// quarters are added in shared memory, always in the same order. A request's
// blocks take turns along its tokens (kTurns), so that the grid does not grow
// with the lengths that a batch might have; where it covers them without, the
// loop's registers are saved (64 ragged requests 107.9 -> 106.8 us).
template <bool kTurns>
__global__ void __launch_bounds__(kWeightThreads) lmc_attend_weights_kernel(const __grid_constant__ AttendPlan P) {
    __shared__ float4 sums[kWeightParts][kWeightTokens / 4];
    const int r = blockIdx.y;
    wait_for_launch();
    let_next_start();
    const Range g = range_of(P, r);
    const int base = g.lo & ~1;  // the logits' first place, and 16-byte aligned
    int first = blockIdx.x * kWeightTokens;
    if (!g.ok || g.L == 0 || first >= g.L - base)
        return;
    const int four = threadIdx.x % (kWeightTokens / 4), part = threadIdx.x / (kWeightTokens / 4);
    const float *lse = P.lse2 + (int64_t)r * P.H;
    const uint32_t step = gridDim.x * kWeightTokens;
    for (;;) {
        const float *x = P.logits + (int64_t)r * P.H * P.logit_stride + first + 4 * four;
        float4 w = {};
        if (first + 4 * four < g.L - base) {
#pragma unroll 8
            for (int h = part; h < P.H; h += kWeightParts) {
                const float top = __ldca(lse + h);
                const float4 v = __ldcs(reinterpret_cast<const float4 *>(x + h * P.logit_stride));
                if (top != -INFINITY) {
                    w.x += exp2_fast(v.x - top);
                    w.y += exp2_fast(v.y - top);
                    w.z += exp2_fast(v.z - top);
                    w.w += exp2_fast(v.w - top);
                }
            }
        }
        sums[part][four] = w;
        __syncthreads();
        const int t = base + first + (int)threadIdx.x;
        if (t >= g.lo && t < g.L) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kWeightParts; k++)
                sum += reinterpret_cast<const float *>(sums[k])[threadIdx.x];
            P.weights[r * P.weights_request_stride + t] += sum;
        }
        if (!kTurns || (uint32_t)(g.L - base - first) <= step)
            break;
        first += step;
        __syncthreads();  // the sums may be written again
    }
}

// ---- host ------------------------------------------------------------------------

bool aligned16(int64_t x) { return (x & 15) == 0; }

struct Work {
    int32_t cols, head_groups, group_heads;
    int64_t logit_stride;
    int64_t segment, part_ml, part_o, lse2, logits, bytes;  // offsets
};

// 0: none (a full-attention layer's spec may hold any number there).
int32_t window_of(const lmc_layout *L, int32_t layer) {
    return L->specs[layer].kind == LMC_LAYER_SWA ? L->specs[layer].window : 0;
}

int work_space(const lmc_layout *L, int32_t layer, int64_t R, int64_t H, int64_t V, int64_t max_length, bool weights,
               Work &W) {
    if (L == nullptr || layer < 0 || (size_t)layer >= L->desc.size() || L->specs[layer].kind == LMC_LAYER_KDA ||
        R < 0 || R > 65535 || H <= 0 || H > 65535 || V <= 0 || V > kMaxValue || max_length <= 0 ||
        max_length > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    W.head_groups = (int32_t)((H + kMaxHeads - 1) / kMaxHeads);
    W.group_heads = (int32_t)((H + W.head_groups - 1) / W.head_groups);
    W.cols = std::max(1, kMaxCols / W.head_groups);
    const int64_t window = window_of(L, layer);
    const int64_t tokens = window > 0 ? std::min(max_length, window) : max_length;
    W.logit_stride = (tokens + 1 + 3) / 4 * 4;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    W.segment = take(2 * W.cols * 16);
    W.part_ml = take(2 * W.cols * H * 8);
    W.part_o = take(2 * W.cols * H * V * 4);
    W.lse2 = take(R * H * 4);
    int64_t logits = 0;
    if (weights && (!lmc::mul_ok(R * H, W.logit_stride, &logits) || !lmc::mul_ok(logits, 4, &logits) ||
                    logits > INT64_MAX / 2))
        return LMC_ERR_OVERFLOW;
    W.logits = take(logits);
    W.bytes = at;
    return LMC_OK;
}

// Short caches: each request is left to one CTA, and nothing has to be joined,
// where a CTA then has at most kWholeTiles tiles, at most kWholeExtra above an
// equal share. (Graphs of calls of 32 heads, whole and shared out: one request of
// 64 tokens 7.8 and 9.3 us, of 128 8.8 and 10.6, of 192 10.5 and 10.7; one of 256
// is shared out, 10.7; 152 requests of 64 tokens 10.7 and 13.1, of 256 14.7 and
// 17.2; 304 of 128 18.5 and 20.8; 608 of 64 27.6 and 30.1. More tiles gain as much
// where all lengths are near the longest, but they may not be.)
constexpr int kWholeTiles = 4, kWholeExtra = 2;

// An upper bound of a request's tiles (exact without a window).
int64_t most_tiles(const AttendPlan &P) {
    if (P.max_length == 0)
        return 0;
    if (P.window == 0 || P.window >= P.max_length) {
        const int last = P.max_length - 1;
        return (int64_t)last / P.span * P.tiles_per_span + last % P.span / kTile + 1;
    }
    const int64_t more = P.window - 1;  // a window begins anywhere in a tile
    return more / std::min(kTile, P.span) + 2 + (P.span > kTile ? more / P.span + 1 : 0);
}

// (values, rows, slices) of 16 bits each, read in boxes of `box` rows of one
// slice: of all panels of 64 values at once (`whole`; the values are a
// multiple of 64 then), or of one.
bool tensor_map(CUtensorMap *map, bool bf16, const void *base, int64_t values, int64_t rows, int64_t slices,
                int64_t row_bytes, int64_t slice_bytes, int box, bool whole) {
    const EncodeTiled fn = encoder();
    if (fn == nullptr)
        return false;
    const cuuint64_t panels = whole ? (cuuint64_t)values / 64 : 1;
    const cuuint64_t dims[4] = {whole ? 64 : (cuuint64_t)values, (cuuint64_t)rows, panels, (cuuint64_t)slices};
    const cuuint64_t strides[3] = {(cuuint64_t)row_bytes, 128, (cuuint64_t)slice_bytes};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, (cuuint32_t)panels, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<void *>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" int lmc_attend_workspace(const lmc_layout *L, int32_t layer, int32_t num_requests, int32_t num_heads,
                                    int32_t value_dim, int64_t max_length, int with_weights, int64_t *out) {
    Work W;
    if (out == nullptr)
        return LMC_ERR_INVALID_ARG;
    const int rc = work_space(L, layer, num_requests, num_heads, value_dim, max_length, with_weights != 0, W);
    if (rc == LMC_OK)
        *out = W.bytes;
    return rc;
}

extern "C" int lmc_attend(const lmc_layout *L, const lmc_entries *e, const void *pool, const lmc_attention *a,
                          void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream) {
    if (const int rc = lmc::check_entries(L, e); rc != LMC_OK)
        return rc;
    if (a == nullptr || status == nullptr || (a->q_dtype != LMC_E_BF16 && a->q_dtype != LMC_E_F16) ||
        (e->dtype != LMC_E_E4M3 && e->dtype != a->q_dtype) || e->entry_dim % 16 != 0 || e->entry_dim > kMaxEntry ||
        a->num_heads <= 0 || a->value_dim <= 0 || a->value_dim % 8 != 0 || a->value_dim > e->entry_dim ||
        a->value_dim > kMaxValue || !std::isfinite(a->softmax_scale))
        return LMC_ERR_INVALID_ARG;
    const float log2_scale = (float)((double)a->softmax_scale * e->scale * 1.4426950408889634);
    if (!std::isfinite(log2_scale))
        return LMC_ERR_INVALID_ARG;
    const int64_t R = e->num_requests, H = a->num_heads;
    if (a->q_request_stride < 0 || a->q_head_stride < 0 || a->out_request_stride < 0 || a->out_head_stride < 0 ||
        a->q_request_stride % 8 != 0 || a->q_head_stride % 8 != 0 || (H > 1 && a->q_head_stride == 0) ||
        (R > 1 && a->q_request_stride == 0) || (H > 1 && a->out_head_stride < a->value_dim) ||
        (R > 1 && a->out_request_stride < a->value_dim) || (a->lse != nullptr && a->lse_request_stride < H) ||
        (a->weights != nullptr && a->weights_request_stride < a->max_length))
        return LMC_ERR_INVALID_ARG;
    Work W;
    if (const int rc = work_space(L, e->layer, R, H, a->value_dim, a->max_length, a->weights != nullptr, W);
        rc != LMC_OK)
        return rc;
    if (R > 0 && (pool == nullptr || a->lengths == nullptr || a->q == nullptr || a->out == nullptr ||
                  workspace == nullptr || workspace_bytes < W.bytes))
        return LMC_ERR_INVALID_ARG;
    const lmc_layer_desc &d = L->desc[e->layer];
    if ((((uintptr_t)status | (uintptr_t)a->lengths | (uintptr_t)a->lse | (uintptr_t)a->weights) & 3) != 0 ||
        !aligned16((int64_t)(uintptr_t)pool) || !aligned16(d.base) || !aligned16(d.stride) ||
        !aligned16((int64_t)(uintptr_t)a->q) || ((uintptr_t)a->out & 1) != 0 || ((uintptr_t)workspace & 255) != 0)
        return LMC_ERR_ALIGN;
    if (R == 0)
        return LMC_OK;
    const int sms = lmc::sm_count();
    if (sms <= 0)
        return LMC_ERR_CUDA;
    const bool fp8 = e->dtype == LMC_E_E4M3, bf16 = a->q_dtype == LMC_E_BF16;
    const int64_t N = L->block_size;
    AttendPlan P = {};
    P.pool = static_cast<const uint8_t *>(pool) + d.base;
    P.block_stride = d.stride;
    P.num_blocks = L->num_blocks;
    P.table = e->table.table;
    P.row_stride = e->table.row_stride;
    P.lengths = a->lengths;
    P.max_length = (int32_t)std::min(a->max_length, (int64_t)std::min<int64_t>(e->table.num_cols, INT32_MAX / N) * N);
    P.q = static_cast<const uint16_t *>(a->q);
    P.q_request_stride = a->q_request_stride;
    P.q_head_stride = a->q_head_stride;
    P.out = static_cast<uint16_t *>(a->out);
    P.out_request_stride = a->out_request_stride;
    P.out_head_stride = a->out_head_stride;
    P.lse = a->lse;
    P.lse_request_stride = a->lse_request_stride;
    P.weights = a->weights;
    P.weights_request_stride = a->weights_request_stride;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.segment = reinterpret_cast<int4 *>(ws + W.segment);
    P.part_ml = reinterpret_cast<float2 *>(ws + W.part_ml);
    P.part_o = reinterpret_cast<float *>(ws + W.part_o);
    P.lse2 = reinterpret_cast<float *>(ws + W.lse2);
    P.logits = a->weights != nullptr ? reinterpret_cast<float *>(ws + W.logits) : nullptr;
    P.logit_stride = W.logit_stride;
    P.status = status;
    P.R = (int32_t)R;
    P.H = (int32_t)H;
    P.E = e->entry_dim;
    P.V = a->value_dim;
    P.window = window_of(L, e->layer);
    P.block_size = (int32_t)N;
    P.token_bytes = (int32_t)L->specs[e->layer].token_bytes;
    // several small pages share a tile where each fills whole 8-row groups of it
    P.pages_per_tile = N < kTile && N % 8 == 0 ? (int32_t)(kTile / N) : 1;
    P.span = (int32_t)N * P.pages_per_tile;
    P.tiles_per_span = (P.span + kTile - 1) / kTile;
    auto inverse = [](int32_t d) { return d == 1 ? ~0u : (uint32_t)(((uint64_t)1 << 32) / (uint32_t)d); };
    P.span_inverse = inverse(P.span);
    P.tiles_inverse = inverse(P.tiles_per_span);
    if (R * (P.max_length / P.span + 1) * P.tiles_per_span > INT32_MAX - kMaxCols)
        return LMC_ERR_OVERFLOW;
    P.head_groups = W.head_groups;
    P.group_heads = W.group_heads;
    P.cols = std::max(1, std::min(W.cols, sms / W.head_groups));
    P.padded_heads = (P.group_heads + 15) / 16 * 16;
    P.value_tiles = (P.V + 127) / 128;
    P.panels = std::max((P.E + 63) / 64, 2 * P.value_tiles);
    P.q_bf16 = bf16;
    P.scale = e->scale;
    P.log2_scale = log2_scale;
    const int64_t turns = ((R + P.cols - 1) / P.cols) * most_tiles(P);
    if (turns <= kWholeTiles && turns <= (R * most_tiles(P) + P.cols - 1) / P.cols + kWholeExtra) {
        // no CTA without a request (32 fp8 requests of 128 tokens 15.3 -> 14.4 us with the next line)
        P.whole = (int32_t)((R + P.cols - 1) / P.cols);
        P.cols = (int32_t)((R + P.whole - 1) / P.whole);
        P.brief = P.weights == nullptr;
    }
    P.cols_inverse = inverse(P.cols);
    const int64_t fixed = (int64_t)((P.E + 63) / 64) * P.padded_heads * 128 + P.padded_heads * 128 + sizeof(Control) + 1024;
    P.stages = (int32_t)std::min<int64_t>(kMaxStages, (kSmemLimit - fixed) / ((int64_t)P.panels * kPanel));
    const size_t smem = std::max<size_t>((size_t)((P.E + 63) / 64) * P.padded_heads * 128 + (size_t)P.padded_heads * 128 +
                                             (size_t)P.stages * P.panels * kPanel,
                                         120 * 1024);  // one CTA per SM: each takes the whole tensor memory
    if (d.stride >= (int64_t)1 << 40 || L->num_blocks > INT32_MAX || a->q_request_stride >= (int64_t)1 << 38 ||
        a->q_head_stride >= (int64_t)1 << 38)
        return LMC_ERR_INVALID_ARG;
    const int row_panels = (P.E + 63) / 64;
    const bool whole = P.E % 64 == 0, tile = P.pages_per_tile == 1;
    const int64_t head_bytes = H > 1 ? a->q_head_stride * 2 : (int64_t)P.E * 2;
    const int64_t request_bytes = R > 1 ? a->q_request_stride * 2 : head_bytes * H;
    P.cache_copies = whole && tile ? 1 : row_panels;
    P.query_copies = whole ? 1 : row_panels;
    if (!tensor_map(&P.query, bf16, a->q, P.E, H, R, head_bytes, request_bytes, P.padded_heads, whole) ||
        (!fp8 && !tensor_map(&P.cache, bf16, P.pool, P.E, N, L->num_blocks, P.token_bytes, d.stride,
                             tile ? kTile : (int)N, whole && tile)))
        return LMC_ERR_CUDA;
    auto kern = fp8 ? lmc_attend_kernel<false, true> : bf16 ? lmc_attend_kernel<true, false> : lmc_attend_kernel<false, false>;
    static std::atomic<uint64_t> allowed[3];
    if (!lmc::allow_shared_memory(allowed[fp8 ? 2 : bf16 ? 1 : 0], kern,
                                  kSmemLimit - (int)((sizeof(Control) + 1023) / 1024 * 1024)))
        return LMC_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!follow(kern, dim3((unsigned)(P.cols * P.head_groups)), fp8 ? kThreads<true> : kThreads<false>, smem, s, P))
        return LMC_ERR_CUDA;
    if (P.whole == 0) {
        // A warp per head where that is a few warps an SM; else a request has
        // many parts and the heads are few (4 x 131072 tokens, 64 heads: 38
        // parts each, 12 us by a warp per head, 6 us by sixteen; 32 requests of
        // 32 heads, 5 parts each: 12 us by sixteen).
        const unsigned splits = (unsigned)std::min<int64_t>(P.cols, R);
        const bool few = (int64_t)splits * H < 4 * (int64_t)sms;
        if (!(few ? follow(lmc_attend_join_kernel<4>, dim3(splits, (unsigned)H), kJoinWarps<4> * 32, 0, s, P)
                  : follow(lmc_attend_join_kernel<1>, dim3(splits, (unsigned)((H + kJoinWarps<1> - 1) / kJoinWarps<1>)),
                           kJoinWarps<1> * 32, 0, s, P)))
            return LMC_ERR_CUDA;
    }
    if (P.weights != nullptr) {
        const int64_t tokens = P.window > 0 ? std::min(P.max_length, P.window) : P.max_length;
        const int64_t all = tokens / kWeightTokens + 1, blocks = std::min(all, ((int64_t)kWeightPerSm * sms + R - 1) / R);
        if (!follow(blocks < all ? lmc_attend_weights_kernel<true> : lmc_attend_weights_kernel<false>,
                    dim3((unsigned)blocks, (unsigned)R), kWeightThreads, 0, s, P))
            return LMC_ERR_CUDA;
    }
    return LMC_OK;  // every launch was asked for its own error
}
