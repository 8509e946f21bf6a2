// tokens.cu -- single tokens' entries of paged attention layers: appending
// new entries by block table, selecting the tokens a request keeps by their
// accumulated attention weight, and moving the kept entries into other
// blocks, for sm_103a. The kernels start up behind the one before them in the
// stream (append of 256 rows in a row 6.2 -> 4.1 us a call, of 131072 rows 39.3
// -> 37.4, a select of two short rows 8.2 -> 5.8).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "follow.cuh"
#include "lmc_internal.h"

namespace cg = cooperative_groups;

namespace {

struct TokenTable {
    const int32_t *ptr;
    int64_t row_stride;
    int32_t num_cols;
};

// The layer pages a token position resolves into.
struct Pages {
    int64_t base;       // pool byte of the first layer's block 0
    int64_t stride;     // bytes between blocks
    int64_t num_blocks;
    int32_t block_size;
    int32_t token_bytes;
};

// Pool byte of the entry at `pos` of request `req` (in range) under the
// table; -1 with the status bit to raise when it has none.
__device__ __forceinline__ int64_t entry_offset(const Pages &G, const TokenTable &T, int64_t req, int32_t pos,
                                                uint32_t &bad) {
    const int32_t page = pos < 0 ? -1 : pos / G.block_size;
    if (page < 0 || page >= T.num_cols) {
        bad |= LMC_ST_BAD_JOB;
        return -1;
    }
    const int32_t block = __ldca(T.ptr + req * T.row_stride + page);
    if (block < 0 || block >= G.num_blocks) {
        bad |= block == -1 ? LMC_ST_NO_BLOCK : LMC_ST_BLOCK_OOR;
        return -1;
    }
    return G.base + (int64_t)block * G.stride + (int64_t)(pos - page * G.block_size) * G.token_bytes;
}

// A piece's row: n / d by a multiplication with m = ceil(2^32 / d), exact
// while n * d < 2^32 (a CTA has at most 4096 pieces, or one row: m = 1 gives
// 0). m = 0 stands for d = 1.
struct Divider {
    uint32_t d, m;
};
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider &D, uint32_t &rem) {
    const uint32_t q = D.m == 0 ? n : __umulhi(n, D.m);
    rem = n - q * D.d;
    return q;
}

constexpr int kRowThreads = 256;
constexpr int kMaxRows = 64;     // rows a CTA resolves at a time
constexpr int kRowUnroll = 4;    // pieces in flight per thread
constexpr int kCodeUnroll = 3;   // and of a row turned to codes (1: 41 us, 3: 39 us at 131072 rows, with 2 us of launch)

// Copies `rows` rows of `pieces` pieces of V each from src[i] to dst[i] (a
// null source skips the row): the CTA's threads take the pieces in order, so
// neighbouring threads touch neighbouring bytes, kRowUnroll loads before the
// matching stores.
template <typename V>
__device__ __forceinline__ void copy_rows(const uint8_t *const *src, uint8_t *const *dst, int rows,
                                          const Divider &pieces) {
    const uint32_t total = (uint32_t)rows * pieces.d;
    for (uint32_t first = threadIdx.x; first < total; first += kRowThreads * kRowUnroll) {
        V v[kRowUnroll];
        V *to[kRowUnroll];
#pragma unroll
        for (int u = 0; u < kRowUnroll; u++) {
            const uint32_t i = first + u * kRowThreads;
            to[u] = nullptr;
            if (i < total) {
                uint32_t at;
                const uint32_t row = divide(i, pieces, at);
                if (src[row] != nullptr) {
                    v[u] = __ldcs(reinterpret_cast<const V *>(src[row]) + at);
                    to[u] = reinterpret_cast<V *>(dst[row]) + at;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kRowUnroll; u++)
            if (to[u] != nullptr)
                __stcs(to[u], v[u]);
    }
}

struct AppendPlan {
    Pages pages;
    TokenTable table;
    const int32_t *requests;
    const int32_t *positions;
    const uint8_t *rows;
    int64_t row_bytes;  // between rows
    uint8_t *pool;
    uint32_t *status;
    int64_t num_rows;
    int32_t num_requests;
    int32_t rows_per_cta;
    Divider pieces;  // pieces of one row
    float scale, inverse;
};

// Source and destination of the CTA's rows.
__device__ __forceinline__ int resolve_append(const AppendPlan &P, const uint8_t **src, uint8_t **dst) {
    const int64_t first = (int64_t)blockIdx.x * P.rows_per_cta;
    const int n = (int)min((int64_t)P.rows_per_cta, P.num_rows - first);
    if ((int)threadIdx.x < n) {
        const int64_t i = first + threadIdx.x;
        const int32_t req = __ldca(P.requests + i);
        const uint8_t *s = nullptr;
        uint8_t *d = nullptr;
        if (req != -1) {
            uint32_t bad = 0;
            int64_t off = -1;
            if (req < 0 || req >= P.num_requests)
                bad = LMC_ST_BAD_JOB;
            else
                off = entry_offset(P.pages, P.table, req, __ldca(P.positions + i), bad);
            if (bad)
                atomicOr(P.status, bad);
            if (off >= 0) {
                s = P.rows + i * P.row_bytes;
                d = P.pool + off;
            }
        }
        src[threadIdx.x] = s;
        dst[threadIdx.x] = d;
    }
    __syncthreads();
    return n;
}

template <typename V>
__global__ void __launch_bounds__(kRowThreads) lmc_append_kernel(const __grid_constant__ AppendPlan P) {
    __shared__ const uint8_t *src[kMaxRows];
    __shared__ uint8_t *dst[kMaxRows];
    lmc::wait_for_launch();
    lmc::let_next_start();
    const int n = resolve_append(P, src, dst);
    copy_rows<V>(src, dst, n, P.pieces);
}

__device__ __forceinline__ float2 to_float2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 to_float2(__half2 v) { return __half22float2(v); }

// The IEEE quotient x / scale. With inverse = RN(1 / scale) given (0 where the
// host found the scale out of range), by Markstein's correction of a
// reciprocal product (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): q0 = RN(x *
// inverse) is within an ulp of the quotient, its residual is exact in one FMA,
// and RN(q0 + residual * inverse) is the correctly rounded quotient while
// nothing underflows (scale in [2^-100, 2^100], significand not all ones; a
// residual only underflows where the code is 0). Far past the largest code
// (an infinity's residual is NaN) q0 itself will do. Sixteen divisions a piece
// bound the kernel by instructions: 45 us for 131072 rows of 576 values, this
// 37 us (6.1 TB/s).
__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
    if (inverse == 0.0f)
        return __fdiv_rn(x, scale);
    const float q = x * inverse;
    const float exact = fmaf(fmaf(-q, scale, x), inverse, q);
    return fabsf(q) < 4096.0f && q != 0.0f ? exact : q;  // (-0 stays -0)
}

// Two values as fp8 codes: saturated (satfinite), half to even, NaN to NaN.
__device__ __forceinline__ uint32_t codes2(float2 v, float scale, float inverse) {
    return __nv_cvt_float2_to_fp8x2(make_float2(quotient(v.x, scale, inverse), quotient(v.y, scale, inverse)),
                                    __NV_SATFINITE, __NV_E4M3);
}

// Rows of 16-bit values T2 (pairs) written as fp8 codes: each piece is 16
// values where the addresses allow (kVec), else one.
template <typename T2, bool kVec>
__global__ void __launch_bounds__(kRowThreads) lmc_append_e4m3_kernel(const __grid_constant__ AppendPlan P) {
    __shared__ const uint8_t *src[kMaxRows];
    __shared__ uint8_t *dst[kMaxRows];
    lmc::wait_for_launch();
    lmc::let_next_start();
    const int n = resolve_append(P, src, dst);
    const uint32_t total = (uint32_t)n * P.pieces.d;
    if constexpr (kVec) {
        // the loads of several pieces before the first is turned to codes
        for (uint32_t first = threadIdx.x; first < total; first += kRowThreads * kCodeUnroll) {
            uint4 in[kCodeUnroll][2];
            uint4 *to[kCodeUnroll];
#pragma unroll
            for (int u = 0; u < kCodeUnroll; u++) {
                const uint32_t i = first + u * kRowThreads;
                to[u] = nullptr;
                if (i < total) {
                    uint32_t at;
                    const uint32_t row = divide(i, P.pieces, at);
                    if (src[row] != nullptr) {
                        const uint4 *s = reinterpret_cast<const uint4 *>(src[row]) + 2 * (size_t)at;
                        in[u][0] = __ldcs(s);
                        in[u][1] = __ldcs(s + 1);
                        to[u] = reinterpret_cast<uint4 *>(dst[row]) + at;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kCodeUnroll; u++) {
                if (to[u] == nullptr)
                    continue;
                const T2 *x = reinterpret_cast<const T2 *>(in[u]);
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; k++)
                    w[k] = codes2(to_float2(x[2 * k]), P.scale, P.inverse) | codes2(to_float2(x[2 * k + 1]), P.scale, P.inverse) << 16;
                __stcs(to[u], make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    } else {
        for (uint32_t i = threadIdx.x; i < total; i += kRowThreads) {
            uint32_t at;
            const uint32_t row = divide(i, P.pieces, at);
            if (src[row] == nullptr)
                continue;
            // a row may hold an odd number of values, on any 2-byte boundary
            T2 x;
            reinterpret_cast<uint16_t *>(&x)[0] = reinterpret_cast<const uint16_t *>(src[row])[at];
            reinterpret_cast<uint16_t *>(&x)[1] = 0;
            dst[row][at] = (uint8_t)codes2(to_float2(x), P.scale, P.inverse);
        }
    }
}

// ---------------------------------------------------------------------------
// Move
// ---------------------------------------------------------------------------

struct MovePlan {
    Pages pages;            // of the group's first layer
    int64_t layer_stride;   // pool bytes between the group's layers
    TokenTable src, dst;
    const int32_t *kept;
    int64_t set_stride;     // 0: one set for all layers
    int64_t request_stride;
    const int32_t *kept_lengths;
    int64_t max_kept;
    uint8_t *pool;
    uint32_t *status;
    int32_t num_requests;
    int32_t rows_per_cta;
    int64_t ctas_per_request;
    Divider pieces;
};

template <typename V>
__global__ void __launch_bounds__(kRowThreads) lmc_move_kernel(const __grid_constant__ MovePlan P) {
    __shared__ const uint8_t *src[kMaxRows];
    __shared__ uint8_t *dst[kMaxRows];
    const int64_t part = blockIdx.x % P.ctas_per_request;
    const int64_t unit = blockIdx.x / P.ctas_per_request;
    const int64_t req = unit % P.num_requests;
    const int64_t layer = unit / P.num_requests;
    lmc::wait_for_launch();
    lmc::let_next_start();
    const int64_t kept = __ldca(P.kept_lengths + req);
    if (kept < 0 || kept > P.max_kept) {
        if (threadIdx.x == 0)
            atomicOr(P.status, LMC_ST_BAD_JOB);
        return;
    }
    const int64_t first = part * P.rows_per_cta;
    if (first >= kept)
        return;
    const int n = (int)min((int64_t)P.rows_per_cta, kept - first);
    if ((int)threadIdx.x < n) {
        const int64_t j = first + threadIdx.x;
        uint32_t bad = 0;
        const int64_t from = entry_offset(P.pages, P.src, req,
                                          __ldca(P.kept + layer * P.set_stride + req * P.request_stride + j), bad);
        const int64_t to = entry_offset(P.pages, P.dst, req, (int32_t)j, bad);
        if (bad)
            atomicOr(P.status, bad);
        const bool ok = from >= 0 && to >= 0;
        src[threadIdx.x] = ok ? P.pool + layer * P.layer_stride + from : nullptr;
        dst[threadIdx.x] = P.pool + layer * P.layer_stride + to;
    }
    __syncthreads();
    copy_rows<V>(src, dst, n, P.pieces);
}

// ---------------------------------------------------------------------------
// Select
// ---------------------------------------------------------------------------

// The `take` highest of a row's candidates, found by their binary32 patterns
// mapped to unsigned keys of the same order, eight bits at a time from the
// top: a histogram of the keys that still match the threshold's known bits
// gives its next eight. A row is shared by the CTAs of a cluster, which read
// one another's histograms through distributed shared memory; each keeps its
// part of the keys in its own shared memory (kCached), so the scores are read
// from HBM once. The floor is that read (75 MB for 96 rows of 131072 with what
// is written: 11 us); the work is bound by instructions, so keys are taken
// four at a time, the first histogram is made while they are loaded, and a
// pass stops the search as soon as a bin is taken whole. The histogram has
// eight columns, by lane: scores share few exponents, and one counter per bin
// would serialise a warp's increments. Then each warp walks its own run of
// tokens in order, and a token's place among the kept is the number kept
// before it: a scan over the lanes adds up four blocks of 128 keys at once (a
// byte each; by ballots and their bit counts it took 56 us, this 54).
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;
constexpr int kSelColumns = 8;
constexpr int kSelBlocks = 4;  // of 128 keys, counted at once by a warp at the end
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSelPerSm = 3;  // CTAs an SM holds (96 rows of 131072: two take 1.4 times as long, four 1.05: they spill)

struct SelectPlan {
    const float *scores;
    int64_t set_stride, request_stride;
    const int32_t *lengths;
    int64_t max_length;
    int32_t *kept;
    float *kept_scores;
    int32_t *kept_lengths;
    uint32_t *status;
    int32_t budget, recent;
    int32_t num_requests;
    int32_t cluster;
};

// Keeps the order of the scores; NaN below every number, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));  // -0 becomes 0
    return x != x ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The score of a key, but for the two that more than one pattern maps to.
__device__ __forceinline__ bool key_score(uint32_t key, float &x) {
    x = __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
    return key != 0u && key != 0x80000000u;
}

struct alignas(16) SelectShared {
    union {
        uint32_t hist[256 * kSelColumns];
        uint32_t all[256];                // the cluster's totals, once hist is summed
        uint16_t picked[kSelWarps][256];  // at the end: positions a warp takes of 256
    };
    uint32_t totals[2][256];              // this CTA's, read by the cluster
    uint32_t warp_above[kSelWarps];
    uint32_t warp_equal[kSelWarps];
    uint32_t counts[2];            // this CTA's kept-for-sure and threshold keys
    uint32_t found[3];             // the pass's bin, what is left to take in it, its keys
};

// Four keys of a thread: positions 4 i .. 4 i + 3 of the CTA's part. Past its
// end a key reads 0, the lowest there is: such keys take part in the search
// (only the row's last part has any, so they come after every real one; take
// is less than the real ones' number, so none is ever reached).
template <bool kCached>
__device__ __forceinline__ uint4 keys_at(const uint32_t *keys, const float *score, int32_t i, int32_t mine) {
    if constexpr (kCached) {
        return reinterpret_cast<const uint4 *>(keys)[i];
    } else {
        uint32_t k[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            k[j] = 4 * i + j < mine ? order_key(__ldca(score + 4 * i + j)) : 0u;
        return make_uint4(k[0], k[1], k[2], k[3]);
    }
}

template <bool kCached>
__global__ void __launch_bounds__(kSelThreads, kSelPerSm) lmc_select_kernel(const __grid_constant__ SelectPlan P) {
    extern __shared__ __align__(16) uint8_t select_mem[];
    SelectShared &S = *reinterpret_cast<SelectShared *>(select_mem);
    uint32_t *const keys = reinterpret_cast<uint32_t *>(select_mem + sizeof(SelectShared));
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / P.cluster;
    const int64_t set = row / P.num_requests, req = row % P.num_requests;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    lmc::wait_for_launch();
    lmc::let_next_start();
    // uniform over the cluster, so leaving here leaves no CTA waiting
    const int64_t L = __ldca(P.lengths + req);
    if (L < 0 || L > P.max_length) {
        if (rank == 0 && tid == 0)
            atomicOr(P.status, LMC_ST_BAD_JOB);
        return;
    }
    if (set == 0 && rank == 0 && tid == 0)
        P.kept_lengths[req] = (int32_t)min(L, (int64_t)P.budget);
    const float *const score = P.scores + set * P.set_stride + req * P.request_stride;
    int32_t *const kept = P.kept + row * P.budget;
    float *const kept_scores = P.kept_scores == nullptr ? nullptr : P.kept_scores + row * P.budget;
    const int64_t step = (int64_t)P.cluster * kSelThreads;
    if (L <= P.budget) {
        for (int64_t t = (int64_t)rank * kSelThreads + tid; t < L; t += step) {
            kept[t] = (int32_t)t;
            if (kept_scores != nullptr)
                kept_scores[t] = score[t];
        }
        return;
    }
    const int32_t n = (int32_t)L - P.recent;      // candidates: [0, n)
    const int32_t take = P.budget - P.recent;     // 0 <= take < n
    for (int32_t j = rank * kSelThreads + tid; j < P.recent; j += (int32_t)step) {
        kept[take + j] = n + j;
        if (kept_scores != nullptr)
            kept_scores[take + j] = score[n + j];
    }
    if (take == 0)
        return;

    // this CTA's candidates (a multiple of four but for the last), in fours
    const int32_t part = (int32_t)((((int64_t)n + P.cluster - 1) / P.cluster + 3) / 4 * 4);
    const int32_t lo = (int32_t)min((int64_t)rank * part, (int64_t)n);
    const int32_t mine = (int32_t)min((int64_t)lo + part, (int64_t)n) - lo;
    const int32_t fours = (mine + 3) / 4;
    const bool wide = (((uintptr_t)(score + lo)) & 15) == 0;
    const int column = lane & (kSelColumns - 1);

    uint32_t prefix = 0, mask = 0, left = (uint32_t)take;
    bool whole = false;
    for (int pass = 0; pass < 4; pass++) {
        const int shift = 24 - 8 * pass, buf = pass & 1;
        for (int i = tid; i < 64 * kSelColumns; i += kSelThreads)
            reinterpret_cast<uint4 *>(S.hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint32_t *const bins = S.hist + column;
        const uint32_t bins_at = (uint32_t)__cvta_generic_to_shared(bins), last = ~mask;
        // a key that matches differs from the prefix in the unknown bits only;
        // predicated, for a branch per key costs twice the rest
        auto count = [&](uint32_t k) {
            const uint32_t t = k ^ prefix;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.le.u32 p, %0, %1;\n\t"
                "@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(t),
                "r"(last), "r"(bins_at + (t >> shift) * (4 * kSelColumns))
                : "memory");
        };
        if (kCached && pass == 0) {
            const float4 *const four = reinterpret_cast<const float4 *>(score + lo);
            const int32_t full = wide ? mine / 4 : 0;
#pragma unroll 4
            for (int32_t i = tid; i < full; i += kSelThreads) {
                const float4 x = __ldcs(four + i);
                const uint4 k = make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
                reinterpret_cast<uint4 *>(keys)[i] = k;
                atomicAdd(bins + (k.x >> 24) * kSelColumns, 1u);
                atomicAdd(bins + (k.y >> 24) * kSelColumns, 1u);
                atomicAdd(bins + (k.z >> 24) * kSelColumns, 1u);
                atomicAdd(bins + (k.w >> 24) * kSelColumns, 1u);
            }
            for (int32_t i = 4 * full + tid; i < 4 * fours; i += kSelThreads) {
                const uint32_t k = i < mine ? order_key(score[lo + i]) : 0u;
                keys[i] = k;
                atomicAdd(bins + (k >> 24) * kSelColumns, 1u);
            }
        } else {
#pragma unroll 4
            for (int32_t i = tid; i < fours; i += kSelThreads) {
                const uint4 k = keys_at<kCached>(keys, score + lo, i, mine);
                count(k.x);
                count(k.y);
                count(k.z);
                count(k.w);
            }
        }
        __syncthreads();
        if (tid < 256) {
            const uint4 *h = reinterpret_cast<const uint4 *>(S.hist + tid * kSelColumns);
            uint32_t sum = 0;
#pragma unroll
            for (int j = 0; j < kSelColumns / 4; j++) {
                const uint4 x = h[(j + (tid >> 2)) & (kSelColumns / 4 - 1)];
                sum += x.x + x.y + x.z + x.w;
            }
            S.totals[buf][tid] = sum;
        }
        cluster.sync();  // also a barrier of this CTA
        if (tid < 256) {
            // (all CTAs' reads in flight at once)
            uint32_t sum = 0;
#pragma unroll
            for (int c = 0; c < kSelMaxCluster; c++)
                if (c < P.cluster)
                    sum += cluster.map_shared_rank(&S.totals[buf][0], c)[tid];
            S.all[tid] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds bins [8 l', 8 l' + 8) counted from the top
            const int top = 255 - 8 * lane;
            uint32_t sum = 0;
#pragma unroll
            for (int j = 0; j < 8; j++)
                sum += S.all[top - j];
            uint32_t before = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o)
                    before += x;
            }
            before -= sum;
            if (before < left && left <= before + sum) {
                for (int j = 0; j < 8; j++) {
                    const uint32_t c = S.all[top - j];
                    if (left <= before + c) {
                        S.found[0] = (uint32_t)(top - j);
                        S.found[1] = left - before;
                        S.found[2] = c;
                        break;
                    }
                    before += c;
                }
            }
        }
        __syncthreads();
        const uint32_t bin = S.found[0], in_bin = S.found[2];
        left = S.found[1];
        prefix |= bin << shift;
        mask |= 255u << shift;
        whole = in_bin == left;
        if (whole)
            break;  // the lower bits do not matter (uniform over the cluster)
    }

    // Keys above `high` are taken. Where the last bin was taken whole that is
    // all; else (equal scores at the border) also the first `left` of the keys
    // from `prefix` to `high`.
    const uint32_t high = whole ? prefix - 1u : prefix | ~mask;
    const int32_t run = (fours + kSelWarps - 1) / kSelWarps;
    const int32_t w0 = min(warp * run, fours), w1 = min(w0 + run, fours);
    uint32_t above = 0, equal = 0;
#pragma unroll 4
    for (int32_t i = w0 + lane; i < w1; i += 32) {
        const uint4 k = keys_at<kCached>(keys, score + lo, i, mine);
        const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            above += v[j] > high;
            if (!whole)
                equal += v[j] >= prefix;
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = whole ? 0u : __reduce_add_sync(0xffffffffu, equal) - above;
    if (lane == 0) {
        S.warp_above[warp] = above;
        S.warp_equal[warp] = equal;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t x = lane < kSelWarps ? S.warp_above[lane] : 0u, y = lane < kSelWarps ? S.warp_equal[lane] : 0u;
        uint32_t a = x, e = y;
        for (int o = 1; o < kSelWarps; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, a, o), w = __shfl_up_sync(0xffffffffu, e, o);
            if (lane >= o) {
                a += u;
                e += w;
            }
        }
        if (lane < kSelWarps) {
            S.warp_above[lane] = a - x;
            S.warp_equal[lane] = e - y;
        }
        if (lane == kSelWarps - 1) {
            S.counts[0] = a;
            S.counts[1] = e;
        }
    }
    cluster.sync();
    uint32_t a_before = S.warp_above[warp], e_before = S.warp_equal[warp];
#pragma unroll
    for (int c = 0; c < kSelMaxCluster - 1; c++)
        if (c < rank) {
            const uint32_t *other = cluster.map_shared_rank(&S.counts[0], c);
            a_before += other[0];
            e_before += other[1];
        }
    uint16_t *const picked = S.picked[warp];
    auto write = [&](int32_t at0, uint32_t first, int32_t picks) {
        int32_t *const to = kept + first;
        for (int32_t q = lane; q < picks; q += 32) {
            const int32_t at = at0 + picked[q];
            to[q] = lo + at;
            if (kept_scores != nullptr) {
                float x = 0.0f;
                if (!kCached || !key_score(keys[at], x))
                    x = score[lo + at];
                kept_scores[first + q] = x;
            }
        }
        __syncwarp();
    };
    for (int32_t i0 = w0; i0 < w1; i0 += 32 * kSelBlocks) {
        // a lane's picks of kSelBlocks blocks of 128 keys, a byte each, summed
        // over the lanes below at once
        auto four = [&](int block) {
            const int32_t i = i0 + 32 * block + lane;
            return i < w1 ? keys_at<kCached>(keys, score + lo, i, mine) : make_uint4(0, 0, 0, 0);
        };
        auto sum_lanes = [&](uint32_t x) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                x += lane >= o ? y : 0u;
            }
            return x;
        };
        uint32_t a_mine = 0;
#pragma unroll
        for (int block = 0; block < kSelBlocks; block++) {
            const uint4 k = four(block);
            const uint32_t n = (k.x > high) + (k.y > high) + (k.z > high) + (k.w > high);
            a_mine += n << (8 * block);
        }
        const uint32_t a_sum = sum_lanes(a_mine), a_all = __shfl_sync(0xffffffffu, a_sum, 31);
        if (whole) {
#pragma unroll
            for (int pair = 0; pair < kSelBlocks; pair += 2) {
                // the warp's picks of two blocks, close together, then written as one run
                uint32_t picks = 0;
#pragma unroll
                for (int block = pair; block < pair + 2; block++) {
                    const uint4 k = four(block);
                    const uint32_t v[4] = {k.x, k.y, k.z, k.w};
                    uint16_t *to = picked + picks + ((a_sum - a_mine) >> (8 * block) & 255u);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (v[j] > high)
                            *to++ = (uint16_t)(4 * (32 * block + lane) + j);
                    picks += a_all >> (8 * block) & 255u;
                }
                __syncwarp();
                write(4 * i0, a_before, (int32_t)picks);
                a_before += picks;
            }
            continue;
        }
        uint32_t e_mine = 0;
#pragma unroll
        for (int block = 0; block < kSelBlocks; block++) {
            const uint4 k = four(block);
            const uint32_t n = (k.x >= prefix) + (k.y >= prefix) + (k.z >= prefix) + (k.w >= prefix);
            e_mine += (i0 + 32 * block + lane < w1 ? n : 0u) << (8 * block);
        }
        e_mine -= a_mine;
        const uint32_t e_sum = sum_lanes(e_mine), e_all = __shfl_sync(0xffffffffu, e_sum, 31);
#pragma unroll 1
        for (int block = 0; block < kSelBlocks; block++) {
            const uint32_t first = a_before + min(e_before, left);
            const uint4 k = four(block);
            const uint32_t v[4] = {k.x, k.y, k.z, k.w};
            const bool real = i0 + 32 * block + lane < w1;
            uint32_t a_at = a_before + ((a_sum - a_mine) >> (8 * block) & 255u);
            uint32_t e_at = e_before + ((e_sum - e_mine) >> (8 * block) & 255u);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool a = v[j] > high, e = real && v[j] >= prefix && !a;
                if (a || (e && e_at < left))
                    picked[a_at + min(e_at, left) - first] = (uint16_t)(4 * (32 * block + lane) + j);
                a_at += a;
                e_at += e;
            }
            a_before += a_all >> (8 * block) & 255u;
            e_before += e_all >> (8 * block) & 255u;
            __syncwarp();
            write(4 * i0, first, (int32_t)(a_before + min(e_before, left) - first));
        }
    }
    cluster.sync();  // no CTA leaves while another may read its counts
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

TokenTable token_table(const lmc_block_table &t) { return TokenTable{t.table, t.row_stride, (int32_t)t.num_cols}; }

// Rows a CTA takes (up to 16 pieces per thread), and the division by a row's
// pieces.
int rows_per_cta(int64_t pieces, Divider &D) {
    const int rows = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRows, kRowThreads * 16 / pieces));
    D.d = (uint32_t)pieces;
    D.m = rows == 1 ? 1u : pieces == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + D.d - 1) / D.d);
    return rows;
}

template <typename Plan>
int launched(void (*kern)(Plan), int64_t grid, cudaStream_t stream, const Plan &P) {
    return lmc::follow(kern, dim3((unsigned)grid), kRowThreads, 0, stream, P) ? LMC_OK : LMC_ERR_CUDA;
}

// The widest piece (16, 4 or 1 bytes) that every one of the values is a multiple of.
int piece_bytes(std::initializer_list<int64_t> values) {
    int64_t all = 0;
    for (int64_t v : values)
        all |= v;
    return (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
}

// Bytes [at, end) of 4-byte elements that a call reads or writes.
struct Extent {
    uint64_t at, end;
    bool meets(const Extent &o) const { return std::max(at, o.at) < std::min(end, o.end); }
};
Extent extent(const void *p, int64_t elements) {
    return Extent{(uint64_t)(uintptr_t)p, (uint64_t)(uintptr_t)p + (p == nullptr ? 0 : 4 * (uint64_t)elements)};
}

}  // namespace

namespace lmc {

int check_entries(const lmc_layout *L, const lmc_entries *e) {
    if (L == nullptr || e == nullptr || e->layer < 0 || (size_t)e->layer >= L->desc.size())
        return LMC_ERR_INVALID_ARG;
    const lmc_layer_spec &spec = L->specs[e->layer];
    const int elem = entry_elem_bytes(e->dtype);
    if (spec.kind == LMC_LAYER_KDA || elem == 0 || e->entry_dim <= 0 ||
        spec.token_bytes != (int64_t)e->entry_dim * elem || e->num_requests < 0 || L->block_size > INT32_MAX ||
        spec.token_bytes > INT32_MAX / 2)
        return LMC_ERR_INVALID_ARG;
    if (!std::isfinite(e->scale) || e->scale <= 0.0f || (e->dtype != LMC_E_E4M3 && e->scale != 1.0f))
        return LMC_ERR_INVALID_ARG;
    return table_ok(e->table, e->num_requests) ? LMC_OK : LMC_ERR_INVALID_ARG;
}

}  // namespace lmc

extern "C" int lmc_append(const lmc_layout *L, const lmc_entries *e, void *pool, const int32_t *requests,
                          const int32_t *positions, const void *rows, int32_t rows_dtype, int64_t row_stride,
                          int64_t num_rows, uint32_t *status, void *stream) {
    if (const int rc = lmc::check_entries(L, e); rc != LMC_OK)
        return rc;
    if (status == nullptr || num_rows < 0 || (rows_dtype != LMC_E_BF16 && rows_dtype != LMC_E_F16) ||
        (e->dtype != LMC_E_E4M3 && e->dtype != rows_dtype) || row_stride < e->entry_dim ||
        row_stride > INT64_MAX / 2)
        return LMC_ERR_INVALID_ARG;
    if (num_rows > 0 && (pool == nullptr || requests == nullptr || positions == nullptr || rows == nullptr))
        return LMC_ERR_INVALID_ARG;
    if ((((uintptr_t)status | (uintptr_t)requests | (uintptr_t)positions) & 3) != 0 || ((uintptr_t)rows & 1) != 0)
        return LMC_ERR_ALIGN;
    if (num_rows == 0)
        return LMC_OK;
    const lmc_layer_desc &d = L->desc[e->layer];
    const int64_t tb = L->specs[e->layer].token_bytes;
    AppendPlan P;
    P.pages = Pages{d.base, d.stride, L->num_blocks, (int32_t)L->block_size, (int32_t)tb};
    P.table = token_table(e->table);
    P.requests = requests;
    P.positions = positions;
    P.rows = static_cast<const uint8_t *>(rows);
    P.row_bytes = row_stride * 2;
    P.pool = static_cast<uint8_t *>(pool);
    P.status = status;
    P.num_rows = num_rows;
    P.num_requests = e->num_requests;
    P.scale = e->scale;
    uint32_t bits;
    std::memcpy(&bits, &P.scale, 4);
    P.inverse = P.scale >= 0x1p-100f && P.scale <= 0x1p100f && (bits & 0x7fffffu) != 0x7fffffu ? 1.0f / P.scale : 0.0f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int wide = piece_bytes({(int64_t)(uintptr_t)pool, d.base, d.stride, tb, (int64_t)(uintptr_t)rows,
                                  P.row_bytes});
    if (e->dtype == LMC_E_E4M3) {
        const bool vec = wide == 16 && e->entry_dim % 16 == 0;
        const int64_t pieces = vec ? e->entry_dim / 16 : e->entry_dim;
        P.rows_per_cta = rows_per_cta(pieces, P.pieces);
        const int64_t grid = (num_rows + P.rows_per_cta - 1) / P.rows_per_cta;
        if (grid > INT32_MAX)
            return LMC_ERR_INVALID_ARG;
        auto kern = rows_dtype == LMC_E_BF16
                        ? (vec ? lmc_append_e4m3_kernel<__nv_bfloat162, true> : lmc_append_e4m3_kernel<__nv_bfloat162, false>)
                        : (vec ? lmc_append_e4m3_kernel<__half2, true> : lmc_append_e4m3_kernel<__half2, false>);
        return launched(kern, grid, s, P);
    }
    P.rows_per_cta = rows_per_cta(tb / wide, P.pieces);
    const int64_t grid = (num_rows + P.rows_per_cta - 1) / P.rows_per_cta;
    if (grid > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    auto kern = wide == 16 ? lmc_append_kernel<uint4> : wide == 4 ? lmc_append_kernel<uint32_t> : lmc_append_kernel<uint8_t>;
    return launched(kern, grid, s, P);
}

extern "C" int lmc_move_tokens(const lmc_layout *L, int32_t kv_group, void *pool, int32_t num_requests,
                               const lmc_block_table *src, const lmc_block_table *dst, const int32_t *kept,
                               int32_t num_sets, int64_t set_stride, int64_t request_stride,
                               const int32_t *kept_lengths, int64_t max_kept, uint32_t *status, void *stream) {
    if (L == nullptr || kv_group < 0 || (size_t)kv_group >= L->kv_group_kind.size() ||
        L->kv_group_kind[kv_group] == LMC_LAYER_KDA || src == nullptr || dst == nullptr || status == nullptr ||
        num_requests < 0 || max_kept < 0 || max_kept > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    const int32_t layers = L->kv_group_size[kv_group];
    if ((num_sets != 1 && num_sets != layers) || set_stride < 0 || request_stride < max_kept ||
        !lmc::table_ok(*src, num_requests) || !lmc::table_ok(*dst, num_requests))
        return LMC_ERR_INVALID_ARG;
    if (((uintptr_t)status & 3) != 0 || (((uintptr_t)kept | (uintptr_t)kept_lengths) & 3) != 0)
        return LMC_ERR_ALIGN;
    if (num_requests == 0 || max_kept == 0)
        return LMC_OK;
    if (pool == nullptr || kept == nullptr || kept_lengths == nullptr)
        return LMC_ERR_INVALID_ARG;
    if (src->table != nullptr && src->table == dst->table)
        return LMC_ERR_OVERLAP;
    // the group's layers have one page size each and lie evenly spaced
    // (padded: one slab apart; packed: one page apart)
    int64_t first = -1, second = -1;
    int32_t layer = -1;
    for (size_t i = 0; i < L->desc.size(); i++)
        if (L->desc[i].kv_group == kv_group) {
            if (L->desc[i].slot == 0) {
                first = L->desc[i].base;
                layer = (int32_t)i;
            } else if (L->desc[i].slot == 1) {
                second = L->desc[i].base;
            }
        }
    const lmc_layer_desc &d = L->desc[layer];
    const int64_t tb = L->specs[layer].token_bytes;
    if (L->block_size > INT32_MAX || tb > INT32_MAX / 2)
        return LMC_ERR_INVALID_ARG;
    MovePlan P;
    P.pages = Pages{first, d.stride, L->num_blocks, (int32_t)L->block_size, (int32_t)tb};
    P.layer_stride = layers > 1 ? second - first : 0;
    P.src = token_table(*src);
    P.dst = token_table(*dst);
    P.kept = kept;
    P.set_stride = num_sets == 1 ? 0 : set_stride;
    P.request_stride = request_stride;
    P.kept_lengths = kept_lengths;
    P.max_kept = max_kept;
    P.pool = static_cast<uint8_t *>(pool);
    P.status = status;
    P.num_requests = num_requests;
    const int wide = piece_bytes({(int64_t)(uintptr_t)pool, first, d.stride, P.layer_stride, tb});
    P.rows_per_cta = rows_per_cta(tb / wide, P.pieces);
    P.ctas_per_request = (max_kept + P.rows_per_cta - 1) / P.rows_per_cta;
    int64_t grid;
    if (!lmc::mul_ok(P.ctas_per_request, (int64_t)num_requests * layers, &grid) || grid > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    auto kern = wide == 16 ? lmc_move_kernel<uint4> : wide == 4 ? lmc_move_kernel<uint32_t> : lmc_move_kernel<uint8_t>;
    return launched(kern, grid, static_cast<cudaStream_t>(stream), P);
}

extern "C" int lmc_select_tokens(const float *scores, int64_t set_stride, int64_t request_stride, int32_t num_sets,
                                 int32_t num_requests, const int32_t *lengths, int64_t max_length, int64_t budget,
                                 int64_t recent, int32_t *kept, float *kept_scores, int32_t *kept_lengths,
                                 uint32_t *status, void *stream) {
    if (num_sets < 0 || num_requests < 0 || max_length < 0 || max_length > INT32_MAX || budget < 0 ||
        budget > INT32_MAX || recent < 0 || recent > budget || set_stride < 0 || request_stride < 0 ||
        status == nullptr)
        return LMC_ERR_INVALID_ARG;
    if ((((uintptr_t)scores | (uintptr_t)lengths | (uintptr_t)kept | (uintptr_t)kept_scores | (uintptr_t)kept_lengths |
          (uintptr_t)status) & 3) != 0)
        return LMC_ERR_ALIGN;
    if (num_sets == 0 || num_requests == 0)
        return LMC_OK;
    if (lengths == nullptr || kept_lengths == nullptr || (scores == nullptr && max_length > 0) ||
        (kept == nullptr && budget > 0))
        return LMC_ERR_INVALID_ARG;
    // A row is read by several CTAs, its length by those of every set: neither
    // may be written meanwhile.
    const int64_t rows = (int64_t)num_sets * num_requests;
    int64_t sets_end, requests_end, kept_count;
    if (!lmc::mul_ok(set_stride, num_sets - 1, &sets_end) || !lmc::mul_ok(request_stride, num_requests - 1, &requests_end) ||
        !lmc::add_ok(sets_end, requests_end, &sets_end) || sets_end > INT64_MAX / 8 || !lmc::mul_ok(rows, budget, &kept_count) ||
        kept_count > INT64_MAX / 8)
        return LMC_ERR_OVERFLOW;
    const Extent in[2] = {extent(scores, max_length > 0 ? sets_end + max_length : 0), extent(lengths, num_requests)};
    const Extent out[3] = {extent(kept, kept_count), extent(kept_scores, kept_count), extent(kept_lengths, num_requests)};
    for (int i = 0; i < 3; i++)
        if (out[i].meets(in[0]) || out[i].meets(in[1]) || out[i].meets(out[(i + 1) % 3]))
            return LMC_ERR_OVERLAP;
    const int sms = lmc::sm_count();
    if (sms <= 0)
        return LMC_ERR_CUDA;
    SelectPlan P;
    P.scores = scores;
    P.set_stride = set_stride;
    P.request_stride = request_stride;
    P.lengths = lengths;
    P.max_length = max_length;
    P.kept = kept;
    P.kept_scores = kept_scores;
    P.kept_lengths = kept_lengths;
    P.status = status;
    P.budget = (int32_t)budget;
    P.recent = (int32_t)recent;
    P.num_requests = num_requests;
    // 16384 keys (64 KB) per CTA let three CTAs share an SM; fewer where there
    // are not enough rows for all SMs. Eight CTAs a row is the most there is: above
    // some 132700 tokens two of their parts fit an SM, above some 210000 one (96
    // rows of 132000 scores 53.0 us, of 133500 63.3, of 196608 80.9, of 262144
    // 160.6), and above some 444000 the scores are read again for every pass
    int c = 1;
    while (c < kSelMaxCluster &&
           (max_length > (int64_t)c * 16384 || (rows * c < sms && max_length > (int64_t)c * 2048)))
        c *= 2;
    P.cluster = c;
    const int64_t most = kSmemLimit - (int64_t)sizeof(SelectShared);
    const int64_t want = ((max_length + c - 1) / c + 7) / 4 * 16;  // a part is rounded up to fours
    const bool cached = want <= most;
    const size_t smem = sizeof(SelectShared) + (cached ? (size_t)(want + 15) / 16 * 16 : 0);
    if (rows * c > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    auto kern = cached ? lmc_select_kernel<true> : lmc_select_kernel<false>;
    static std::atomic<uint64_t> allowed[2];
    if (!lmc::allow_shared_memory(allowed[cached], kern, kSmemLimit))
        return LMC_ERR_CUDA;
    return lmc::follow(kern, dim3((unsigned)(rows * c)), kSelThreads, smem, static_cast<cudaStream_t>(stream), P,
                       (unsigned)c)
               ? LMC_OK
               : LMC_ERR_CUDA;
}
