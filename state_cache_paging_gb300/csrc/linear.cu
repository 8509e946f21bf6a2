// linear.cu -- linear attention with a decay for each head, its states in the pages
// of state layers, for sm_103a: a token per request, and prompts.
//
// Mathematics. S_t = exp(g_t) S_(t-1) + k_t v_t^T, out_t = scale S_t^T q_t. One
// token: as it stands. Prompts: for a tile of up to 64 tokens and G_t = g_1 + .. +
// g_t (from the state S before the tile, all of it turned: values down, tokens across),
//   out_t = scale (exp(G_t) S^T q_t + sum_(j <= t) exp(G_t - G_j) (q_t . k_j) v_j),
//   S' = exp(G_64) S + sum_j k_j (exp(G_64 - G_j) v_j)^T,
// four matrix products per tile: Q K^T, its weighted product with V, S^T Q^T and the
// update. What leaves a tile for the next is only S, in binary32.
//
// One token is bound by reading and writing the states: 256 requests of 32 heads of
// 128 x 128 take 166 us, 96 % of the measured copy rate. Prompts are bound by the
// instructions between the products: 32 requests of 8192 tokens of 32 heads in bf16
// take 1670 us, 82 % of what reading q, k and v and writing the results takes at the
// copy rate (in f16 some 55 %: binary32's range is brought into f16's row by row).
// What brought it there from 3245 us: one role per kind of work (a warp waits for
// nothing that it does not need), four exact bf16 parts of v instead of three truncated
// ones, loops that stay in the instruction cache, two binary32 operations an
// instruction, and results that leave by TMA.
//
// Long requests are cut where there are fewer heads than SMs: a first pass finds what
// each segment adds to the state (updates taking turns in two places of tensor memory:
// 347 us became 339), a second one joins them, and the third makes the results of all
// segments at once (131072 tokens of one request, 8 heads: 344 us, the first two passes
// some 145 of them). The first writes down whose segment it made in each place: a
// request is continued only from places that are all its own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

constexpr int kMaxDim = 128;
constexpr float kLeastDecay = -1000.0f;  // its exponential is 0 in binary32

struct LinearPlan {
    float *pages;        // the pool's first state of block 0
    int64_t page_stride; // floats between blocks
    int64_t num_blocks;
    const int32_t *table;
    int64_t row_stride;
    int64_t cols;
    const int32_t *lengths;
    const int32_t *starts;  // NULL: one row per request
    const uint16_t *q, *k, *v;
    uint16_t *out;
    const float *decay;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head, decay_row, decay_head;
    int64_t num_rows;
    uint32_t *status;
    int32_t R, H, shared;   // shared: heads of a key head
    int32_t dk, dv;
    int32_t block_size;
    int32_t bf16;
    float scale;
};

// A request's tokens of this call and the states before and after them.
struct Span {
    int64_t row;        // its first row
    int64_t before;     // tokens before
    int64_t count;      // its tokens; 0: nothing to do
    int32_t first;      // block of the state before them; -1: none
    int32_t last;       // block of the state after them
    uint32_t bad;       // status bits
};

// The larger one; NaN where x is.
__device__ __forceinline__ float fmaxf_nan(float x, float least) { return x < least ? least : x; }

__device__ __forceinline__ Span span_of(const LinearPlan &P, int r) {
    Span S;
    S.row = r;
    S.count = 1;
    S.first = S.last = -1;
    S.bad = 0;
    S.before = __ldca(P.lengths + r);
    if (P.starts != nullptr) {
        S.row = __ldca(P.starts + r);
        const int64_t end = __ldca(P.starts + r + 1);
        S.count = end - S.row;
        if (S.row < 0 || end > P.num_rows || S.count < 0)
            S.bad = LMC_ST_BAD_JOB;
    }
    if (S.bad == 0 && S.before != -1 && S.count > 0) {
        const int64_t last = S.before + S.count - 1;
        if (S.before < 0 || last / P.block_size >= P.cols) {
            S.bad = LMC_ST_BAD_JOB;
        } else {
            const int32_t *blocks = P.table + r * P.row_stride;
            S.last = __ldca(blocks + last / P.block_size);
            if (S.before > 0) {
                S.first = __ldca(blocks + (S.before - 1) / P.block_size);
                if (S.first < 0 || S.first >= P.num_blocks)
                    S.bad |= S.first == -1 ? LMC_ST_NO_SNAPSHOT : LMC_ST_BLOCK_OOR;
            }
            if (S.last < 0 || S.last >= P.num_blocks)
                S.bad |= S.last == -1 ? LMC_ST_NO_SNAPSHOT : LMC_ST_BLOCK_OOR;
        }
    }
    if (S.bad != 0 || S.before < 0)
        S.count = 0;
    return S;
}

// ---------------------------------------------------------------------------
// One token at a time
// ---------------------------------------------------------------------------

// A CTA holds 4 kLanes columns of a head's state in registers: kLanes lanes take a
// row's (four columns each), 256 / kLanes rows at a time. Bound by reading and
// writing the state: 2 x 64 KB for a head of 128 x 128, 2 KB of everything else.
constexpr int kStepThreads = 256;
constexpr int kStepLanes = 16;     // (256 requests of 32 heads of 128 x 128: 8 lanes 193 us, 16 167, 32 184)

template <int kLanes>
__global__ void __launch_bounds__(kStepThreads) lmc_linear_step_kernel(const __grid_constant__ LinearPlan P) {
    constexpr int kRows = kStepThreads / kLanes;   // at a time
    constexpr int kTurns = kMaxDim / kRows;
    __shared__ float qs[kMaxDim], ks[kMaxDim];
    __shared__ float4 sums[kRows][kLanes];
    const int parts = (P.dv + 4 * kLanes - 1) / (4 * kLanes);
    const int part = (int)(blockIdx.x % parts), h = (int)(blockIdx.x / parts % P.H);
    const int64_t r = blockIdx.x / parts / P.H;
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes, c = 4 * (part * kLanes + lane);
    wait_for_launch();
    let_next_start();
    const Span S = span_of(P, (int)r);
    if (S.bad && h == 0 && part == 0 && threadIdx.x == 0)
        atomicOr(P.status, S.bad);
    if (S.count == 0)
        return;
    const bool mine = c < P.dv;
    float4 s[kTurns] = {};
    const int64_t at = (int64_t)h * P.dk * P.dv + c;
    if (S.first >= 0 && mine) {
        const float *page = P.pages + S.first * P.page_stride + at;
#pragma unroll
        for (int i = 0; i < kTurns; i++)
            if (row + i * kRows < P.dk)
                s[i] = __ldcs(reinterpret_cast<const float4 *>(page + (int64_t)(row + i * kRows) * P.dv));
    }
    const int kh = h / P.shared;
    if ((int)threadIdx.x < P.dk)
        qs[threadIdx.x] = from_q(P.q[r * P.q_row + kh * P.q_head + threadIdx.x], P.bf16);
    else if (threadIdx.x >= kMaxDim && (int)threadIdx.x - kMaxDim < P.dk)
        ks[threadIdx.x - kMaxDim] = from_q(P.k[r * P.k_row + kh * P.k_head + threadIdx.x - kMaxDim], P.bf16);
    float4 v = {}, o = {};
    if (mine) {
        const uint2 w = *reinterpret_cast<const uint2 *>(P.v + r * P.v_row + h * P.v_head + c);
        v = make_float4(from_q(w.x & 0xffff, P.bf16), from_q(w.x >> 16, P.bf16), from_q(w.y & 0xffff, P.bf16),
                        from_q(w.y >> 16, P.bf16));
    }
    // a state that decays slowly keeps its own digits: s + (decay - 1) s (a decay
    // near 1 rounded to 24 bits would let it drift by 2^-25 a token)
    const float g = fmaxf_nan(P.decay[r * P.decay_row + h * P.decay_head], kLeastDecay);
    const bool slow = g > -0.5f && g < 0.5f;
    const float grow = slow ? expm1f(g) : expf(g), keep = slow ? 1.0f : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurns; i++) {
        const int j = row + i * kRows;
        if (j < P.dk) {
            const float k = ks[j], q = qs[j];
            s[i].x = fmaf(keep, s[i].x, fmaf(k, v.x, grow * s[i].x));
            s[i].y = fmaf(keep, s[i].y, fmaf(k, v.y, grow * s[i].y));
            s[i].z = fmaf(keep, s[i].z, fmaf(k, v.z, grow * s[i].z));
            s[i].w = fmaf(keep, s[i].w, fmaf(k, v.w, grow * s[i].w));
            o.x = fmaf(q, s[i].x, o.x);
            o.y = fmaf(q, s[i].y, o.y);
            o.z = fmaf(q, s[i].z, o.z);
            o.w = fmaf(q, s[i].w, o.w);
        }
    }
    if (mine) {
        float *page = P.pages + S.last * P.page_stride + at;
#pragma unroll
        for (int i = 0; i < kTurns; i++)
            if (row + i * kRows < P.dk)
                __stcs(reinterpret_cast<float4 *>(page + (int64_t)(row + i * kRows) * P.dv), s[i]);
    }
    sums[row][lane] = o;
    __syncthreads();
    const int col = part * 4 * kLanes + threadIdx.x;
    if (threadIdx.x < 4 * kLanes && col < P.dv) {
        float y = 0.0f;
#pragma unroll 8
        for (int i = 0; i < kRows; i++)
            y += reinterpret_cast<const float *>(sums[i])[threadIdx.x];
        P.out[r * P.out_row + h * P.out_head + col] = to_out(y * P.scale, P.bf16);
    }
}

// ---------------------------------------------------------------------------
// Prompts: 64 tokens at a time on the tensor cores
// ---------------------------------------------------------------------------

constexpr int kTile = 64;             // tokens of a tile, all of one block of a request
constexpr int kPanel = kTile * 128;   // bytes of 64 values of a tile's rows
constexpr int kStages = 4;
constexpr int kStageBytes = 6 * kPanel;  // q, k, v, two panels each
constexpr int kStateWarps = 8;
constexpr int kFirstPartWarp = 8, kPartWarps = 8;
constexpr int kFirstWeightWarp = 16, kWeightWarps = 4;
constexpr int kFirstResultWarp = 20, kResultWarps = 4;
constexpr int kLoadWarp = 24, kForwardWarp = 25, kStateProductWarp = 26, kDecayWarp = 27;
constexpr int kScanThreads = 28 * 32;
// Registers per thread of the warpgroups: 2 x 112 + 2 x 64 + 56 + 56 + 40 of the 7 x
// 72 the CTA starts with.
constexpr int kStateRegisters = 112, kPartRegisters = 64, kWeightRegisters = 56, kResultRegisters = 56, kOtherRegisters = 40;
static_assert(2 * kStateRegisters + 2 * kPartRegisters + kWeightRegisters + kResultRegisters + kOtherRegisters == 7 * 72,
              "a split of more registers than the CTA has would wait forever");
// shared memory behind the stages: the weights, the result on its way
constexpr int kWeightsAt = kStages * kStageBytes, kResultAt = kWeightsAt + kPanel;
constexpr int kWarpResult = kTile * 64;  // bytes of a warp's part of a result: 32 values of each token
constexpr int kScanMemory = kResultAt + kResultWarps * kWarpResult;
constexpr int kLooks = 1 << 17;   // at barriers in vain, of up to
constexpr uint32_t kLook = 20000;  // so many ns each
// columns of tensor memory
constexpr uint32_t kScores = 0, kUpdate = 64, kFromState = 192, kFromTile = 256, kState = 320, kParts = 384;
constexpr uint32_t kPartColumns = kTile / 2;
constexpr uint32_t kOtherUpdate = kFromState;  // where only states are made: updates in turns
constexpr int kRing = 4;              // tiles whose decays are at hand
constexpr int kSms = 152;
constexpr int64_t kLeastSegment = 512;  // tokens

struct ScanPlan {
    CUtensorMap q, k, v, out;
    LinearPlan L;
    int64_t segment;     // a request of n of these tokens (n >= 2) is cut into n segments
    float *slots;        // [num_rows / segment][H][dk][dv]: the states before segments
    float2 *totals;      // [num_rows / segment][H]: the decay over the segment before, in units of log 2 (high, low)
    int32_t *owners;     // [cuts]: the request whose segment the states pass made, -1: none
    int64_t cuts;        // num_rows / segment
    int32_t k_copies, v_copies, k_panels, v_panels;  // copies for all panels, panels
    int32_t wide_out;    // whole tiles of the result are written by TMA, others 16 bytes at a time
};

// A CTA's tokens: a segment of a request, one head.
struct Item {
    int32_t row;         // first row
    int32_t page;        // its block position,
    int32_t phase;       // and the tokens of the block before it
    int32_t count;       // tokens
    int32_t r, h;
    int32_t first;       // block of the state before them, -1: none
    int32_t last;        // block of the state after the request's
    int32_t slot;        // of the segment; -1: the request is not cut
    int32_t ends;        // the request ends with it
    int32_t work;
    int32_t tiles;
};

// What a tile's tokens' decays give.
struct alignas(16) Decays {
    float2 log[kTile];      // sum up to and with the token, in units of log 2 (high, low)
    uint4 left[kTile / 2];  // from the token to the tile's end, two tokens: three bf16 parts f2, f3, f1 with a 0 behind it; or (f16) as it is
    float since[kTile];     // from the tile's start up to the token, times the call's scale
    float lift[kTile];      // f16: what the token's weights were divided by
    float unit[kMaxDim];    // f16: what a value's row of v times its decay was divided by
    float grow;             // decay over the tile
};
static_assert(sizeof(Decays) % 16 == 0, "two tokens' logs are read at once");

struct ScanControl {
    uint64_t full[kStages], free[kStages];
    uint64_t decays_full[kRing];
    uint64_t unit_full[kRing], lift_full[2], down_full[2];  // f16
    uint64_t score_full, score_free;
    uint64_t weight_full, weight_free;
    uint64_t parts_full[2], parts_free[2];  // the lower and the upper parts
    uint64_t update_full[2], update_free[2];  // (one, but where only states are made)
    uint64_t state_full, state_free, out_full, out_free;
    uint64_t ended[2];
    uint32_t tmem;
    uint32_t gave_up;
    uint32_t tiles;      // that were asked for
    Item item;
    Decays decays[kRing];
    float row_top[2][kMaxDim];   // f16: largest of the state's rows, by halves;
    float down[2][kMaxDim];      // and what they were divided by, in turns
};

// The tiles of an item, in order; every role walks them by itself.
struct Tiles {
    int32_t done, total, phase, N;
    int32_t rows;        // of the current tile
    int32_t row, page;   // its first row; its block position
    bool block_ends;
    uint32_t n;

    __device__ __forceinline__ Tiles(const Item &I, int32_t block_size)
        : done(0), total(I.count), phase(I.phase), N(block_size), rows(0), row(I.row), page(I.page), block_ends(false),
          n(~0u) {}
    __device__ __forceinline__ bool next() {
        done += rows;
        row += rows;
        phase += rows;
        if (phase == N) {
            phase = 0;
            page += rows > 0;
        }
        if (done >= total)
            return false;
        rows = min(min(kTile, total - done), N - phase);
        block_ends = phase + rows == N;
        n++;
        return true;
    }
    __device__ __forceinline__ bool last() const { return done + rows == total; }
};

// The loops of all roles together have to stay in the SM's instruction cache: from
// some 40 KB on, instructions come at 0.38 a clock and scheduler (measured with
// loops of sums), and the call's time doubles. So loops are not unrolled where they
// need not be, and what is not expected lies behind.
//
// Waits for a phase. Each role has so many looks to waste altogether (each of up to
// kLook ns; hardly any wait takes two). When they run out it waits no more, runs to
// its end, and says so: no more copies are asked for, and the status word tells.
__device__ __forceinline__ void scan_wait(ScanControl &C, uint64_t *bar, uint32_t parity, int &looks) {
    uint32_t done;
    do {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity), "r"(kLook)
            : "memory");
        if (done == 0 && --looks < 0) {
            *(volatile uint32_t *)&C.gave_up = 1;
            return;
        }
    } while (done == 0);
}

// Products with descriptors given by their lower words (the upper one is the same for
// all of a kind: strides and swizzle): half of what has to be brought to uniform
// registers. The first with A from shared memory, the second from tensor memory.
constexpr uint32_t kMatrixUpper = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t lower(uint32_t addr, uint32_t leading) { return (addr >> 4 & 0x3FFF) | (leading >> 4) << 16; }
__device__ __forceinline__ void multiply(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kMatrixUpper)
        : "memory");
}
__device__ __forceinline__ void multiply_held(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kMatrixUpper)
        : "memory");
}

// A box of the result, of a tile's rows and 32 values, to (x, row y, head w). Its
// rows lie in shared memory as the map's 64-byte swizzle has them.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int x, int y, int w) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
                 "r"(x), "r"(y), "r"(0), "r"(w), "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Rows of two panels behind a tile's last one, cleared by `threads` threads: they
// belong to others, and take part in products times 0, which infinities and NaN
// would not bear. `twice`: or that take the tile's rows a second time, half a tile on.
__device__ __forceinline__ void clear_rows(uint8_t *panels, int rows, int tid, int threads, bool twice = false) {
    constexpr int kHalf = kTile / 2;
#pragma unroll 1
    for (int c = tid; c < 2 * (kPanel / 16); c += threads) {
        const int row = c >> 3 & (kTile - 1);
        uint4 *const at = reinterpret_cast<uint4 *>(panels + c * 16);
        if (row >= rows)
            *at = twice && row >= kHalf && row - kHalf < rows ? at[-kHalf * 8] : make_uint4(0, 0, 0, 0);
    }
}

// 16 lanes x 16 columns, as load_s.
__device__ __forceinline__ void load_s8(uint32_t (&s)[8], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7])
                 : "r"(addr)
                 : "memory");
}

// 32 lanes x 8 columns: a lane's row.
__device__ __forceinline__ void load_o8(uint32_t (&o)[8], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void store_o8(const uint32_t (&o)[8], uint32_t addr) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(o[0]), "r"(o[1]),
                 "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(addr)
                 : "memory");
}

// Four 8 x 8 matrices of 16 bits, turned: a lane gives one of their rows'
// addresses and gets row l / 4, columns 2 (l % 4) and the next, of each column by
// column.
__device__ __forceinline__ void load_turned(uint32_t *v, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void store_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
// 16 lanes x 16 columns of tensor memory: lane l of the warp holds rows l / 4
// (v[2 i]) and l / 4 + 8 (v[2 i + 1]), column 4 i + l % 4.
__device__ __forceinline__ void store_part(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t plus_product(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t minus(uint32_t a) {
    uint32_t r;
    asm("neg.bf16x2 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// 2^e for e in [-126, 127], and the e that brings x into [2^14, 2^15).
// The greatest of a >= 0, |x| and |y|.
__device__ __forceinline__ float greatest(float a, float x, float y) {
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(x), "f"(y));
    return a;
}
// a - b
__device__ __forceinline__ float2 less(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a); }
__device__ __forceinline__ float2 from_halves(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float inverse_power(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }
__device__ __forceinline__ int lift_of(float x) {
    const int e = (int)(__float_as_uint(x) >> 23 & 255u) - 127;  // x >= 0
    return x == 0.0f ? 0 : max(-112, min(126, 14 - e));
}

// The request whose segments v lies among: the largest r in [0, R) with starts[r] /
// segment <= v; -1: none. A warp together: 32 places at a time. (Where starts
// decrease it finds one of them or another, the same every time.)
__device__ __forceinline__ int request_of(const ScanPlan &P, int64_t v) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = P.L.R;
    for (;;) {
        const int64_t step = (hi - lo + 31) / 32, i = lo + step * lane;
        const bool below = i < hi && __ldca(P.L.starts + i) / P.segment <= v;
        const int found = __popc(__ballot_sync(0xffffffffu, below));
        if (found == 0)
            return -1;
        lo += step * (found - 1);
        hi = min(hi, lo + step);
        if (hi - lo <= 1)
            return (int)lo;
    }
}

// First token of segment i of n of a request of T tokens after `before`: near i
// T / n, where the tiles of a block begin anyway.
__device__ __forceinline__ int64_t cut(int64_t T, int64_t i, int64_t n, int64_t before, int32_t N) {
    if (i == 0 || i == n)
        return i == 0 ? 0 : T;
    const int64_t t = T * i / n;
    return t - (before + t) % N % kTile;
}

// Whether the states before all n segments of request r, in the slots from `slot`
// on, are the states pass's own work for r, by a warp together. It is so wherever
// starts do not decrease: a request's segments are then found one behind the other,
// and others' slots lie apart from its own. Where starts decrease the search may miss
// segments, and others' may be written to the same slots: the ones of v write slot v +
// 1, a request's first one slot v, too.
__device__ __forceinline__ bool made_whole(const ScanPlan &P, int r, int64_t slot, int64_t n) {
    bool whole = true;
    for (int64_t v = slot - 1 + (threadIdx.x & 31); v < slot + n; v += 32)
        if (v >= 0 && v < P.cuts)
            whole = whole && __ldca(P.owners + v) == (v >= slot && v < slot + n - 1 ? r : -1);
    return __all_sync(0xffffffffu, whole);
}

// States only: all segments but a request's last, segment v of all. Results: a CTA
// for each request (its first segment, or all of it), then one for segment v + 1.
template <bool kStatesOnly>
__device__ __forceinline__ void find_item(const ScanPlan &P, Item &I) {
    const int lane = threadIdx.x & 31;
    const int64_t x = blockIdx.x / P.L.H;
    const bool extra = kStatesOnly || x >= P.L.R;
    const int64_t v = !kStatesOnly && extra ? x - P.L.R : x;
    const int r = extra ? request_of(P, v) : (int)x;
    Item J = {};
    J.h = (int)(blockIdx.x % P.L.H);
    J.r = r;
    if (r >= 0) {
        const Span S = span_of(P.L, r);
        uint32_t bad = S.bad;
        const int64_t slot = __ldca(P.L.starts + r) / P.segment, n = max((int64_t)1, S.count / P.segment);
        const int64_t i = !extra ? 0 : v - slot + (kStatesOnly ? 0 : 1);
        // (a segment before the first: starts that decrease)
        bool work = S.count > 0 && i >= 0 && i < (kStatesOnly ? n - 1 : n) && (kStatesOnly || !extra || i > 0);
        if (!kStatesOnly && work && n > 1 && !made_whole(P, r, slot, n)) {
            work = false;
            bad = LMC_ST_BAD_JOB;
        }
        if (work) {
            const int64_t a = cut(S.count, i, n, S.before, P.L.block_size), b = cut(S.count, i + 1, n, S.before, P.L.block_size);
            J.row = (int)(S.row + a);
            J.page = (int)((S.before + a) / P.L.block_size);
            J.phase = (int)((S.before + a) % P.L.block_size);
            J.count = (int)(b - a);
            J.first = S.first;
            J.last = S.last;
            J.slot = n > 1 ? (int)(slot + i) : -1;
            J.ends = i == n - 1;
            J.work = 1;
            // tiles of the first block, of whole ones, and of the last
            const int N = P.L.block_size, head = min(J.count, N - J.phase), rest = J.count - head;
            auto tiles = [](int tokens) { return (tokens + kTile - 1) / kTile; };
            J.tiles = tiles(head) + rest / N * tiles(N) + tiles(rest % N);
        }
        if (!extra && bad != 0 && J.h == 0 && lane == 0)  // every request is looked at once
            atomicOr(P.L.status, bad);
    }
    if (kStatesOnly && J.h == 0 && lane == 0)
        P.owners[v] = J.work ? r : -1;
    if (lane == 0)
        I = J;
}

// A sum held in two numbers, its error in the lower (Knuth's two-sum; exact but for
// the lower ones' own rounding, 2^-48 of the sum).
struct Twice {
    float high, low;
};
__device__ __forceinline__ Twice plus(const Twice &x, float high, float low) {
    const float s = x.high + high, part = s - x.high;
    return Twice{s, (x.high - (s - part)) + (high - part) + (x.low + low)};
}

// A tile's decays, by one warp: lane l's are those of tokens 2 l and 2 l + 1. Their
// sums are held twice as long as binary32, so that sums far from 0 lose nothing of
// the differences that count.
// `drift`: how much the tiles' rounded decays lack of the exact ones so far,
// relatively; a tile's makes up for it, so that a state that decays slowly by
// the same factor tile after tile keeps its digits.
// `ready` waits until they may be written.
template <bool kBf16, typename Ready>
__device__ __forceinline__ void sum_decays(Decays &D, float g0, float g1, int rows, float scale, float &drift,
                                           Ready ready) {
    const int lane = threadIdx.x & 31;
    // (a NaN is not clamped, and makes one of everything behind it)
    auto log2_of = [](float g) {
        g = g < kLeastDecay ? kLeastDecay : g;
        return (g > -kLeastDecay ? -kLeastDecay : g) * 1.44269504088896340736f;
    };
    const float a = log2_of(g0), b = log2_of(g1);
    Twice sum = plus(Twice{a, 0.0f}, b, 0.0f);
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const float high = __shfl_up_sync(0xffffffffu, sum.high, o), low = __shfl_up_sync(0xffffffffu, sum.low, o);
        if (lane >= o)
            sum = plus(sum, high, low);
    }
    const Twice total = {__shfl_sync(0xffffffffu, sum.high, 31), __shfl_sync(0xffffffffu, sum.low, 31)};
    const Twice first = plus(sum, -b, 0.0f);
    const float2 since = make_float2(exp2_fast(first.high + first.low) * scale, exp2_fast(sum.high + sum.low) * scale);
    const float f0 = 2 * lane < rows ? exp2_fast((total.high - first.high) + (total.low - first.low)) : 0.0f;
    const float f1 = 2 * lane + 1 < rows ? exp2_fast((total.high - sum.high) + (total.low - sum.low)) : 0.0f;
    uint4 left;
    if constexpr (kBf16) {
        const uint32_t p = pack<true>(f0, f1);
        const float r0 = f0 - from_q(p & 0xffff, true), r1 = f1 - from_q(p >> 16, true);
        const uint32_t q = pack<true>(r0, r1);
        left = make_uint4(q, pack<true>(r0 - from_q(q & 0xffff, true), r1 - from_q(q >> 16, true)), p, 0);
    } else {
        left = make_uint4(__float_as_uint(f0), __float_as_uint(f1), 0, 0);
    }
    const float x = total.high + total.low;
    float grow;
    if (x > -0.7f && x < 0.7f) {
        // exp(y) - 1 by its series: |y| < 0.486, what is left out is below 2^-29 of y
        const float y = x * 0.693147180559945309417f;
        float less = 1.0f / 362880.0f;
        less = fmaf(less, y, 1.0f / 40320.0f);
        less = fmaf(less, y, 1.0f / 5040.0f);
        less = fmaf(less, y, 1.0f / 720.0f);
        less = fmaf(less, y, 1.0f / 120.0f);
        less = fmaf(less, y, 1.0f / 24.0f);
        less = fmaf(less, y, 1.0f / 6.0f);
        less = fmaf(less, y, 0.5f);
        less = fmaf(less * y, y, y);
        const float high = 1.0f + less;
        const float low = fmaf(high, drift, less - (high - 1.0f));
        grow = high + low;
        drift = __fdividef((high - grow) + low, grow);
    } else {
        grow = exp2_fast(x);
        drift = 0.0f;
    }
    ready();
    *reinterpret_cast<float4 *>(&D.log[2 * lane]) = make_float4(first.high, first.low, sum.high, sum.low);
    *reinterpret_cast<float2 *>(&D.since[2 * lane]) = since;
    D.left[lane] = left;
    if (lane == 0)
        D.grow = grow;
}

// The roles that only ask for copies and products are one thread each.

// q, k and v of each tile by TMA. (Rows behind a tile's last one come along; they
// are not read into a result.)
template <bool kStatesOnly>
__device__ __forceinline__ void load_tiles(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const int h = C.item.h, kh = h / P.L.shared;
    const uint32_t bytes = (uint32_t)((kStatesOnly ? 1 : 2) * P.k_panels + P.v_panels) * kPanel;
    uint32_t asked = 0;
#pragma unroll 1
    while (T.next()) {
        const uint32_t st = asked % kStages;
        if (asked >= kStages)
            scan_wait(C, &C.free[st], (asked / kStages - 1) & 1, looks);
        if (*(volatile uint32_t *)&C.gave_up)
            break;
        uint8_t *to = mem + st * kStageBytes;
        uint64_t *bar = &C.full[st];
        bar_expect(bar, bytes);
#pragma unroll 1
        for (int i = 0; i < P.k_copies; i++)
            tma_box(&P.k, to + 2 * kPanel + i * kPanel, i * 64, T.row, kh, bar);
#pragma unroll 1
        for (int i = 0; i < P.v_copies; i++)
            tma_box(&P.v, to + 4 * kPanel + i * kPanel, i * 64, T.row, h, bar);
        if (!kStatesOnly) {
#pragma unroll 1
            for (int i = 0; i < P.k_copies; i++)
                tma_box(&P.q, to + i * kPanel, i * 64, T.row, kh, bar);
        }
        asked++;
    }
    C.tiles = asked;
}

// One warp: each tile's decays. They go to their place of the ring when the stage
// of the tile behind is free: the products of that stage's last tile are done, so
// the result of the tile before it has been read, whose place this was. (Where only
// states are made, updates take turns, and it is the tile before that one: the stage
// of two tiles behind.)
template <bool kBf16, bool kStatesOnly>
__device__ __forceinline__ void tell_decays(const ScanPlan &P, ScanControl &C) {
    static_assert(kRing >= kStages, "a place is read until the next tile's result is made");
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const int lane = threadIdx.x & 31, end = C.item.row + C.item.count;
    const float *const decay = P.L.decay + (int64_t)C.item.h * P.L.decay_head;
    float drift = 0.0f, g0, g1;
    // of 64 tokens from a row on, a tile ahead (whose tokens they are shows later)
    auto fetch = [&](int row) {
        const int64_t x = (int64_t)row + 2 * lane;
        const float *const at = decay + x * P.L.decay_row;
        g0 = x < end ? *at : 0.0f;
        g1 = x + 1 < end ? at[P.L.decay_row] : 0.0f;
    };
    fetch(C.item.row);
    while (T.next()) {
        const uint32_t n = T.n;
        const float h0 = 2 * lane < T.rows ? g0 : 0.0f, h1 = 2 * lane + 1 < T.rows ? g1 : 0.0f;
        fetch(T.row + T.rows);
        sum_decays<kBf16>(C.decays[n % kRing], h0, h1, T.rows, P.L.scale, drift, [&] {
            constexpr uint32_t kAhead = kStatesOnly ? 2 : 1;
            if (n + kAhead >= kStages)
                scan_wait(C, &C.free[(n + kAhead) % kStages], ((n + kAhead) / kStages - 1) & 1, looks);
        });
        __syncwarp();
        if (lane == 0)
            bar_arrive(&C.decays_full[n % kRing]);
    }
}

// The products that need no state. Scores Q K^T [tokens x tokens], and what the
// tile adds to the state, turned: (V decayed)^T K [values x keys].
template <bool kBf16, bool kStatesOnly>
__device__ __forceinline__ void multiply_forward(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    constexpr uint32_t tmem = 0;  // all of it: see the kernel
    const int keys = 64 * P.k_panels, steps = (P.L.dk + 15) / 16, tiles = C.item.tiles;
    const uint32_t scores = instruction(kBf16, false, 64, kTile);
    const uint32_t update = instruction(kBf16, false, 128, keys) | 1u << 16;  // B turned
    constexpr int kSteps = (kBf16 ? 2 : 1) * (kTile / 16);  // of a half of the parts
    const uint32_t q0 = lower(smem_addr(mem), 16);
    const uint32_t k0 = lower(smem_addr(mem) + 2 * kPanel, kPanel);
#pragma unroll 1
    for (int n = 0; n < tiles; n++) {
        const int st = n % kStages;
        const uint32_t q = q0 + st * (kStageBytes >> 4), k = k0 + st * (kStageBytes >> 4);
        scan_wait(C, &C.full[st], (n / kStages) & 1, looks);
        if (!kStatesOnly) {
            if (n >= 1)
                scan_wait(C, &C.score_free, (n - 1) & 1, looks);
            fence_after();
#pragma unroll
            for (int s = 0; s < kMaxDim / 16; s++)
                if (s < steps)
                    multiply(tmem + kScores, q + ((s >> 2) * (kPanel >> 4) + (s & 3) * 2),
                        q + ((2 * kPanel >> 4) + (s >> 2) * (kPanel >> 4) + (s & 3) * 2), scores, s > 0);
            commit(&C.score_full);
        }
        // as the parts come: the lower one or two, then the upper. (A sum is cut off
        // below its last place by each product: of the large part there are four.)
        const int b = kStatesOnly ? n & 1 : 0, use = kStatesOnly ? n >> 1 : n;
        const uint32_t to = tmem + (b ? kOtherUpdate : kUpdate);
        if (use >= 1)
            scan_wait(C, &C.update_free[b], (use - 1) & 1, looks);
#pragma unroll 1
        for (int half = 0; half < 2; half++) {
            scan_wait(C, &C.parts_full[half], n & 1, looks);
            fence_after();
#pragma unroll
            for (int s = 0; s < kSteps; s++)
                multiply_held(to, tmem + kParts + kSteps * 8 * half + 8 * s, k + (s & 3) * (2048 >> 4), update,
                              s > 0 || half > 0);
            commit(&C.parts_free[half]);
        }
        commit(&C.update_full[b]);
        commit(&C.free[st]);
    }
}

// The products that make the result, turned: S^T Q^T from the state before the
// tile, V^T P^T from the tile's own tokens [values x tokens].
template <bool kBf16>
__device__ __forceinline__ void multiply_state(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    constexpr uint32_t tmem = 0;
    const int steps = (P.L.dk + 15) / 16, tiles = C.item.tiles;
    const uint32_t from_state = instruction(kBf16, false, 128, kTile), from_tile = instruction(kBf16, true, 128, kTile);
    const uint32_t weight = lower(smem_addr(mem) + kWeightsAt, 16);
    const uint32_t q0 = lower(smem_addr(mem), 16);
    const uint32_t v0 = lower(smem_addr(mem) + 4 * kPanel, kPanel);
#pragma unroll 1
    for (int n = 0; n < tiles; n++) {
        const int st = n % kStages;
        const uint32_t q = q0 + st * (kStageBytes >> 4), v = v0 + st * (kStageBytes >> 4);
        scan_wait(C, &C.full[st], (n / kStages) & 1, looks);
        scan_wait(C, &C.state_full, n & 1, looks);
        if (n >= 1)
            scan_wait(C, &C.out_free, (n - 1) & 1, looks);
        fence_after();
#pragma unroll
        for (int s = 0; s < kMaxDim / 16; s++)
            if (s < steps)
                multiply_held(tmem + kFromState, tmem + kState + 8 * s, q + ((s >> 2) * (kPanel >> 4) + (s & 3) * 2), from_state,
                         s > 0);
        commit(&C.state_free);
        scan_wait(C, &C.weight_full, n & 1, looks);
        fence_after();
#pragma unroll
        for (int s = 0; s < kTile / 16; s++)
            multiply(tmem + kFromTile, v + s * (2048 >> 4), weight + s * 2, from_tile, s > 0);
        commit(&C.out_full);
        commit(&C.weight_free);
        commit(&C.free[st]);
    }
}

// What a lane holds of 16 values and 32 tokens from `first` on (load_turned): those
// behind the tile's last row become 0.
__device__ __forceinline__ void keep_rows(uint32_t (&v)[8], int first, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const int t = first + 8 * (k >> 1) + 2 * (lane & 3);
        v[k] &= (t < rows ? 0xffffu : 0u) | (t + 1 < rows ? 0xffff0000u : 0u);
    }
}

// Eight warps: v times the decay to the tile's end, turned, in parts of 16 bits, to
// tensor memory: of values 32 w .. 32 w + 31 warp w takes the first 16, w + 4 the
// last.
//
// What is added to the state keeps binary32's digits: with f = f1 + f2 + f3 in
// bf16, v f = A + B + C + D where A = rn(v f1), B = v f1 - A (exact: a product of
// two numbers of 8 bits has 16), C = rn(v f2) and D = rn(v f3 + (v f2 - C)), each
// a bf16: off by 2^-26. In pairs of bf16 that is five instructions for two values
// (three truncated parts of a binary32 product are fifteen).
template <bool kBf16>
__device__ __forceinline__ void split(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kFirstPartWarp, quarter = warp & 3, block = warp >> 2;
    const uint32_t to = C.tmem + ((uint32_t)(quarter * 32 + 16 * block) << 16) + kParts;
    // the row of four 8 x 8 matrices that this lane names: tokens 8 (lane / 16) +
    // lane % 8 of a step's, values 8 (lane / 8 % 2) .. of 16
    const uint32_t values = smem_addr(mem) + 4 * kPanel + (quarter >> 1) * kPanel + (8 * (lane >> 4) + (lane & 7)) * 128;
    const int chunk = 4 * (quarter & 1) + 2 * block + (lane >> 3 & 1);
    while (T.next()) {
        const uint32_t n = T.n;
        const int st = n % kStages;
        Decays &D = C.decays[n % kRing];
        scan_wait(C, &C.decays_full[n % kRing], (n / kRing) & 1, looks);
        scan_wait(C, &C.full[st], (n / kStages) & 1, looks);
        if (T.rows < kTile) {  // the products' other side
            clear_rows(mem + st * kStageBytes + 2 * kPanel, T.rows, threadIdx.x - kFirstPartWarp * 32, kPartWarps * 32);
            fence_async();
        }
        const uint32_t from = values + st * kStageBytes + ((chunk ^ (lane & 7)) << 4);
        // Lower parts first (the state is off by 1e-7, not 5e-7): their products run
        // while the upper are made, and the next tile's lower parts are made while the
        // upper's run. (f16's two parts are made together, and go into one half each.)
        if constexpr (kBf16) {
#pragma unroll 1
            for (int upper = 0; upper < 2; upper++) {
                if (n >= 1)
                    scan_wait(C, &C.parts_free[upper], (n - 1) & 1, looks);
                fence_after();
#pragma unroll 1
                for (int half = 0; half < 2; half++) {  // 32 tokens
                    uint32_t v[8], a[8], b[8];
#pragma unroll
                    for (int s = 0; s < 2; s++)
                        load_turned(v + 4 * s, from + (2 * half + s) * 2048);
                    if (T.rows < kTile)
                        keep_rows(v, 32 * half, T.rows);
                    // x = rn(v f) and y = v f - x + v g, g: f3, and 0 in the upper parts
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const uint2 f = reinterpret_cast<const uint2 *>(&D.left[16 * half + 4 * (k >> 1) + (lane & 3)])[upper];
                        a[k] = times(v[k], f.x);
                        b[k] = plus_product(v[k], f.y, plus_product(v[k], f.x, minus(a[k])));
                    }
                    store_part(to + 2 * kPartColumns * upper + 16 * half, b);
                    store_part(to + 2 * kPartColumns * upper + kPartColumns + 16 * half, a);
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&C.parts_full[upper]);
            }
        } else {
            // two rounded parts of the product, whose row (a value's, of 64 tokens:
            // four lanes) is brought below 2^15 by a power of two
            float top[2] = {0.0f, 0.0f};
#pragma unroll 1
            for (int half = 0; half < 2; half++) {
                uint32_t v[8];
#pragma unroll
                for (int s = 0; s < 2; s++)
                    load_turned(v + 4 * s, from + (2 * half + s) * 2048);
                if (T.rows < kTile)
                    keep_rows(v, 32 * half, T.rows);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float2 f = *reinterpret_cast<const float2 *>(&D.left[16 * half + 4 * (k >> 1) + (lane & 3)]);
                    const float2 x = __fmul2_rn(from_halves(v[k]), f);
                    top[k & 1] = greatest(top[k & 1], x.x, x.y);
                }
            }
            float up[2];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2));
                const int e = lift_of(top[k]);
                up[k] = power(e);
                if ((lane & 3) == 0)
                    D.unit[32 * quarter + 16 * block + 8 * k + lane / 4] = power(-e);
            }
            if (n >= 1) {
                scan_wait(C, &C.parts_free[0], (n - 1) & 1, looks);
                scan_wait(C, &C.parts_free[1], (n - 1) & 1, looks);
            }
            fence_after();
#pragma unroll 1
            for (int half = 0; half < 2; half++) {
                uint32_t v[8], a[8], b[8];
#pragma unroll
                for (int s = 0; s < 2; s++)
                    load_turned(v + 4 * s, from + (2 * half + s) * 2048);
                if (T.rows < kTile)
                    keep_rows(v, 32 * half, T.rows);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float2 f = *reinterpret_cast<const float2 *>(&D.left[16 * half + 4 * (k >> 1) + (lane & 3)]);
                    float2 x = __fmul2_rn(__fmul2_rn(from_halves(v[k]), f), make_float2(up[k & 1], up[k & 1]));
                    a[k] = pack<false>(x.x, x.y);
                    x = less(x, from_halves(a[k]));
                    b[k] = pack<false>(x.x, x.y);
                }
                store_part(to + 16 * half, b);
                store_part(to + kPartColumns + 16 * half, a);
            }
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(&C.unit_full[n % kRing]);
                bar_arrive(&C.parts_full[0]);
                bar_arrive(&C.parts_full[1]);
            }
        }
    }
}

// Four warps: the weights P = (Q K^T) * decays, of tokens up to the row's own (warp
// w: rows 16 w .. 16 w + 15).
//
// They are rounded to 16 bits, which over many of them makes the result's error
// sqrt(2) of what rounding it alone makes. Over few it can be 2.5 times that (one
// weight is a factor of a head's whole result), so tiles of at most 32 tokens hold
// what rounding took off as weights of the same tokens, half a tile on: the products
// are there anyway.
template <bool kBf16>
__device__ __forceinline__ void weigh(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) - kFirstWeightWarp;
    const uint32_t lanes = C.tmem + ((uint32_t)(quarter * 32) << 16);
    const int ra = quarter * 16 + lane / 4, rb = ra + 8;  // this thread's rows of P
    uint8_t *const pa = mem + kWeightsAt + ra * 128 + 4 * (lane & 3), *const pb = pa + 8 * 128;
    bool held = false;  // the rows' second halves hold something
    while (T.next()) {
        const uint32_t n = T.n;
        const bool twice = T.rows <= kTile / 2;
        Decays &D = C.decays[n % kRing];
        scan_wait(C, &C.decays_full[n % kRing], (n / kRing) & 1, looks);
        if (T.rows < kTile) {
            scan_wait(C, &C.full[n % kStages], (n / kStages) & 1, looks);
            clear_rows(mem + (n % kStages) * kStageBytes + 4 * kPanel, T.rows, threadIdx.x - kFirstWeightWarp * 32, kWeightWarps * 32,
                       twice);
        }
        scan_wait(C, &C.score_full, n & 1, looks);
        fence_after();
        const float2 la = D.log[ra], lb = D.log[rb];
        // 16 tokens' weights of the thread's rows at a time, up to the rows' own (the
        // others are 0 from the start): (ra, c), (ra, c + 1), (rb, c), (rb, c + 1) with
        // c = 16 u + 8 i + 2 (lane % 4)
        auto make = [&](int u, float (&p)[2][4]) {
            uint32_t raw[8];
            load_s8(raw, lanes + kScores + 16 * u);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int c = 16 * u + 8 * i + 2 * (lane & 3);
                const float4 lc = *reinterpret_cast<const float4 *>(&D.log[c]);
                const float2 l0 = make_float2(lc.x, lc.y), l1 = make_float2(lc.z, lc.w);
                const float2 d0 = less(la, l0), d1 = less(la, l1), d2 = less(lb, l0), d3 = less(lb, l1);
                const float2 unit = make_float2(P.L.scale, P.L.scale);
                float2 x = __fmul2_rn(make_float2(__uint_as_float(raw[4 * i]), __uint_as_float(raw[4 * i + 1])), unit);
                float2 y = __fmul2_rn(make_float2(__uint_as_float(raw[4 * i + 2]), __uint_as_float(raw[4 * i + 3])), unit);
                x = __fmul2_rn(x, make_float2(exp2_fast(d0.x + d0.y), exp2_fast(d1.x + d1.y)));
                y = __fmul2_rn(y, make_float2(exp2_fast(d2.x + d2.y), exp2_fast(d3.x + d3.y)));
                p[i][0] = c <= ra ? x.x : 0.0f;
                p[i][1] = c < ra ? x.y : 0.0f;
                p[i][2] = c <= rb ? y.x : 0.0f;
                p[i][3] = c < rb ? y.y : 0.0f;
            }
        };
        float ua = 1.0f, ub = 1.0f;
        bool some_a = false, some_b = false;  // f16: a product is not 0
        if constexpr (!kBf16) {
            // f16 has not binary32's range: a row's weights are brought below 2^15, by
            // the largest of its products (decays are at most 1), which is far from the
            // largest weight where that product's token has been forgotten: see below
            float ta = 0.0f, tb = 0.0f;
#pragma unroll 1
            for (int u = 0; u <= quarter; u++) {
                uint32_t raw[8];
                load_s8(raw, lanes + kScores + 16 * u);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int c = 16 * u + 8 * i + 2 * (lane & 3);
                    ta = greatest(ta, c <= ra ? __uint_as_float(raw[4 * i]) : 0.0f,
                                  c < ra ? __uint_as_float(raw[4 * i + 1]) : 0.0f);
                    tb = greatest(tb, c <= rb ? __uint_as_float(raw[4 * i + 2]) : 0.0f,
                                  c < rb ? __uint_as_float(raw[4 * i + 3]) : 0.0f);
                }
            }
            for (int o = 1; o < 4; o <<= 1) {
                ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, o));
                tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, o));
            }
            const float unit = fabsf(P.L.scale);
            const int ea = lift_of(ta * unit), eb = lift_of(tb * unit);
            ua = power(ea);
            ub = power(eb);
            some_a = ta != 0.0f;
            some_b = tb != 0.0f;
        }
        if (n >= 1)
            scan_wait(C, &C.weight_free, (n - 1) & 1, looks);
        float wa = 0.0f, wb = 0.0f;  // f16: the largest of this thread's weights
        for (bool again = false;; again = true) {
#pragma unroll 1
            for (int u = 0; u <= quarter; u++) {
                float p[2][4];
                make(u, p);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int at = ((2 * u + i) ^ (ra & 7)) << 4;  // rb & 7 is the same
                    *reinterpret_cast<uint32_t *>(pa + at) = pack<kBf16>(p[i][0] * ua, p[i][1] * ua);
                    *reinterpret_cast<uint32_t *>(pb + at) = pack<kBf16>(p[i][2] * ub, p[i][3] * ub);
                    if (!kBf16) {
                        wa = greatest(wa, p[i][0], p[i][1]);
                        wb = greatest(wb, p[i][2], p[i][3]);
                    }
                }
            }
            if (kBf16 || again)
                break;
            // Rows whose largest weight was brought below 2^6 are made again, by that
            // one: a weight keeps f16's steps down to 2^-20 of its row's largest. (A
            // row's four lanes hold a quarter of its weights each. Looking costs 2 to 4 %
            // of the call; finding the largest weight first 9 %.)
            uint32_t fine = __ballot_sync(0xffffffffu, wa * ua >= 64.0f || !some_a || ra >= T.rows);
            uint32_t both = __ballot_sync(0xffffffffu, wb * ub >= 64.0f || !some_b || rb >= T.rows);
            fine |= fine >> 1, both |= both >> 1;
            fine |= fine >> 2, both |= both >> 2;
            if ((fine & both & 0x11111111u) == 0x11111111u)
                break;
            for (int o = 1; o < 4; o <<= 1) {
                wa = fmaxf(wa, __shfl_xor_sync(0xffffffffu, wa, o));
                wb = fmaxf(wb, __shfl_xor_sync(0xffffffffu, wb, o));
            }
            ua = power(lift_of(wa));
            ub = power(lift_of(wb));
        }
        if (!kBf16 && (lane & 3) == 0) {
            D.lift[ra] = inverse_power(ua);
            D.lift[rb] = inverse_power(ub);
        }
        if (__builtin_expect(held || twice, false) && quarter < 2) {
#pragma unroll 1
            for (int u = 0; u < 2; u++) {
                float p[2][4] = {};
                if (twice && u <= quarter)
                    make(u, p);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int at = ((2 * u + i) ^ 4 ^ (ra & 7)) << 4;
                    auto rest = [](float x, float y) {
                        const uint32_t w = pack<kBf16>(x, y);
                        return pack<kBf16>(x - from_q(w & 0xffff, kBf16), y - from_q(w >> 16, kBf16));
                    };
                    *reinterpret_cast<uint32_t *>(pa + at) = rest(p[i][0] * ua, p[i][1] * ua);
                    *reinterpret_cast<uint32_t *>(pb + at) = rest(p[i][2] * ub, p[i][3] * ub);
                }
            }
            held = twice;
        }
        fence_before();
        fence_async();
        __syncwarp();
        if (lane == 0) {
            bar_arrive(&C.score_free);
            if (!kBf16)
                bar_arrive(&C.lift_full[n & 1]);
            bar_arrive(&C.weight_full);
        }
    }
}

// Eight warps: the state, turned, in registers: warps w and w + 4 hold values 32 w
// .. 32 w + 31 (a lane each), w the first 64 keys, w + 4 the others.
template <bool kBf16, bool kStatesOnly>
__device__ __forceinline__ void carry(const ScanPlan &P, ScanControl &C) {
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const LinearPlan &L = P.L;
    const Item &I = C.item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = C.tmem + ((uint32_t)(quarter * 32) << 16);
    const int j = quarter * 32 + lane, i0 = 64 * half;
    const bool mine = i0 < L.dk;
    const int64_t head = (int64_t)I.h * L.dk * L.dv, at = (int64_t)i0 * L.dv + j;
    const int64_t slot_size = (int64_t)L.H * L.dk * L.dv;
    float2 s[32];  // pairs of keys: two products an instruction
#pragma unroll
    for (int i = 0; i < 32; i++)
        s[i] = make_float2(0.0f, 0.0f);
    auto read = [&](const float *from) {
        if (j < L.dv) {
            from += at;
#pragma unroll
            for (int g = 0; g < 64; g += 8)
                if (i0 + g < L.dk)
#pragma unroll
                    for (int i = g; i < g + 8; i++, from += L.dv)
                        (i & 1 ? s[i / 2].y : s[i / 2].x) = __ldcs(from);
        }
    };
    auto write = [&](float *to) {
        if (j < L.dv) {
            to += at;
#pragma unroll
            for (int g = 0; g < 64; g += 8)
                if (i0 + g < L.dk)
#pragma unroll
                    for (int i = g; i < g + 8; i++, to += L.dv)
                        __stcs(to, i & 1 ? s[i / 2].y : s[i / 2].x);
        }
    };
    // The state as A of its product with q, in 16 bits; what is to be multiplied
    // to its row's results (f16, which has not binary32's range: rows are brought
    // below 2^15).
    auto hand_over = [&](uint32_t n) {
        float up = 1.0f;
        if constexpr (!kBf16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; i++)
                top = greatest(top, s[i].x, s[i].y);
            C.row_top[half][j] = top;
            asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
            top = fmaxf(top, C.row_top[half ^ 1][j]);
            const int e = lift_of(top);
            up = power(e);
            if (half == 0)
                C.down[n & 1][j] = power(-e);
        }
        if (mine) {
#pragma unroll
            for (int c = 0; c < 4; c++) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 y = kBf16 ? s[8 * c + i] : __fmul2_rn(s[8 * c + i], make_float2(up, up));
                    x[i] = pack<kBf16>(y.x, y.y);
                }
                store_o8(x, lanes + kState + 32 * half + 8 * c);
            }
            wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
            if (!kBf16)
                bar_arrive(&C.down_full[n & 1]);
            bar_arrive(&C.state_full);
        }
    };
    // where a state is at hand before the item's tokens
    float *const slot = P.slots + (int64_t)I.slot * slot_size + head;
    const bool first = kStatesOnly && I.row == __ldca(L.starts + I.r);  // the request's first segment
    const float *const from = !kStatesOnly && I.slot >= 0                     ? slot
                              : I.first >= 0 && (!kStatesOnly || first) ? L.pages + I.first * L.page_stride + head
                                                                        : nullptr;
    if (from != nullptr)
        read(from);
    if (first)
        write(slot);
    // log2 of the decay over the item, as two numbers: one would round the same way
    // tile after tile (some 2^-25 of it each, under one decay for all tokens)
    Twice total = {0.0f, 0.0f};
    if (!kStatesOnly && I.count > 0)
        hand_over(0);
    while (T.next()) {
        const uint32_t n = T.n;
        const Decays &D = C.decays[n % kRing];
        // the block that is written to, asked for early
        int32_t block = -1;
        if (!kStatesOnly && (T.block_ends || (I.ends && T.last()))) {
            block = __ldca(L.table + I.r * L.row_stride + T.page);
            // (a page that stands at several positions is written by the last one
            // alone: segments do not take turns)
            if (block == I.last && !(I.ends && T.last()))
                block = -1;
        }

        scan_wait(C, &C.decays_full[n % kRing], (n / kRing) & 1, looks);
        const float grow = D.grow;
        if (kStatesOnly)
            total = plus(total, D.log[kTile - 1].x, D.log[kTile - 1].y);
        if (!kBf16)
            scan_wait(C, &C.unit_full[n % kRing], (n / kRing) & 1, looks);
        const float unit = kBf16 ? 1.0f : D.unit[j];
        const int b = kStatesOnly ? n & 1 : 0;
        scan_wait(C, &C.update_full[b], (kStatesOnly ? n >> 1 : n) & 1, looks);
        fence_after();
        if (mine) {
#pragma unroll
            for (int c = 0; c < 8; c++) {
                uint32_t u[8];
                load_o8(u, lanes + (b ? kOtherUpdate : kUpdate) + i0 + 8 * c);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float2 y = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                    if constexpr (!kBf16)
                        y = __fmul2_rn(y, make_float2(unit, unit));
                    s[4 * c + i] = __ffma2_rn(make_float2(grow, grow), s[4 * c + i], y);
                }
            }
        }
        fence_before();
        __syncwarp();
        if (lane == 0)
            bar_arrive(&C.update_free[b]);
        if (block >= 0 && block < L.num_blocks)
            write(L.pages + block * L.page_stride + head);
        else if (block != -1 && threadIdx.x == 0)
            atomicOr(L.status, LMC_ST_BLOCK_OOR);
        __syncwarp();
        if (!kStatesOnly && !T.last()) {
            scan_wait(C, &C.state_free, n & 1, looks);
            fence_after();
            hand_over(n + 1);
        }
    }
    if (kStatesOnly) {
        write(slot + slot_size);
        if (threadIdx.x == 0)
            P.totals[((int64_t)I.slot + 1) * L.H + I.h] = make_float2(total.high, total.low);
    }
}

// Four warps: the result of each tile. Warp w takes values 32 w .. 32 w + 31.
template <bool kBf16>
__device__ __forceinline__ void deliver(const ScanPlan &P, ScanControl &C, uint8_t *mem) {
    int looks = kLooks;
    Tiles T(C.item, P.L.block_size);
    const LinearPlan &L = P.L;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) - kFirstResultWarp;
    const uint32_t lanes = C.tmem + ((uint32_t)(quarter * 32) << 16);
    uint8_t *const mine = mem + kResultAt + quarter * kWarpResult;
    // A row of 32 values, 64 bytes, per token; its 16-byte pieces change places
    // from row to row, so that no two of eight rows' fall into the same banks.
    // The row of four 8 x 8 matrices that this lane names:
    const int named = 8 * (lane >> 4) + (lane & 7), piece = lane >> 3 & 1;
    const uint32_t staged = smem_addr(mine) + named * 64, turn = named >> 1 & 3;
    const int64_t out_at = (int64_t)C.item.h * L.out_head + quarter * 32;
    while (T.next()) {
        const uint32_t n = T.n;
        const Decays &D = C.decays[n % kRing];
        scan_wait(C, &C.decays_full[n % kRing], (n / kRing) & 1, looks);
        if (!kBf16) {
            scan_wait(C, &C.lift_full[n & 1], (n >> 1) & 1, looks);
            scan_wait(C, &C.down_full[n & 1], (n >> 1) & 1, looks);
        }
        scan_wait(C, &C.out_full, n & 1, looks);
        fence_after();
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the tile before's
        __syncwarp();
        float2 since[4];
#pragma unroll 1
        for (int part = 0; part < 4; part++) {  // 32 tokens, 16 values
            const int half = part >> 1, b16 = part & 1;
            if (b16 == 0)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    since[i] = *reinterpret_cast<const float2 *>(&D.since[32 * half + 8 * i + 2 * (lane & 3)]);
            uint32_t a[16], b[16];
            const uint32_t at = lanes + ((uint32_t)(16 * b16) << 16) + 32 * half;
            load_s(a, at + kFromState);
            load_s(b, at + kFromTile);
            float da = 1.0f, db = 1.0f;
            if constexpr (!kBf16) {
                da = C.down[n & 1][32 * quarter + 16 * b16 + lane / 4];
                db = C.down[n & 1][32 * quarter + 16 * b16 + lane / 4 + 8];
            }
            wait_ld();
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 e = since[i];
                float2 g = make_float2(1.0f, 1.0f);
                if constexpr (!kBf16)
                    g = *reinterpret_cast<const float2 *>(&D.lift[32 * half + 8 * i + 2 * (lane & 3)]);
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    float2 x = make_float2(__uint_as_float(a[4 * i + 2 * k]), __uint_as_float(a[4 * i + 2 * k + 1]));
                    float2 z = make_float2(__uint_as_float(b[4 * i + 2 * k]), __uint_as_float(b[4 * i + 2 * k + 1]));
                    if constexpr (!kBf16) {
                        x = __fmul2_rn(x, k ? make_float2(db, db) : make_float2(da, da));
                        z = __fmul2_rn(z, g);
                    }
                    x = __ffma2_rn(x, e, z);
                    y[2 * i + k] = pack<kBf16>(x.x, x.y);
                }
            }
            const uint32_t to = staged + half * 32 * 64 + (((2 * b16 + piece) ^ turn) << 4);
            store_turned(to, y[0], y[1], y[2], y[3]);
            store_turned(to + 16 * 64, y[4], y[5], y[6], y[7]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0)
            bar_arrive(&C.out_free);
        if (P.wide_out && T.rows == kTile) {
            fence_async();
            __syncwarp();
            if (lane == 0 && quarter * 32 < L.dv)
                tma_store(&P.out, mine, quarter * 32, T.row, C.item.h);
        } else if (P.wide_out) {
            const int v = 8 * (lane & 3), t0 = lane >> 2;
            uint16_t *out = L.out + ((int64_t)T.row + t0) * L.out_row + out_at + v;
            const bool inside = quarter * 32 + v < L.dv;
#pragma unroll 1
            for (int i = 0; i < 8; i++) {
                const int t = 8 * i + t0;
                const uint4 x = *reinterpret_cast<const uint4 *>(mine + t * 64 + (((lane & 3) ^ (t >> 1 & 3)) << 4));
                if (inside && t < T.rows)
                    __stcs(reinterpret_cast<uint4 *>(out), x);
                out += 8 * L.out_row;
            }
        } else if (quarter * 32 + lane < L.dv) {
#pragma unroll 1
            for (int t = 0; t < T.rows; t++)
                L.out[((int64_t)T.row + t) * L.out_row + out_at + lane] =
                    *reinterpret_cast<const uint16_t *>(mine + t * 64 + (((lane >> 3) ^ (t >> 1 & 3)) << 4) + 2 * (lane & 7));
        }
        __syncwarp();
    }
    if (lane == 0)
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A CTA that gave up: what it left running ends (or the limit runs out) before
// its memory goes to another.
__device__ __forceinline__ void scan_outlast(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 22) && !bar_try(bar, parity); i++) {
    }
}

__device__ void scan_wind_up(ScanControl &C, int warp) {
    if (warp == kForwardWarp || warp == kStateProductWarp) {
        uint64_t *const done = &C.ended[warp - kForwardWarp];
        if (elect())
            commit(done);
        __syncwarp();
        scan_outlast(done, 0);
    } else if (warp == kLoadWarp) {
        for (uint32_t k = C.tiles > kStages ? C.tiles - kStages : 0; k < C.tiles; k++)
            scan_outlast(&C.full[k % kStages], (k / kStages) & 1);
    }
}

template <bool kBf16, bool kStatesOnly>
__global__ void __launch_bounds__(kScanThreads, 1) lmc_linear_scan_kernel(const __grid_constant__ ScanPlan P) {
    extern __shared__ __align__(1024) uint8_t scan_mem[];
    __shared__ ScanControl C;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; i++) {
            bar_init(&C.full[i], 1);
            bar_init(&C.free[i], kStatesOnly ? 1 : 2);
        }
        for (int i = 0; i < kRing; i++) {
            bar_init(&C.decays_full[i], 1);
            bar_init(&C.unit_full[i], kPartWarps);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(&C.lift_full[i], kWeightWarps);
            bar_init(&C.down_full[i], kStateWarps);
            bar_init(&C.ended[i], 1);
            bar_init(&C.parts_full[i], kPartWarps);
            bar_init(&C.parts_free[i], 1);
            bar_init(&C.update_full[i], 1);
            bar_init(&C.update_free[i], kStateWarps);
        }
        bar_init(&C.weight_full, kWeightWarps);
        bar_init(&C.weight_free, 1);
        bar_init(&C.score_full, 1);
        bar_init(&C.score_free, kWeightWarps);
        bar_init(&C.state_full, kStateWarps);
        bar_init(&C.out_full, 1);
        bar_init(&C.state_free, 1);
        bar_init(&C.out_free, kResultWarps);
        C.gave_up = 0;
        C.tiles = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // weights of tokens behind a row's own are never written: 0
    for (int i = threadIdx.x; i < kPanel / 16; i += kScanThreads)
        reinterpret_cast<uint4 *>(scan_mem + kWeightsAt)[i] = make_uint4(0, 0, 0, 0);
    fence_async();
    wait_for_launch();
    if (warp == 0)
        find_item<kStatesOnly>(P, C.item);
    __syncthreads();
    if (!C.item.work)
        return;
    // (asked for after the wait: a kernel before this one may still hold it)
    if (warp == kForwardWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&C.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    let_next_start();

    if (warp < kStateWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegisters));
        carry<kBf16, kStatesOnly>(P, C);
    } else if (warp < kFirstWeightWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPartRegisters));
        split<kBf16>(P, C, scan_mem);
    } else if (warp < kFirstResultWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWeightRegisters));
        if (!kStatesOnly)
            weigh<kBf16>(P, C, scan_mem);
    } else if (warp < kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kResultRegisters));
        if (!kStatesOnly)
            deliver<kBf16>(P, C, scan_mem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
        if (warp == kDecayWarp) {
            tell_decays<kBf16, kStatesOnly>(P, C);
        } else if (elect()) {
            if (warp == kLoadWarp)
                load_tiles<kStatesOnly>(P, C, scan_mem);
            else if (warp == kForwardWarp)
                multiply_forward<kBf16, kStatesOnly>(P, C, scan_mem);
            else if (!kStatesOnly)
                multiply_state<kBf16>(P, C, scan_mem);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (C.gave_up) {
        if (threadIdx.x == 0)
            atomicOr(P.L.status, LMC_ST_TIMEOUT);
        scan_wind_up(C, warp);
        __syncthreads();
    }
    if (warp == kForwardWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(C.tmem));
}

// The states before a cut request's segments, from what each segment adds: slot
// i + 1 holds the state after segment 0 (i = 0), or what segment i adds, and
// gets the state after it.
constexpr int kJoinThreads = 256;
static_assert(kJoinThreads >= kSms, "a thread for each segment of a request");

__global__ void __launch_bounds__(kJoinThreads) lmc_linear_join_kernel(const __grid_constant__ ScanPlan P) {
    __shared__ int32_t first, cuts;
    __shared__ float2 decays[kSms];  // of segments: (a, keep), the state before becomes keep s + a s
    const LinearPlan &L = P.L;
    const int parts = (L.dk * L.dv / 4 + kJoinThreads - 1) / kJoinThreads;
    const int part = blockIdx.x % parts, h = blockIdx.x / parts % L.H;
    const int64_t v = blockIdx.x / parts / L.H;
    wait_for_launch();
    let_next_start();
    if (threadIdx.x < 32) {
        const int r = request_of(P, v);
        int n = 0;
        int64_t slot = -1;
        if (r >= 0) {
            slot = __ldca(L.starts + r) / P.segment;
            n = (int)(span_of(L, r).count / P.segment);
            if (slot == v && n > 2 && !made_whole(P, r, slot, n))
                n = 0;
        }
        if (threadIdx.x == 0) {
            first = slot == v ? 1 : 0;
            cuts = n;
        }
    }
    __syncthreads();
    if (!first || cuts < 3)
        return;
    if ((int)threadIdx.x < cuts) {
        const float2 total = __ldca(P.totals + (v + threadIdx.x) * L.H + h);
        // a slow decay as s + (decay - 1) s, as in a step
        const bool slow = total.x > -0.7f && total.x < 0.7f;
        decays[threadIdx.x] = slow ? make_float2(expm1f((total.x + total.y) * 0.693147180559945309417f), 1.0f)
                                   : make_float2(exp2f(total.x) * fmaf(total.y, 0.693147180559945309417f, 1.0f), 0.0f);
    }
    __syncthreads();
    const int e = part * kJoinThreads + threadIdx.x;
    if (e >= L.dk * L.dv / 4)
        return;
    const int64_t stride = (int64_t)L.H * L.dk * L.dv / 4;
    float4 *at = reinterpret_cast<float4 *>(P.slots) + (v + 1) * stride + (int64_t)h * (L.dk * L.dv / 4) + e;
    float4 s = __ldcg(at);
#pragma unroll 8
    for (int i = 2; i < cuts; i++) {
        at += stride;
        const float4 u = __ldcg(at);
        const float a = decays[i].x, keep = decays[i].y;
        s.x = fmaf(keep, s.x, fmaf(a, s.x, u.x));
        s.y = fmaf(keep, s.y, fmaf(a, s.y, u.y));
        s.z = fmaf(keep, s.z, fmaf(a, s.z, u.z));
        s.w = fmaf(keep, s.w, fmaf(a, s.w, u.w));
        __stcg(at, s);
    }
}

// ---- host ------------------------------------------------------------------------

bool aligned16(int64_t x) { return (x & 15) == 0; }

// Rows of heads as the products read them (rows <= 1 and heads <= 1: any stride).
bool input_ok(int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t dim) {
    return (rows <= 1 || (row >= dim && row % 8 == 0)) && (heads <= 1 || (head >= dim && head % 8 == 0)) && row >= 0 &&
           head >= 0 && row < (int64_t)1 << 36 && head < (int64_t)1 << 36;
}

// Bytes from a tensor's first element to behind its last one.
bool extent(const void *p, int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t dim, int64_t bytes,
            uint64_t *at, uint64_t *end) {
    int64_t a = 0, b = 0;
    if (!mul_ok(row, rows - 1, &a) || !mul_ok(head, heads - 1, &b) || !add_ok(a, b, &a) || !add_ok(a, dim, &a) ||
        a > INT64_MAX / 8)
        return false;
    *at = (uint64_t)(uintptr_t)p;
    *end = *at + (uint64_t)a * bytes;
    return true;
}

int check_linear(const lmc_layout *L, const lmc_linear *a, int64_t rows, const void *pool, const uint32_t *status) {
    if (L == nullptr || a == nullptr || a->layer < 0 || (size_t)a->layer >= L->desc.size() || status == nullptr ||
        L->specs[a->layer].kind != LMC_LAYER_KDA || (a->dtype != LMC_E_BF16 && a->dtype != LMC_E_F16) || rows < 0 ||
        a->num_requests < 0 || a->num_requests > 1 << 20 || a->num_heads <= 0 || a->num_heads > 65535 ||
        a->num_key_heads <= 0 || a->num_heads % a->num_key_heads != 0 || a->key_dim <= 0 || a->key_dim > kMaxDim ||
        a->key_dim % 8 != 0 || a->value_dim <= 0 || a->value_dim > kMaxDim || a->value_dim % 8 != 0 ||
        !std::isfinite(a->scale) || L->block_size > INT32_MAX ||
        L->specs[a->layer].rec_bytes != (int64_t)a->num_heads * a->key_dim * a->value_dim * 4 ||
        !table_ok(a->table, a->num_requests))
        return LMC_ERR_INVALID_ARG;
    const int64_t H = a->num_heads, K = a->num_key_heads;
    if (!input_ok(rows, a->q_row_stride, K, a->q_head_stride, a->key_dim) ||
        !input_ok(rows, a->k_row_stride, K, a->k_head_stride, a->key_dim) ||
        !input_ok(rows, a->v_row_stride, H, a->v_head_stride, a->value_dim) || a->out_row_stride < 0 ||
        a->out_head_stride < 0 || a->decay_row_stride < 0 || a->decay_head_stride < 0 ||
        (rows > 1 && a->out_row_stride < a->value_dim) || (H > 1 && a->out_head_stride < a->value_dim))
        return LMC_ERR_INVALID_ARG;
    if (rows > 0 && (pool == nullptr || a->lengths == nullptr || a->q == nullptr || a->k == nullptr || a->v == nullptr ||
                     a->out == nullptr || a->decay == nullptr))
        return LMC_ERR_INVALID_ARG;
    const lmc_layer_desc &d = L->desc[a->layer];
    if ((((uintptr_t)status | (uintptr_t)a->lengths | (uintptr_t)a->decay) & 3) != 0 || ((uintptr_t)a->out & 1) != 0 ||
        !aligned16((int64_t)((uintptr_t)pool | (uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->v)) ||
        !aligned16(d.base | d.stride | L->specs[a->layer].conv_bytes))
        return LMC_ERR_ALIGN;
    if (rows == 0)
        return LMC_OK;
    uint64_t at, end, from, to;
    if (!extent(a->out, rows, a->out_row_stride, H, a->out_head_stride, a->value_dim, 2, &at, &end))
        return LMC_ERR_INVALID_ARG;
    // heads of one result may not overlap, in either order
    if (rows > 1 && H > 1 && a->out_row_stride < (H - 1) * a->out_head_stride + a->value_dim &&
        a->out_head_stride < (rows - 1) * a->out_row_stride + a->value_dim)
        return LMC_ERR_INVALID_ARG;
    for (int i = 0; i < 4; i++) {
        const bool fits =
            i == 0   ? extent(a->q, rows, a->q_row_stride, K, a->q_head_stride, a->key_dim, 2, &from, &to)
            : i == 1 ? extent(a->k, rows, a->k_row_stride, K, a->k_head_stride, a->key_dim, 2, &from, &to)
            : i == 2 ? extent(a->v, rows, a->v_row_stride, H, a->v_head_stride, a->value_dim, 2, &from, &to)
                     : extent(a->decay, rows, a->decay_row_stride, H, a->decay_head_stride, 1, 4, &from, &to);
        if (!fits)
            return LMC_ERR_INVALID_ARG;
        if (std::max(at, from) < std::min(end, to))
            return LMC_ERR_OVERLAP;
    }
    return LMC_OK;
}

void plan_linear(LinearPlan &P, const lmc_layout *L, const lmc_linear *a, int64_t rows, void *pool, uint32_t *status) {
    const lmc_layer_desc &d = L->desc[a->layer];
    P.pages = reinterpret_cast<float *>(static_cast<uint8_t *>(pool) + d.base + L->specs[a->layer].conv_bytes);
    P.page_stride = d.stride / 4;
    P.num_blocks = L->num_blocks;
    P.table = a->table.table;
    P.row_stride = a->table.row_stride;
    P.cols = a->table.num_cols;
    P.lengths = a->lengths;
    P.q = static_cast<const uint16_t *>(a->q);
    P.k = static_cast<const uint16_t *>(a->k);
    P.v = static_cast<const uint16_t *>(a->v);
    P.out = static_cast<uint16_t *>(a->out);
    P.decay = a->decay;
    P.q_row = a->q_row_stride, P.q_head = a->q_head_stride;
    P.k_row = a->k_row_stride, P.k_head = a->k_head_stride;
    P.v_row = a->v_row_stride, P.v_head = a->v_head_stride;
    P.out_row = a->out_row_stride, P.out_head = a->out_head_stride;
    P.decay_row = a->decay_row_stride, P.decay_head = a->decay_head_stride;
    P.num_rows = rows;
    P.status = status;
    P.R = a->num_requests;
    P.H = a->num_heads;
    P.shared = a->num_heads / a->num_key_heads;
    P.dk = a->key_dim;
    P.dv = a->value_dim;
    P.block_size = (int32_t)L->block_size;
    P.bf16 = a->dtype == LMC_E_BF16;
    P.scale = a->scale;
}

int launch_steps(const LinearPlan &P, cudaStream_t stream) {
    const int64_t grid = (int64_t)P.R * P.H * ((P.dv + 4 * kStepLanes - 1) / (4 * kStepLanes));
    if (grid > INT32_MAX)
        return LMC_ERR_OVERFLOW;
    return follow(lmc_linear_step_kernel<kStepLanes>, dim3((unsigned)grid), kStepThreads, 0, stream, P) ? LMC_OK : LMC_ERR_CUDA;
}

// Tokens of an SM's even share: no request is cut into segments shorter than that.
int64_t segment_of(int64_t num_rows, int64_t H) {
    return std::max(kLeastSegment, ((num_rows * H + kSms - 1) / kSms + kTile - 1) / kTile * kTile);
}

struct ScanWork {
    int64_t segment, slots, totals, owners, bytes;  // tokens; offsets
};

ScanWork scan_work(int64_t rec_bytes, int64_t H, int64_t num_rows) {
    ScanWork W;
    W.segment = segment_of(num_rows, H);
    // at least num_rows / segment, and never less for more rows: memory for the largest
    // call serves all smaller ones
    const int64_t n = std::min(num_rows / kLeastSegment, kSms / H);
    W.slots = 0;
    W.totals = (n * rec_bytes + 255) / 256 * 256;
    W.owners = W.totals + n * H * 8;
    W.bytes = std::max<int64_t>(256, (W.owners + n * 4 + 255) / 256 * 256);
    return W;
}

// (values, rows, heads) of 16 bits each, read in boxes of a tile's rows of one
// head: of both panels of 64 values at once (`whole`), or of one; or written (`result`)
// in boxes of 32 values.
bool rows_map(CUtensorMap *map, bool bf16, const void *base, int64_t dim, int64_t rows, int64_t heads, int64_t row,
              int64_t head, bool whole, bool result = false) {
    const EncodeTiled fn = encoder();
    if (fn == nullptr)
        return false;
    const cuuint64_t panels = whole ? (cuuint64_t)dim / 64 : 1;
    const cuuint64_t row_bytes = rows > 1 ? (cuuint64_t)row * 2 : (cuuint64_t)dim * 2;
    const cuuint64_t head_bytes = heads > 1 ? (cuuint64_t)head * 2 : (cuuint64_t)dim * 2;
    const cuuint64_t dims[4] = {whole ? 64 : (cuuint64_t)dim, (cuuint64_t)rows, panels, (cuuint64_t)heads};
    const cuuint64_t strides[3] = {row_bytes, 128, head_bytes};
    const cuuint32_t boxes[4] = {result ? 32u : 64u, kTile, (cuuint32_t)panels, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<void *>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              result ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" int lmc_linear_step(const lmc_layout *L, const lmc_linear *a, void *pool, uint32_t *status, void *stream) {
    if (a == nullptr)
        return LMC_ERR_INVALID_ARG;
    if (const int rc = check_linear(L, a, a->num_requests, pool, status); rc != LMC_OK || a->num_requests == 0)
        return rc;
    LinearPlan P = {};
    plan_linear(P, L, a, a->num_requests, pool, status);
    return launch_steps(P, static_cast<cudaStream_t>(stream));
}

extern "C" int lmc_linear_scan_workspace(const lmc_layout *L, int32_t layer, int32_t num_requests, int64_t num_rows,
                                         int32_t num_heads, int64_t *out) {
    if (L == nullptr || layer < 0 || (size_t)layer >= L->desc.size() || L->specs[layer].kind != LMC_LAYER_KDA ||
        num_requests < 0 || num_requests > 1 << 20 || num_rows < 0 || num_rows > INT32_MAX || num_heads <= 0 ||
        num_heads > 65535 || out == nullptr)
        return LMC_ERR_INVALID_ARG;
    *out = scan_work(L->specs[layer].rec_bytes, num_heads, num_rows).bytes;
    return LMC_OK;
}

extern "C" int lmc_linear_scan(const lmc_layout *L, const lmc_linear *a, const int32_t *starts, int64_t num_rows,
                               void *pool, void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream) {
    if (const int rc = check_linear(L, a, num_rows, pool, status); rc != LMC_OK)
        return rc;
    if (num_rows > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    const ScanWork W = scan_work(L->specs[a->layer].rec_bytes, a->num_heads, num_rows);
    if (workspace == nullptr || workspace_bytes < W.bytes || starts == nullptr)
        return LMC_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0 || ((uintptr_t)starts & 3) != 0)
        return LMC_ERR_ALIGN;
    if (num_rows == 0 || a->num_requests == 0)
        return LMC_OK;
    ScanPlan P = {};
    plan_linear(P.L, L, a, num_rows, pool, status);
    P.L.starts = starts;
    P.segment = W.segment;
    P.slots = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + W.slots);
    P.totals = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + W.totals);
    P.owners = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + W.owners);
    P.k_panels = (P.L.dk + 63) / 64;
    P.v_panels = (P.L.dv + 63) / 64;
    const bool bf16 = P.L.bf16, whole_k = P.L.dk % 64 == 0, whole_v = P.L.dv % 64 == 0;
    P.wide_out = ((uintptr_t)a->out & 15) == 0 && (num_rows == 1 || a->out_row_stride % 8 == 0) &&
                 (a->num_heads == 1 || a->out_head_stride % 8 == 0) &&
                 a->out_row_stride < (int64_t)1 << 36 && a->out_head_stride < (int64_t)1 << 36;
    P.k_copies = whole_k ? 1 : P.k_panels;
    P.v_copies = whole_v ? 1 : P.v_panels;
    const int64_t H = a->num_heads, K = a->num_key_heads;
    const int64_t cuts = P.cuts = num_rows / W.segment;
    const int64_t grid = (cuts + a->num_requests) * H, states = cuts * H;
    if (grid > INT32_MAX)
        return LMC_ERR_OVERFLOW;
    if (!rows_map(&P.q, bf16, a->q, P.L.dk, num_rows, K, a->q_row_stride, a->q_head_stride, whole_k) ||
        !rows_map(&P.k, bf16, a->k, P.L.dk, num_rows, K, a->k_row_stride, a->k_head_stride, whole_k) ||
        !rows_map(&P.v, bf16, a->v, P.L.dv, num_rows, H, a->v_row_stride, a->v_head_stride, whole_v) ||
        (P.wide_out &&
         !rows_map(&P.out, bf16, a->out, P.L.dv, num_rows, H, a->out_row_stride, a->out_head_stride, false, true)))
        return LMC_ERR_CUDA;
    auto scan = bf16 ? lmc_linear_scan_kernel<true, false> : lmc_linear_scan_kernel<false, false>;
    auto segments = bf16 ? lmc_linear_scan_kernel<true, true> : lmc_linear_scan_kernel<false, true>;
    static std::atomic<uint64_t> allowed[4];
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!allow_shared_memory(allowed[bf16], scan, kScanMemory) ||
        !allow_shared_memory(allowed[2 + bf16], segments, kScanMemory))
        return LMC_ERR_CUDA;
    if (cuts >= 2) {  // a request may be cut
        if (!follow(segments, dim3((unsigned)states), kScanThreads, kScanMemory, s, P))
            return LMC_ERR_CUDA;
        const int64_t parts = (P.L.dk * P.L.dv / 4 + kJoinThreads - 1) / kJoinThreads;
        if (cuts >= 3 && !follow(lmc_linear_join_kernel, dim3((unsigned)(states * parts)), kJoinThreads, 0, s, P))
            return LMC_ERR_CUDA;
    }
    return follow(scan, dim3((unsigned)grid), kScanThreads, kScanMemory, s, P) ? LMC_OK : LMC_ERR_CUDA;
}
