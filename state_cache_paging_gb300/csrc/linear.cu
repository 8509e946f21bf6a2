// linear.cu -- linear attention with a decay for each head over the states that
// KDA layers' pages hold, for sm_103a.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
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
    uint32_t bad;       // status bits
};

__device__ __forceinline__ Span span_of(const LinearPlan &P, int r) {
    Span S;
    S.row = r;
    S.count = 1;
    S.first = -1;
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
            const int32_t end = __ldca(blocks + last / P.block_size);
            if (S.before > 0) {
                S.first = __ldca(blocks + (S.before - 1) / P.block_size);
                if (S.first < 0 || S.first >= P.num_blocks)
                    S.bad |= S.first == -1 ? LMC_ST_NO_SNAPSHOT : LMC_ST_BLOCK_OOR;
            }
            if (end < 0 || end >= P.num_blocks)
                S.bad |= end == -1 ? LMC_ST_NO_SNAPSHOT : LMC_ST_BLOCK_OOR;
        }
    }
    if (S.bad != 0 || S.before < 0)
        S.count = 0;
    return S;
}

// ---------------------------------------------------------------------------
// One token at a time
// ---------------------------------------------------------------------------

// A CTA holds a head's state in registers: kLanes lanes take a row (four
// columns each), 256 / kLanes rows at a time. Bound by reading and writing the
// state: 2 x 64 KB for a head of 128 x 128, 7 KB of everything else.
constexpr int kStepThreads = 256;

template <int kLanes>
__global__ void __launch_bounds__(kStepThreads) lmc_linear_step_kernel(const __grid_constant__ LinearPlan P) {
    constexpr int kRows = kStepThreads / kLanes;   // at a time
    constexpr int kTurns = kMaxDim / kRows;
    __shared__ float qs[kMaxDim], ks[kMaxDim];
    __shared__ float4 sums[kRows][kLanes];
    const int h = blockIdx.x % P.H, r = blockIdx.x / P.H;
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes, c = 4 * lane;
    wait_for_launch();
    let_next_start();
    const Span S = span_of(P, r);
    if (S.bad && h == 0 && threadIdx.x == 0)
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
    for (int64_t t = 0; t < S.count; t++) {
        const int64_t x = S.row + t;
        if (t > 0)
            __syncthreads();
        if ((int)threadIdx.x < P.dk)
            qs[threadIdx.x] = from_q(P.q[x * P.q_row + kh * P.q_head + threadIdx.x], P.bf16);
        else if (threadIdx.x >= kMaxDim && (int)threadIdx.x - kMaxDim < P.dk)
            ks[threadIdx.x - kMaxDim] = from_q(P.k[x * P.k_row + kh * P.k_head + threadIdx.x - kMaxDim], P.bf16);
        float4 v = {}, o = {};
        if (mine) {
            const uint2 w = *reinterpret_cast<const uint2 *>(P.v + x * P.v_row + h * P.v_head + c);
            v = make_float4(from_q(w.x & 0xffff, P.bf16), from_q(w.x >> 16, P.bf16), from_q(w.y & 0xffff, P.bf16),
                            from_q(w.y >> 16, P.bf16));
        }
        const float a = expf(fmaxf(P.decay[x * P.decay_row + h * P.decay_head], kLeastDecay));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTurns; i++) {
            const int j = row + i * kRows;
            if (j < P.dk) {
                const float k = ks[j], q = qs[j];
                s[i].x = fmaf(k, v.x, a * s[i].x);
                s[i].y = fmaf(k, v.y, a * s[i].y);
                s[i].z = fmaf(k, v.z, a * s[i].z);
                s[i].w = fmaf(k, v.w, a * s[i].w);
                o.x = fmaf(q, s[i].x, o.x);
                o.y = fmaf(q, s[i].y, o.y);
                o.z = fmaf(q, s[i].z, o.z);
                o.w = fmaf(q, s[i].w, o.w);
            }
        }
        // the state after a block's last token, and after the call's
        const int64_t done = S.before + t + 1;
        if (t + 1 == S.count || done % P.block_size == 0) {
            const int32_t block = __ldca(P.table + r * P.row_stride + (done - 1) / P.block_size);
            if (block >= 0 && block < P.num_blocks) {
                if (mine) {
                    float *page = P.pages + block * P.page_stride + at;
#pragma unroll
                    for (int i = 0; i < kTurns; i++)
                        if (row + i * kRows < P.dk)
                            __stcs(reinterpret_cast<float4 *>(page + (int64_t)(row + i * kRows) * P.dv), s[i]);
                }
            } else if (block != -1 && threadIdx.x == 0) {
                atomicOr(P.status, LMC_ST_BLOCK_OOR);
            }
        }
        sums[row][lane] = o;
        __syncthreads();
        if ((int)threadIdx.x < P.dv) {
            float y = 0.0f;
#pragma unroll 8
            for (int i = 0; i < kRows; i++)
                y += reinterpret_cast<const float *>(sums[i])[threadIdx.x];
            P.out[x * P.out_row + h * P.out_head + threadIdx.x] = to_out(y * P.scale, P.bf16);
        }
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
    const int64_t grid = (int64_t)P.R * P.H;
    if (grid > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    auto kern = P.dv <= 32 ? lmc_linear_step_kernel<8> : P.dv <= 64 ? lmc_linear_step_kernel<16> : lmc_linear_step_kernel<32>;
    return follow(kern, dim3((unsigned)grid), kStepThreads, 0, stream, P) ? LMC_OK : LMC_ERR_CUDA;
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
        num_requests < 0 || num_requests > 1 << 20 || num_rows < 0 || num_heads <= 0 || num_heads > 65535 || out == nullptr)
        return LMC_ERR_INVALID_ARG;
    *out = 256;
    return LMC_OK;
}

extern "C" int lmc_linear_scan(const lmc_layout *L, const lmc_linear *a, const int32_t *starts, int64_t num_rows,
                               void *pool, void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream) {
    if (const int rc = check_linear(L, a, num_rows, pool, status); rc != LMC_OK)
        return rc;
    if (workspace == nullptr || workspace_bytes < 256 || starts == nullptr)
        return LMC_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0 || ((uintptr_t)starts & 3) != 0)
        return LMC_ERR_ALIGN;
    if (num_rows == 0 || a->num_requests == 0)
        return LMC_OK;
    LinearPlan P = {};
    plan_linear(P, L, a, num_rows, pool, status);
    P.starts = starts;
    return launch_steps(P, static_cast<cudaStream_t>(stream));
}
