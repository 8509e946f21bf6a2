// attend.cu -- attention of one new token per request over the paged entries
// of an MLA or SWA layer, for sm_103a.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "lmc_internal.h"

namespace {

constexpr int kMaxEntry = 576;
constexpr int kMaxValue = 512;

struct AttendPlan {
    const uint8_t *pool;  // + the layer's base
    int64_t block_stride;
    int64_t num_blocks;
    int32_t block_size;
    int32_t token_bytes;
    const int32_t *table;
    int64_t row_stride;
    int64_t num_cols;
    const int32_t *lengths;
    int64_t max_length;
    int64_t window;  // 0: none
    const uint16_t *q;
    int64_t q_request_stride, q_head_stride;
    uint16_t *out;
    int64_t out_request_stride, out_head_stride;
    float *lse;  // caller's, or NULL
    int64_t lse_request_stride;
    float *weights;
    int64_t weights_request_stride;
    float *lse_all;  // workspace [R][H]
    uint32_t *status;
    float softmax_scale;
    float scale;
    int32_t E, V, H;
    int32_t dtype, q_dtype;
};

__device__ __forceinline__ float load16(uint16_t bits, int32_t dtype) {
    return dtype == LMC_E_BF16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits));
}

__device__ __forceinline__ float load_entry(const uint8_t *e, int32_t i, const AttendPlan &P) {
    if (P.dtype == LMC_E_E4M3)
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(e[i], __NV_E4M3))) * P.scale;
    return load16(reinterpret_cast<const uint16_t *>(e)[i], P.dtype);
}

// First token of the request's range; false when the request is not served.
__device__ __forceinline__ bool token_range(const AttendPlan &P, int64_t r, int64_t &lo, int64_t &L) {
    L = __ldg(P.lengths + r);
    lo = P.window > 0 ? max((int64_t)0, L - P.window) : 0;
    return L >= 0 && L <= P.max_length && L <= P.num_cols * P.block_size;
}

__device__ __forceinline__ const uint8_t *entry_at(const AttendPlan &P, int64_t r, int64_t t, uint32_t &bad) {
    const int64_t page = t / P.block_size;
    const int32_t block = __ldg(P.table + r * P.row_stride + page);
    if (block < 0 || block >= P.num_blocks) {
        bad |= block == -1 ? LMC_ST_NO_BLOCK : LMC_ST_BLOCK_OOR;
        return nullptr;
    }
    return P.pool + (int64_t)block * P.block_stride + (t - page * P.block_size) * P.token_bytes;
}

constexpr int kWarps = 8;
constexpr int kPer = kMaxEntry / 32;
constexpr int kValPer = kMaxValue / 32;

// One CTA per (head, request), a token per warp at a time: the entry's values
// lie across the lanes, the running maximum and sum of each warp are joined
// at the end.
__global__ void __launch_bounds__(32 * kWarps) lmc_attend_kernel(const __grid_constant__ AttendPlan P) {
    const int64_t r = blockIdx.y;
    const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t lo, L;
    if (!token_range(P, r, lo, L)) {
        if (threadIdx.x == 0)
            atomicOr(P.status, LMC_ST_BAD_JOB);
        return;
    }
    float q[kPer], acc[kValPer];
#pragma unroll
    for (int i = 0; i < kPer; i++)
        q[i] = lane + 32 * i < P.E
                   ? load16(P.q[r * P.q_request_stride + h * P.q_head_stride + lane + 32 * i], P.q_dtype)
                   : 0.0f;
#pragma unroll
    for (int i = 0; i < kValPer; i++)
        acc[i] = 0.0f;
    float m = -INFINITY, sum = 0.0f;
    uint32_t bad = 0;
    for (int64_t t = lo + warp; t < L; t += kWarps) {
        const uint8_t *e = entry_at(P, r, t, bad);
        if (e == nullptr)
            continue;
        float v[kPer], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            v[i] = lane + 32 * i < P.E ? load_entry(e, lane + 32 * i, P) : 0.0f;
            dot = fmaf(q[i], v[i], dot);
        }
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = dot * P.softmax_scale;
        const float top = fmaxf(m, x);
        const float keep = m == top ? 1.0f : expf(m - top), p = expf(x - top);
        m = top;
        sum = sum * keep + p;
#pragma unroll
        for (int i = 0; i < kValPer; i++)
            acc[i] = acc[i] * keep + p * v[i];
    }
    if (bad)
        atomicOr(P.status, bad);
    __shared__ float s_m[kWarps], s_sum[kWarps], s_acc[kWarps][kMaxValue];
    if (lane == 0) {
        s_m[warp] = m;
        s_sum[warp] = sum;
    }
    for (int i = 0; i < kValPer; i++)
        s_acc[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; w++)
        top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kWarps; w++)
        total += s_sum[w] == 0.0f ? 0.0f : s_sum[w] * expf(s_m[w] - top);
    for (int v = threadIdx.x; v < P.V; v += blockDim.x) {
        float x = 0.0f;
        for (int w = 0; w < kWarps; w++)
            x += s_sum[w] == 0.0f ? 0.0f : s_acc[w][v] * expf(s_m[w] - top);
        x = total == 0.0f ? 0.0f : x / total;
        P.out[r * P.out_request_stride + h * P.out_head_stride + v] =
            P.q_dtype == LMC_E_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
    }
    if (threadIdx.x == 0) {
        const float lse = total == 0.0f ? -INFINITY : top + logf(total);
        P.lse_all[r * P.H + h] = lse;
        if (P.lse != nullptr)
            P.lse[r * P.lse_request_stride + h] = lse;
    }
}

// One warp per token: the sum over the heads of its probability.
__global__ void __launch_bounds__(32 * kWarps) lmc_attend_weights_kernel(const __grid_constant__ AttendPlan P) {
    const int64_t r = blockIdx.y;
    const int lane = threadIdx.x & 31;
    int64_t lo, L;
    if (!token_range(P, r, lo, L))
        return;
    for (int64_t t = lo + blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5); t < L; t += (int64_t)gridDim.x * kWarps) {
        uint32_t bad = 0;
        const uint8_t *e = entry_at(P, r, t, bad);
        if (e == nullptr)
            continue;
        float v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++)
            v[i] = lane + 32 * i < P.E ? load_entry(e, lane + 32 * i, P) : 0.0f;
        float w = 0.0f;
        for (int h = 0; h < P.H; h++) {
            const uint16_t *q = P.q + r * P.q_request_stride + h * P.q_head_stride;
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; i++)
                if (lane + 32 * i < P.E)
                    dot = fmaf(load16(q[lane + 32 * i], P.q_dtype), v[i], dot);
            for (int o = 16; o > 0; o >>= 1)
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            w += expf(dot * P.softmax_scale - P.lse_all[r * P.H + h]);
        }
        if (lane == 0)
            P.weights[r * P.weights_request_stride + t] += w;
    }
}

bool aligned16(int64_t x) { return (x & 15) == 0; }

}  // namespace

extern "C" int lmc_attend_workspace(const lmc_layout *L, int32_t layer, int32_t num_requests, int32_t num_heads,
                                    int32_t value_dim, int64_t max_length, int with_weights, int64_t *out) {
    (void)with_weights;
    if (L == nullptr || out == nullptr || layer < 0 || (size_t)layer >= L->desc.size() ||
        L->specs[layer].kind == LMC_LAYER_KDA || num_requests < 0 || num_heads <= 0 || value_dim <= 0 ||
        value_dim > kMaxValue || max_length <= 0 || max_length > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    int64_t n;
    if (!lmc::mul_ok((int64_t)num_requests * 4, num_heads, &n))
        return LMC_ERR_OVERFLOW;
    *out = n;
    return LMC_OK;
}

extern "C" int lmc_attend(const lmc_layout *L, const lmc_entries *e, const void *pool, const lmc_attention *a,
                          void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream) {
    if (const int rc = lmc::check_entries(L, e); rc != LMC_OK)
        return rc;
    if (a == nullptr || status == nullptr || (a->q_dtype != LMC_E_BF16 && a->q_dtype != LMC_E_F16) ||
        (e->dtype != LMC_E_E4M3 && e->dtype != a->q_dtype) || e->entry_dim % 16 != 0 || e->entry_dim > kMaxEntry ||
        a->num_heads <= 0 || a->value_dim <= 0 || a->value_dim % 8 != 0 || a->value_dim > e->entry_dim ||
        a->value_dim > kMaxValue || !std::isfinite(a->softmax_scale) || a->max_length <= 0 ||
        a->max_length > INT32_MAX)
        return LMC_ERR_INVALID_ARG;
    const int64_t R = e->num_requests, H = a->num_heads;
    if (a->q_request_stride < 0 || a->q_head_stride < 0 || a->out_request_stride < 0 || a->out_head_stride < 0 ||
        a->q_request_stride % 8 != 0 || a->q_head_stride % 8 != 0 || (H > 1 && a->out_head_stride < a->value_dim) ||
        (R > 1 && a->out_request_stride < a->value_dim) ||
        (a->lse != nullptr && a->lse_request_stride < H) ||
        (a->weights != nullptr && a->weights_request_stride < a->max_length))
        return LMC_ERR_INVALID_ARG;
    int64_t need;
    if (const int rc = lmc_attend_workspace(L, e->layer, e->num_requests, a->num_heads, a->value_dim, a->max_length,
                                            a->weights != nullptr, &need); rc != LMC_OK)
        return rc;
    if (R > 0 && (pool == nullptr || a->lengths == nullptr || a->q == nullptr || a->out == nullptr ||
                  workspace == nullptr || workspace_bytes < need))
        return LMC_ERR_INVALID_ARG;
    const lmc_layer_desc &d = L->desc[e->layer];
    if ((((uintptr_t)status | (uintptr_t)a->lengths | (uintptr_t)a->lse | (uintptr_t)a->weights) & 3) != 0 ||
        !aligned16((int64_t)(uintptr_t)pool) || !aligned16(d.base) || !aligned16(d.stride) ||
        !aligned16((int64_t)(uintptr_t)a->q) || ((uintptr_t)a->out & 1) != 0 || ((uintptr_t)workspace & 255) != 0)
        return LMC_ERR_ALIGN;
    if (R == 0)
        return LMC_OK;
    AttendPlan P = {};
    P.pool = static_cast<const uint8_t *>(pool) + d.base;
    P.block_stride = d.stride;
    P.num_blocks = L->num_blocks;
    P.block_size = (int32_t)L->block_size;
    P.token_bytes = (int32_t)L->specs[e->layer].token_bytes;
    P.table = e->table.table;
    P.row_stride = e->table.row_stride;
    P.num_cols = e->table.num_cols;
    P.lengths = a->lengths;
    P.max_length = a->max_length;
    P.window = L->specs[e->layer].kind == LMC_LAYER_SWA ? L->specs[e->layer].window : 0;
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
    P.lse_all = static_cast<float *>(workspace);
    P.status = status;
    P.softmax_scale = a->softmax_scale;
    P.scale = e->scale;
    P.E = e->entry_dim;
    P.V = a->value_dim;
    P.H = a->num_heads;
    P.dtype = e->dtype;
    P.q_dtype = a->q_dtype;
    if (R > 65535 || H > 65535)
        return LMC_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    lmc_attend_kernel<<<dim3((unsigned)H, (unsigned)R), 32 * kWarps, 0, s>>>(P);
    if (a->weights != nullptr) {
        const unsigned n = (unsigned)std::min<int64_t>(512, (a->max_length + kWarps - 1) / kWarps);
        lmc_attend_weights_kernel<<<dim3(n, (unsigned)R), 32 * kWarps, 0, s>>>(P);
    }
    return cudaGetLastError() == cudaSuccess ? LMC_OK : LMC_ERR_CUDA;
}
