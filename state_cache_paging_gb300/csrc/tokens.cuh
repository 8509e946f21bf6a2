// tokens.cuh -- what the kernels that write single tokens' entries share: where
// an entry lies, and values turned to fp8 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "lmc_internal.h"

namespace lmc {

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
__device__ __forceinline__ float quotient_by_inverse(float x, float scale, float inverse) {
    const float q = x * inverse;
    const float exact = fmaf(fmaf(-q, scale, x), inverse, q);
    return fabsf(q) < 4096.0f && q != 0.0f ? exact : q;  // (-0 stays -0)
}
__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
    return inverse == 0.0f ? __fdiv_rn(x, scale) : quotient_by_inverse(x, scale, inverse);
}

// Two values as fp8 codes: saturated (satfinite), half to even, NaN to NaN.
__device__ __forceinline__ uint32_t codes2(float2 v, float scale, float inverse) {
    return __nv_cvt_float2_to_fp8x2(make_float2(quotient(v.x, scale, inverse), quotient(v.y, scale, inverse)),
                                    __NV_SATFINITE, __NV_E4M3);
}

inline TokenTable token_table(const lmc_block_table &t) { return TokenTable{t.table, t.row_stride, (int32_t)t.num_cols}; }

// RN(1 / scale) for quotient(); 0 where its correction would not hold.
inline float inverse_scale(float scale) {
    uint32_t bits;
    std::memcpy(&bits, &scale, 4);
    return scale >= 0x1p-100f && scale <= 0x1p100f && (bits & 0x7fffffu) != 0x7fffffu ? 1.0f / scale : 0.0f;
}

}  // namespace lmc
