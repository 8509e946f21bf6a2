// rotate.cu -- norms and position rotations of heads, for sm_103a: queries (and
// keys) as activations, and entries on their way into a paged attention layer.
//
// Mathematics. y = x / sqrt(mean(x^2) + eps) * w on a head's first values, then
// pairs turned by t = position * frequency. The angle is kept as a whole number
// of 2^-64 turns: a step F = frequency * 2^64 / (2 pi), from the frequency's
// significand times a 128-bit constant, times the position modulo 2^64. Its upper
// 32 bits are the angle to 2^-32 turns however far the position is, without
// 64-bit floating point (which this GPU is slow at).
//
// Bound: the copy rate. A row's angles are the same for all its heads, so a CTA
// takes whole rows, makes their cosines and sines once in shared memory, and
// then a group of 4 to 32 lanes takes a head: it holds the head's values in
// registers between the sum of squares and the result, so they are read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "follow.cuh"
#include "lmc_internal.h"
#include "tokens.cuh"

namespace {

using namespace lmc;

constexpr int kThreads = 256;
constexpr int kMaxRows = 64;           // of a CTA
constexpr int kMaxAngles = 2048;       // of a CTA's rows together (16 KB), where it has several
constexpr int kMaxHeadDim = 4096;

constexpr int kManyCtas = 152 * 16;   // waves of CTAs enough to even out

// Activations; a page's entries, as they are or as fp8 codes (kDivided: of a scale that
// has no inverse to multiply by, or too large a one; such calls are rare and take the
// slower kernel).
enum Result { kRows, kEntries, kCodes, kDivided };
__host__ __device__ constexpr bool codes(Result to) { return to == kCodes || to == kDivided; }

struct RotatePlan {
    const uint16_t *x;
    int64_t x_row, x_head;      // strides, elements
    uint16_t *out;
    int64_t out_row, out_head;
    const float *weight;
    const float *frequencies;
    const int32_t *angles;      // positions they are made from
    // entries
    Pages pages;
    TokenTable table;
    const int32_t *requests;
    const int32_t *positions;
    uint8_t *pool;
    uint32_t *status;
    int32_t num_requests;
    float code_scale, code_inverse;
    int64_t num_rows;
    int32_t rows_per_cta;
    int32_t heads, head_dim, norm_dim, rot_first, half;
    int32_t rest;               // values behind the heads, taken as they are,
    int32_t rest_unit;          // so many at a time
    int32_t units;              // heads and units of the rest, per row
    int32_t turned;             // a head's items that are turned,
    int32_t items;              // and all of them
    int32_t group;              // lanes of a head
    int32_t row_step, unit_step; // from a group's unit to its next
    int32_t angle_rows, angle_step; // from a thread's angle to its next
    int32_t pairs;
    int32_t touch_only;         // the result lies where x does
    float eps, mscale, inverse_norm_dim;
};

// frequency * 2^64 / (2 pi), the nearest whole number modulo 2^64: the significand
// times 2^128 / (2 pi), three words, shifted by the exponent. (Off by half, which 2^31
// positions make 2^-34 turns.)
__device__ __forceinline__ uint64_t step_of(float frequency) {
    const uint32_t bits = __float_as_uint(frequency);
    const int exponent = (int)(bits >> 23 & 255u);
    const uint64_t m = (bits & 0x7fffffu) | (exponent > 0 ? 0x800000u : 0u);
    const uint64_t c1 = 2935890503282001226ull, c0 = 9154082963658192752ull;
    const int down = 150 - max(exponent, 1);  // frequency = m * 2^-down
    const uint64_t w0 = m * c0, carried = __umul64hi(m, c0), w1 = m * c1 + carried;
    const uint64_t w2 = __umul64hi(m, c1) + (w1 < carried);
    uint64_t f = 0;
    if (down < 0)
        f = down > -64 ? w1 << -down | w0 >> (64 + down) : 0;
    else if (down == 0)
        f = w1 + (w0 >> 63);
    else if (down < 64)
        f = (w1 >> down | w2 << (64 - down)) + (w1 >> (down - 1) & 1);
    else if (down == 64)
        f = w2 + (w1 >> 63);
    else if (down < 128)
        f = (w2 >> (down - 64)) + (w2 >> (down - 65) & 1);
    return bits >> 31 ? 0 - f : f;
}

// (cos, sin) of position steps: the nearest quarter turn apart, the rest r, at most
// an eighth of a turn, by the series of sine and cosine (what is left out is below
// 2^-28 of the result). sincospif takes twice the instructions.
__device__ __forceinline__ float2 turn(int32_t position, uint64_t step) {
    const uint64_t phase = (uint64_t)(int64_t)position * step;
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const float r = (float)(int32_t)((phase - ((uint64_t)quarter << 62)) >> 32) * (6.28318530717958647693f * 0x1p-32f);
    const float x = r * r;
    float s = fmaf(x, 1.0f / 362880.0f, -1.0f / 5040.0f), c = fmaf(x, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    s = fmaf(s, x, 1.0f / 120.0f);
    c = fmaf(c, x, -1.0f / 720.0f);
    s = fmaf(s, x, -1.0f / 6.0f);
    c = fmaf(c, x, 1.0f / 24.0f);
    s = fmaf(s * x, r, r);
    c = fmaf(c, x, -0.5f);
    c = fmaf(c, x, 1.0f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

template <typename T2>
__device__ __forceinline__ float2 widen(uint32_t v) {
    return to_float2(*reinterpret_cast<const T2 *>(&v));
}
template <typename T2>
__device__ __forceinline__ uint32_t narrow(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat162>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half2>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A head's items: what is turned comes first (W pairs of pieces a half apart,
// or pieces of W whole pairs; single pairs where W is 1), then the pieces of W
// values that are not. First value of item i's piece (and of its second one).
template <int W>
__device__ __forceinline__ int first_value(const RotatePlan &P, int i, int &second) {
    if (i < P.turned) {
        if (W == 1 && P.pairs) {
            second = P.rot_first + 2 * i + 1;
            return P.rot_first + 2 * i;
        }
        second = P.pairs ? -1 : P.rot_first + P.half + i * W;
        return P.rot_first + i * W;
    }
    second = -1;
    const int v = (i - P.turned) * W;
    return v < P.rot_first ? v : v + 2 * P.half;
}

template <int W>
__device__ __forceinline__ void load_values(uint32_t (&raw)[(W + 1) / 2], const uint16_t *at) {
    if constexpr (W == 8) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(at));
        raw[0] = v.x, raw[1] = v.y, raw[2] = v.z, raw[3] = v.w;
    } else {
        raw[0] = *at;
    }
}

template <typename T2, int W>
__device__ __forceinline__ void widen_values(float (&x)[W], const uint32_t (&raw)[(W + 1) / 2]) {
    if constexpr (W == 8) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float2 v = widen<T2>(raw[k]);
            x[2 * k] = v.x, x[2 * k + 1] = v.y;
        }
    } else {
        x[0] = widen<T2>(raw[0]).x;
    }
}

// What is to be divided by the scale, or has been multiplied by its inverse already
// (`scaled`), as a pair of codes.
template <Result kTo>
__device__ __forceinline__ uint32_t code_pair(const RotatePlan &P, float x, float y, bool scaled) {
    if (kTo == kDivided)
        x = __fdiv_rn(x, P.code_scale), y = __fdiv_rn(y, P.code_scale);
    else if (!scaled)
        x = quotient_by_inverse(x, P.code_scale, P.code_inverse), y = quotient_by_inverse(y, P.code_scale, P.code_inverse);
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// Values of a result; codes: `scaled` if the scale's inverse is in them (what was
// turned, and most of what was normalised).
template <typename T2, int W, Result kTo>
__device__ __forceinline__ void store_values(const RotatePlan &P, uint8_t *at, const float (&y)[W], bool scaled) {
    if constexpr (codes(kTo) && W == 8) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = code_pair<kTo>(P, y[2 * k], y[2 * k + 1], scaled);
        __stcs(reinterpret_cast<uint2 *>(at), make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16));
    } else if constexpr (codes(kTo)) {
        *at = (uint8_t)code_pair<kTo>(P, y[0], 0.0f, scaled);
    } else if constexpr (W == 8) {
        __stcs(reinterpret_cast<uint4 *>(at), make_uint4(narrow<T2>(y[0], y[1]), narrow<T2>(y[2], y[3]),
                                                         narrow<T2>(y[4], y[5]), narrow<T2>(y[6], y[7])));
    } else {
        *reinterpret_cast<uint16_t *>(at) = (uint16_t)narrow<T2>(y[0], 0.0f);
    }
}

// One item of a head (or of the rest): normalised, turned, written.
template <typename T2, int W, Result kTo>
__device__ __forceinline__ void finish(const RotatePlan &P, const float2 *cs, uint8_t *dst, int i, int first, int second,
                                       float norm, bool head, const uint32_t (&lo)[(W + 1) / 2],
                                       const uint32_t (&hi)[(W + 1) / 2]) {
    constexpr int kBytes = codes(kTo) ? 1 : 2;
    float a[W], b[W];
    widen_values<T2, W>(a, lo);
    widen_values<T2, W>(b, hi);
    const bool turned = head && i < P.turned;
    if (head && first < P.norm_dim) {
#pragma unroll
        for (int k = 0; k < W; k++)
            a[k] = a[k] * norm * (P.weight != nullptr ? __ldca(P.weight + first + k) : 1.0f);
    }
    if (turned && second >= 0) {
        if (second < P.norm_dim) {
#pragma unroll
            for (int k = 0; k < W; k++)
                b[k] = b[k] * norm * (P.weight != nullptr ? __ldca(P.weight + second + k) : 1.0f);
        }
#pragma unroll
        for (int k = 0; k < W; k++) {
            const float2 r = cs[i * W + k];
            const float x = a[k], y = b[k];
            a[k] = x * r.x - y * r.y;
            b[k] = x * r.y + y * r.x;
        }
        store_values<T2, W, kTo>(P, dst + (int64_t)second * kBytes, b, true);
    } else if (W == 8 && turned) {
#pragma unroll
        for (int k = 0; k < W / 2; k++) {
            const float2 r = cs[i * (W / 2) + k];
            const float x = a[2 * k], y = a[2 * k + 1];
            a[2 * k] = x * r.x - y * r.y;
            a[2 * k + 1] = x * r.y + y * r.x;
        }
    }
    store_values<T2, W, kTo>(P, dst + (int64_t)first * kBytes, a, turned);
}

// Steps of the angles and the rows' cosines and sines in shared memory; where the
// rows' entries lie.
//
// kHalvesOrder, kPairsOrder: in the order in which lanes of consecutive pieces of eight values read
// them, 16 bytes at a time without bank conflicts: a piece's first 16 bytes of all
// pieces, then the second ones. For kHalvesOrder that is the cosines of two angles
// and their sines, for kPairsOrder (cosine, sine) of two angles.
enum Order { kPlainOrder, kHalvesOrder, kPairsOrder };

template <Result kTo, Order kOrder = kPlainOrder>
__device__ __forceinline__ void make_angles(const RotatePlan &P, float2 *cs, uint64_t *steps, uint8_t **dst, int64_t row0,
                                            int rows) {
    if (kTo != kRows && (int)threadIdx.x < rows) {
        const int64_t i = row0 + threadIdx.x;
        const int32_t req = __ldca(P.requests + i);
        int64_t at = -1;
        if (req != -1) {
            uint32_t bad = 0;
            if (req < 0 || req >= P.num_requests)
                bad = LMC_ST_BAD_JOB;
            else
                at = entry_offset(P.pages, P.table, req, __ldca(P.positions + i), bad);
            if (bad)
                atomicOr(P.status, bad);
        }
        dst[threadIdx.x] = at < 0 ? nullptr : P.pool + at;
    }
    for (int k = threadIdx.x; k < P.half; k += kThreads)
        steps[k] = step_of(__ldca(P.frequencies + k));
    __syncthreads();
    // codes: times what the values are divided by, too
    const float scale = kTo == kCodes ? P.mscale * P.code_inverse : P.mscale;
    if (P.half == 0)
        return;
    int row = threadIdx.x / P.half, k = threadIdx.x - row * P.half;
    while (row < rows) {
        const float2 r = turn(__ldca(P.angles + row0 + row), steps[k]);
        if constexpr (kOrder == kHalvesOrder) {
            float *const at = reinterpret_cast<float *>(cs + row * P.half) + ((k >> 1 & 3) * (P.half >> 3) + (k >> 3)) * 4 + (k & 1);
            at[0] = r.x * scale;
            at[2] = r.y * scale;
        } else if constexpr (kOrder == kPairsOrder) {
            cs[row * P.half + ((k >> 1 & 1) * (P.half >> 2) + (k >> 2)) * 2 + (k & 1)] = make_float2(r.x * scale, r.y * scale);
        } else {
            cs[row * P.half + k] = make_float2(r.x * scale, r.y * scale);
        }
        row += P.angle_rows;
        k += P.angle_step;
        if (k >= P.half) {
            k -= P.half;
            row++;
        }
    }
}

// Two binary32 operations at once.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float x, float y) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two plus_product(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Eight values as four pairs: from a piece, times a factor and the weights of the
// values from `at` on (first halves of all pieces, then second ones), turned as the
// head's `piece` (two whole pairs to a float4 of angles, or with the piece half a
// turned part away), and written.
template <typename T2>
__device__ __forceinline__ void open(Two (&x)[4], const uint4 &raw) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 v = widen<T2>(w[k]);
        x[k] = two(v.x, v.y);
    }
}
__device__ __forceinline__ void weigh(Two (&x)[4], const float *weights, int head_dim, float f, int at) {
    const float4 v = *reinterpret_cast<const float4 *>(weights + at / 2);
    const float4 w = *reinterpret_cast<const float4 *>(weights + (head_dim + at) / 2);
    const Two g = two(f, f);
    x[0] = x[0] * g * two(v.x, v.y);
    x[1] = x[1] * g * two(v.z, v.w);
    x[2] = x[2] * g * two(w.x, w.y);
    x[3] = x[3] * g * two(w.z, w.w);
}
__device__ __forceinline__ void turn_pairs(Two (&a)[4], const float2 *angles, int half, int piece) {
    const float4 *const r = reinterpret_cast<const float4 *>(angles) + piece;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const float4 c = r[k * (half >> 2)];
        const float2 u = apart(a[2 * k]), v = apart(a[2 * k + 1]);
        a[2 * k] = plus_product(two(u.x, u.x), two(c.x, c.y), two(u.y, u.y) * two(-c.y, c.x));
        a[2 * k + 1] = plus_product(two(v.x, v.x), two(c.z, c.w), two(v.y, v.y) * two(-c.w, c.z));
    }
}
__device__ __forceinline__ void turn_halves(Two (&a)[4], Two (&b)[4], const float2 *angles, int half, int piece) {
    const float4 *const r = reinterpret_cast<const float4 *>(angles) + piece;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float4 c = r[k * (half >> 3)];
        const Two u = a[k], v = b[k], cosine = two(c.x, c.y);
        a[k] = plus_product(u, cosine, v * two(-c.z, -c.w));
        b[k] = plus_product(v, cosine, u * two(c.z, c.w));
    }
}
// `plain`: codes of values that were neither normalised nor turned, as lmc_append does.
template <typename T2, Result kTo>
__device__ __forceinline__ void put(const RotatePlan &P, uint8_t *at, const Two (&x)[4], bool plain = false) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 v = apart(x[k]);
        y[2 * k] = v.x;
        y[2 * k + 1] = v.y;
    }
    if (codes(kTo) && plain)
        store_values<T2, 8, kTo>(P, at, y, false);
    else
        store_values<T2, 8, kTo>(P, at, y, true);
}

// Pieces of eight values (16 bytes), a head's items held in registers by a group of
// lanes, kItems each: a lane has the same items of every head, so where they lie is
// found once, and asks for its next head's before it turns this one's. Values are
// widened once and multiplied by pairs; angles and weights (1 where there is no norm)
// lie in shared memory as lanes read them. (32768 rows of 32 heads of 128 values,
// normalised and turned: 90 us, 88 % of the copy rate, 112 with the angles one after
// another; 374000 ragged rows of 8 key heads of 64 and as many values: 280 us, 81 %;
// what is left are waits for loads, five CTAs a SM are better than four there.)
constexpr int eights_ctas(int items) { return items == 1 ? 5 : 5 - items; }  // an SM's: 48, 80, 128 registers

template <typename T2, int kItems, bool kPairs, Result kTo>
__global__ void __launch_bounds__(kThreads, eights_ctas(kItems)) lmc_rotate_eights_kernel(const __grid_constant__ RotatePlan P) {
    extern __shared__ __align__(16) float2 cs[];  // [rows][half], the steps [half], the weights [head_dim]
    __shared__ uint8_t *dst[kMaxRows];
    constexpr int kBytes = codes(kTo) ? 1 : 2;
    constexpr int kSecond = kPairs ? 1 : kItems;   // items with a piece half a turned part away
    const int64_t row0 = (int64_t)blockIdx.x * P.rows_per_cta;
    const int rows = (int)min((int64_t)P.rows_per_cta, P.num_rows - row0);
    const int lane = threadIdx.x & (P.group - 1), first_unit = threadIdx.x / P.group;
    const uint32_t mine = (P.group == 32 ? ~0u : (1u << P.group) - 1) << (threadIdx.x & 31 & ~(P.group - 1));
    uint64_t *const steps = reinterpret_cast<uint64_t *>(cs + P.rows_per_cta * P.half);
    float *const weights = reinterpret_cast<float *>(steps + (P.half + 1) / 2 * 2);
    int place[kItems];
    bool there[kItems], turned[kItems], plain[kItems];
#pragma unroll
    for (int n = 0; n < kItems; n++) {
        const int i = lane + n * P.group;
        int second;
        place[n] = first_value<8>(P, i, second);
        turned[n] = i < P.turned;
        plain[n] = !turned[n] && place[n] >= P.norm_dim;
        // (not: an item that is neither normalised nor turned, where it lies already)
        there[n] = i < P.items && !(kTo == kRows && P.touch_only && plain[n]);
    }
    wait_for_launch();
    let_next_start();

    int row = first_unit / P.units, unit = first_unit - row * P.units;
    uint4 lo[kItems], hi[kSecond];
    auto load = [&] {
        const uint16_t *src = P.x + (row0 + row) * P.x_row;
        if (unit < P.heads) {
            src += unit * P.x_head;
#pragma unroll
            for (int n = 0; n < kItems; n++) {
                if (there[n]) {
                    lo[n] = __ldcs(reinterpret_cast<const uint4 *>(src + place[n]));
                    if (!kPairs && turned[n])
                        hi[kPairs ? 0 : n] = __ldcs(reinterpret_cast<const uint4 *>(src + place[n] + P.half));
                }
            }
        } else {
            const int from = (unit - P.heads) * P.rest_unit, most = min(P.rest_unit, P.rest - from) / 8;
            src += P.heads * P.head_dim + from;
#pragma unroll
            for (int n = 0; n < kItems; n++)
                if (lane + n * P.group < most)
                    lo[n] = __ldcs(reinterpret_cast<const uint4 *>(src) + lane + n * P.group);
        }
    };
#pragma unroll
    for (int n = 0; n < kItems; n++)
        lo[n] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < kSecond; n++)
        hi[n] = make_uint4(0, 0, 0, 0);
    if (row < rows)
        load();  // while the angles are made
    if (P.norm_dim > 0)
        for (int k = threadIdx.x; k < P.head_dim; k += kThreads)
            weights[(k >> 2 & 1) * (P.head_dim >> 1) + (k >> 3) * 4 + (k & 3)] =
                P.weight != nullptr && k < P.norm_dim ? __ldca(P.weight + k) : 1.0f;
    make_angles<kTo, kPairs ? kPairsOrder : kHalvesOrder>(P, cs, steps, dst, row0, rows);
    __syncthreads();

    // codes: what is not turned is brought to its scale by the norm's factor
    const float code = kTo == kCodes ? P.code_inverse : 1.0f;
    while (row < rows) {
        uint8_t *to = nullptr;
        if (kTo == kRows)
            to = reinterpret_cast<uint8_t *>(P.out + (row0 + row) * P.out_row + unit * P.out_head);
        else
            to = dst[row];
        if (unit < P.heads) {
            Two a[kItems][4], b[kSecond][4];
#pragma unroll
            for (int n = 0; n < kItems; n++)
                open<T2>(a[n], lo[n]);
            if constexpr (!kPairs) {
#pragma unroll
                for (int n = 0; n < kItems; n++)
                    open<T2>(b[n], hi[n]);
            }
            const int here = row, here_unit = unit;
            row += P.row_step;
            unit += P.unit_step;
            if (unit >= P.units) {
                unit -= P.units;
                row++;
            }
            if (row < rows)
                load();
            if (P.norm_dim > 0) {
                Two sum = two(0.0f, 0.0f);
#pragma unroll
                for (int n = 0; n < kItems; n++) {
                    if (there[n] && place[n] < P.norm_dim) {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            sum = plus_product(a[n][k], a[n][k], sum);
                    }
                    if constexpr (!kPairs) {
                        if (there[n] && turned[n] && place[n] + P.half < P.norm_dim) {
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                sum = plus_product(b[n][k], b[n][k], sum);
                        }
                    }
                }
                const float2 halves = apart(sum);
                float all = halves.x + halves.y;
                for (int o = P.group / 2; o > 0; o >>= 1)
                    all += __shfl_xor_sync(mine, all, o);
                const float norm = rsqrtf(fmaf(all, P.inverse_norm_dim, P.eps));
#pragma unroll
                for (int n = 0; n < kItems; n++) {
                    if (there[n]) {
                        weigh(a[n], weights, P.head_dim, place[n] >= P.norm_dim ? 1.0f : turned[n] ? norm : norm * code, place[n]);
                        if constexpr (!kPairs) {
                            if (turned[n])
                                weigh(b[n], weights, P.head_dim, place[n] + P.half < P.norm_dim ? norm : 1.0f, place[n] + P.half);
                        }
                    }
                }
            }
            if (to != nullptr) {
                if (kTo != kRows)
                    to += here_unit * P.head_dim * kBytes;
                const float2 *const angles = cs + here * P.half;
#pragma unroll
                for (int n = 0; n < kItems; n++) {
                    if (!there[n])
                        continue;
                    uint8_t *const at = to + place[n] * kBytes;
                    if (turned[n]) {
                        if constexpr (kPairs) {
                            turn_pairs(a[n], angles, P.half, lane + n * P.group);
                        } else {
                            turn_halves(a[n], b[n], angles, P.half, lane + n * P.group);
                            put<T2, kTo>(P, at + P.half * kBytes, b[n]);
                        }
                    }
                    put<T2, kTo>(P, at, a[n], plain[n]);
                }
            }
        } else {
            const int from = (unit - P.heads) * P.rest_unit, most = to == nullptr ? 0 : min(P.rest_unit, P.rest - from) / 8;
            to += (P.heads * P.head_dim + from) * kBytes;
            uint4 x[kItems];
#pragma unroll
            for (int n = 0; n < kItems; n++)
                x[n] = lo[n];
            row += P.row_step;
            unit += P.unit_step;
            if (unit >= P.units) {
                unit -= P.units;
                row++;
            }
            if (row < rows)
                load();
#pragma unroll
            for (int n = 0; n < kItems; n++) {
                if (lane + n * P.group < most) {
                    uint8_t *const at = to + 8 * (lane + n * P.group) * kBytes;
                    if constexpr (kTo == kCodes) {
                        const uint32_t raw[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
                        float y[8];
                        widen_values<T2, 8>(y, raw);
                        store_values<T2, 8, kTo>(P, at, y, false);
                    } else {
                        __stcs(reinterpret_cast<uint4 *>(at), x[n]);
                    }
                }
            }
        }
    }
}

// Heads of more than 32 pieces: eight lanes take one, up to kLongItems pieces each,
// which are widened twice. A latent's 72 pieces fill such a group's nine rounds (of 32
// lanes' three they would fill three quarters), four heads' sums of squares take three
// shuffles together instead of five each, and 32 heads a CTA keep many CTAs at
// different steps. (131072 fp8 entries of 576 values: 63 us; 1024 of them 6.0. With a
// warp per head and the next one's pieces asked for ahead 77 and 7.6; two heads a group
// one after another 72; CTAs that stay 84.)
constexpr int kLongItems = 9, kLongGroup = 8, kLongCtas = 4;

template <typename T2, bool kPairs, Result kTo>
__global__ void __launch_bounds__(kThreads, kLongCtas) lmc_rotate_long_kernel(const __grid_constant__ RotatePlan P) {
    extern __shared__ __align__(16) float2 cs[];  // [rows][half], the steps [half], the weights [head_dim]
    __shared__ uint8_t *dst[kMaxRows];
    constexpr int kBytes = codes(kTo) ? 1 : 2;
    const int64_t row0 = (int64_t)blockIdx.x * P.rows_per_cta;
    const int rows = (int)min((int64_t)P.rows_per_cta, P.num_rows - row0);
    const int lane = threadIdx.x & (kLongGroup - 1);
    const int row = (int)(threadIdx.x / kLongGroup) / P.units, unit = threadIdx.x / kLongGroup - row * P.units;
    uint64_t *const steps = reinterpret_cast<uint64_t *>(cs + P.rows_per_cta * P.half);
    float *const weights = reinterpret_cast<float *>(steps + (P.half + 1) / 2 * 2);
    int place[kLongItems];
#pragma unroll
    for (int n = 0; n < kLongItems; n++) {
        int second;
        place[n] = first_value<8>(P, lane + n * kLongGroup, second);
    }
    wait_for_launch();
    let_next_start();
    uint4 lo[kLongItems] = {}, hi = {};  // halves: only a lane's first piece has a second one
    if (row < rows) {                    // while the angles are made
        const uint16_t *const src = P.x + (row0 + row) * P.x_row + unit * P.x_head;
#pragma unroll
        for (int n = 0; n < kLongItems; n++)
            if (lane + n * kLongGroup < P.items)
                lo[n] = __ldcs(reinterpret_cast<const uint4 *>(src + place[n]));
        if (!kPairs && lane < P.turned)
            hi = __ldcs(reinterpret_cast<const uint4 *>(src + place[0] + P.half));
    }
    if (P.norm_dim > 0)
        for (int k = threadIdx.x; k < P.head_dim; k += kThreads)
            weights[(k >> 2 & 1) * (P.head_dim >> 1) + (k >> 3) * 4 + (k & 3)] =
                P.weight != nullptr && k < P.norm_dim ? __ldca(P.weight + k) : 1.0f;
    make_angles<kTo, kPairs ? kPairsOrder : kHalvesOrder>(P, cs, steps, dst, row0, rows);
    __syncthreads();
    if (row >= rows)
        return;
    uint8_t *to;
    if (kTo == kRows)
        to = reinterpret_cast<uint8_t *>(P.out + (row0 + row) * P.out_row + unit * P.out_head);
    else if ((to = dst[row]) != nullptr)
        to += unit * P.head_dim * kBytes;
    float norm = 1.0f;
    if (P.norm_dim > 0) {
        Two sum = two(0.0f, 0.0f);
        auto add = [&](const uint4 &raw) {
            Two x[4];
            open<T2>(x, raw);
#pragma unroll
            for (int k = 0; k < 4; k++)
                sum = plus_product(x[k], x[k], sum);
        };
#pragma unroll
        for (int n = 0; n < kLongItems; n++)
            if (lane + n * kLongGroup < P.items && place[n] < P.norm_dim)
                add(lo[n]);
        if (!kPairs && lane < P.turned && place[0] + P.half < P.norm_dim)
            add(hi);
        const float2 halves = apart(sum);
        float all = halves.x + halves.y;
#pragma unroll
        for (int o = kLongGroup / 2; o > 0; o >>= 1)
            all += __shfl_xor_sync(0xffu << (threadIdx.x & 24), all, o);
        norm = rsqrtf(fmaf(all, P.inverse_norm_dim, P.eps));
    }
    if (to == nullptr)
        return;
    const float2 *const angles = cs + row * P.half;
    // codes: what is not turned is brought to its scale by the norm's factor
    const float straight = kTo == kCodes ? norm * P.code_inverse : norm;
#pragma unroll
    for (int n = 0; n < kLongItems; n++) {
        const bool turned = lane + n * kLongGroup < P.turned, plain = !turned && place[n] >= P.norm_dim;
        if (lane + n * kLongGroup >= P.items || (kTo == kRows && P.touch_only && plain))
            continue;
        Two a[4], b[4];
        open<T2>(a, lo[n]);
        if (P.norm_dim > 0)
            weigh(a, weights, P.head_dim, place[n] >= P.norm_dim ? 1.0f : turned ? norm : straight, place[n]);
        uint8_t *const at = to + place[n] * kBytes;
        if (turned) {
            if constexpr (kPairs) {
                turn_pairs(a, angles, P.half, lane + n * kLongGroup);
            } else if (n == 0) {
                open<T2>(b, hi);
                if (P.norm_dim > 0)
                    weigh(b, weights, P.head_dim, place[n] + P.half < P.norm_dim ? norm : 1.0f, place[n] + P.half);
                turn_halves(a, b, angles, P.half, lane);
                put<T2, kTo>(P, at + P.half * kBytes, b);
            }
        }
        put<T2, kTo>(P, at, a, plain);
    }
}

// Longer heads, and rows that do not lie on multiples of 16 bytes: W values of a piece
// (8, or 1), a head's items one after another, read a second time after the norm.
template <typename T2, int W, Result kTo>
__global__ void __launch_bounds__(kThreads) lmc_rotate_kernel(const __grid_constant__ RotatePlan P) {
    extern __shared__ __align__(16) float2 cs[];  // [rows][half], then the steps [half]
    __shared__ uint8_t *dst[kMaxRows];
    constexpr int kBytes = codes(kTo) ? 1 : 2;
    const int64_t row0 = (int64_t)blockIdx.x * P.rows_per_cta;
    const int rows = (int)min((int64_t)P.rows_per_cta, P.num_rows - row0);
    wait_for_launch();
    let_next_start();
    make_angles<kTo>(P, cs, reinterpret_cast<uint64_t *>(cs + P.rows_per_cta * P.half), dst, row0, rows);
    __syncthreads();

    const int lane = threadIdx.x & (P.group - 1);
    const uint32_t mine = (P.group == 32 ? ~0u : (1u << P.group) - 1) << (threadIdx.x & 31 & ~(P.group - 1));
    const int all = rows * P.units;
    for (int u = threadIdx.x / P.group; u < all; u += kThreads / P.group) {
        const int row = u / P.units, unit = u - row * P.units;
        const bool head = unit < P.heads;
        const uint16_t *src = P.x + (row0 + row) * P.x_row;
        uint8_t *to;
        int items = P.items;
        if (head) {
            src += unit * P.x_head;
            if (kTo == kRows)
                to = reinterpret_cast<uint8_t *>(P.out + (row0 + row) * P.out_row + unit * P.out_head);
            else
                to = dst[row] + (int64_t)unit * P.head_dim * kBytes;
        } else {
            const int from = (unit - P.heads) * P.rest_unit;
            src += P.heads * P.head_dim + from;
            to = dst[row] + (int64_t)(P.heads * P.head_dim + from) * kBytes;
            items = min(P.rest_unit, P.rest - from) / W;
        }
        if (kTo != kRows && dst[row] == nullptr)
            continue;
        float sum = 0.0f, norm = 1.0f;
        if (P.norm_dim > 0 && head) {  // (a group's lanes are at one unit)
            for (int i = lane; i * W < P.norm_dim; i += P.group) {
                uint32_t raw[(W + 1) / 2];
                load_values<W>(raw, src + i * W);
                float x[W];
                widen_values<T2, W>(x, raw);
#pragma unroll
                for (int k = 0; k < W; k++)
                    sum = fmaf(x[k], x[k], sum);
            }
            for (int o = P.group / 2; o > 0; o >>= 1)
                sum += __shfl_xor_sync(mine, sum, o);
            norm = rsqrtf(fmaf(sum, P.inverse_norm_dim, P.eps));
        }
        for (int i = lane; i < items; i += P.group) {
            int second = -1;
            const int first = head ? first_value<W>(P, i, second) : i * W;
            // an item that is neither normalised nor turned, where it lies already
            if (kTo == kRows && P.touch_only && i >= P.turned && first >= P.norm_dim)
                continue;
            uint32_t lo[(W + 1) / 2], hi[(W + 1) / 2] = {};
            load_values<W>(lo, src + first);
            if (second >= 0)
                load_values<W>(hi, src + second);
            finish<T2, W, kTo>(P, cs + row * P.half, to, i, first, second, norm, head, lo, hi);
        }
    }
}

// ---- host ------------------------------------------------------------------------

// The rules on the norm and the rotation that do not depend on the rows.
int check_rotation(const lmc_rotation *r) {
    if (r == nullptr || r->num_heads <= 0 || r->head_dim <= 0 || r->head_dim > kMaxHeadDim || r->norm_dim < 0 ||
        r->norm_dim > r->head_dim || r->rot_first < 0 || r->rot_dim < 0 || r->rot_dim % 2 != 0 ||
        r->rot_first > r->head_dim || r->rot_dim > r->head_dim - r->rot_first ||
        (r->rot_mode != LMC_ROT_HALVES && r->rot_mode != LMC_ROT_PAIRS) || !std::isfinite(r->eps) || r->eps < 0.0f ||
        !std::isfinite(r->mscale) || (r->rot_dim > 0 && r->frequencies == nullptr))
        return LMC_ERR_INVALID_ARG;
    if ((((uintptr_t)r->norm_weight | (uintptr_t)r->frequencies | (uintptr_t)r->positions) & 3) != 0)
        return LMC_ERR_ALIGN;
    return LMC_OK;
}

// Fills in what follows from the rotation, and how a head is shared out over lanes.
void plan_heads(RotatePlan &P, const lmc_rotation *r, int width) {
    P.weight = r->norm_weight;
    P.frequencies = r->frequencies;
    P.heads = r->num_heads;
    P.head_dim = r->head_dim;
    P.norm_dim = r->norm_dim;
    P.rot_first = r->rot_first;
    P.half = r->rot_dim / 2;
    P.pairs = r->rot_mode == LMC_ROT_PAIRS;
    P.eps = r->eps;
    P.mscale = r->mscale;
    P.inverse_norm_dim = r->norm_dim > 0 ? 1.0f / (float)r->norm_dim : 0.0f;
    P.turned = width == 1 ? P.half : P.pairs ? r->rot_dim / width : P.half / width;
    P.items = P.turned + (P.head_dim - r->rot_dim) / width;
    if (P.touch_only && P.norm_dim == 0)
        P.items = P.turned;
    P.group = 4;
    while (P.group < 32 && P.group < P.items)
        P.group *= 2;
    P.rest_unit = std::max(1, P.items) * width;
    P.units = P.heads + (P.rest + P.rest_unit - 1) / P.rest_unit;
}

template <typename T2, Result kTo>
int launch(RotatePlan &P, int width, cudaStream_t stream) {
    const bool eight_lanes = kTo != kDivided && width == 8 && P.items > 32 && P.items <= kLongItems * kLongGroup && P.rest == 0 &&
                             (P.pairs || P.turned <= kLongGroup) && P.units <= kThreads / kLongGroup;
    if (eight_lanes)
        P.group = kLongGroup;
    // Rows of a CTA: enough heads for every group of lanes a few times, so that
    // the angles are made while other CTAs' loads run.
    const int at_once = kThreads / P.group;
    // (more of them where there are enough CTAs: what a lane finds out once is
    // spread over more heads)
    int64_t rows = std::max<int64_t>(1, (int64_t)at_once * 4 / P.units);
    while (P.num_rows / rows > kManyCtas && rows * P.units < (int64_t)at_once * 16)
        rows *= 2;
    if (eight_lanes)  // a head per group and turn
        rows = std::max(1, at_once / P.units);
    rows = std::min<int64_t>({rows, kMaxRows, std::max(1, kMaxAngles / std::max(1, P.half))});
    P.rows_per_cta = (int32_t)rows;
    int64_t grid = (P.num_rows + rows - 1) / rows;
    if (grid > INT32_MAX)
        return kTo == kRows ? LMC_ERR_OVERFLOW : LMC_ERR_INVALID_ARG;  // (lmc_append's own)
    P.angle_rows = P.half > 0 ? kThreads / P.half : 0;
    P.angle_step = P.half > 0 ? kThreads % P.half : 0;
    P.row_step = at_once / P.units;
    P.unit_step = at_once % P.units;
    const int per_lane = (P.items + P.group - 1) / P.group;
    void (*kern)(RotatePlan) = nullptr;
    const bool in_registers = kTo != kDivided && width == 8 && (eight_lanes || per_lane <= 3);
    if constexpr (kTo != kDivided) {
        if (eight_lanes)
            kern = P.pairs ? lmc_rotate_long_kernel<T2, true, kTo> : lmc_rotate_long_kernel<T2, false, kTo>;
        else if (!in_registers)
            ;
        else if (P.pairs)
            kern = per_lane == 3   ? lmc_rotate_eights_kernel<T2, 3, true, kTo>
                   : per_lane == 2 ? lmc_rotate_eights_kernel<T2, 2, true, kTo>
                                   : lmc_rotate_eights_kernel<T2, 1, true, kTo>;
        else
            kern = per_lane == 3   ? lmc_rotate_eights_kernel<T2, 3, false, kTo>
                   : per_lane == 2 ? lmc_rotate_eights_kernel<T2, 2, false, kTo>
                                   : lmc_rotate_eights_kernel<T2, 1, false, kTo>;
    }
    if (!in_registers)
        kern = width == 8 ? lmc_rotate_kernel<T2, 8, kTo> : lmc_rotate_kernel<T2, 1, kTo>;
    const size_t smem = (size_t)rows * P.half * sizeof(float2) + (size_t)(P.half + 1) / 2 * 2 * sizeof(uint64_t) +
                        (in_registers && P.norm_dim > 0 ? (size_t)P.head_dim * sizeof(float) : 0);
    return follow(kern, dim3((unsigned)grid), kThreads, smem, stream, P) ? LMC_OK : LMC_ERR_CUDA;
}

// Whether 1 / scale fits into the factors that values are multiplied by anyway, mscale
// and the norm's (at most 2^75, of a sum of squares that is not 0): an infinite factor
// would make NaN of zeros.
bool inverse_fits(const lmc_rotation *r, float inverse) {
    const double norm = r->norm_dim > 0 ? std::min(1.0 / std::sqrt((double)r->eps), 0x1p75) : 0.0;
    return inverse != 0.0f && (double)inverse * std::max(norm, std::fabs((double)r->mscale)) <= 0x1p127;
}

// Whether every piece of eight values lies on a multiple of its size.
bool eights(const lmc_rotation *r, std::initializer_list<int64_t> bytes16) {
    int64_t all = (int64_t)(uintptr_t)r->norm_weight;
    for (int64_t b : bytes16)
        all |= b;
    return (all & 15) == 0 && r->head_dim % 8 == 0 && r->norm_dim % 8 == 0 && r->rot_first % 8 == 0 &&
           r->rot_dim % (r->rot_mode == LMC_ROT_PAIRS ? 8 : 16) == 0;
}

// Elements [0, end) that heads of rows take up; false where heads overlap or the
// extent does not fit.
bool heads_extent(int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t dim, int64_t *end) {
    if ((rows > 1 && row < dim) || (heads > 1 && head < dim) || row < 0 || head < 0)
        return false;
    int64_t by_rows = 0, by_heads = 0;
    if ((rows > 1 && !mul_ok(row, rows - 1, &by_rows)) || (heads > 1 && !mul_ok(head, heads - 1, &by_heads)) ||
        !add_ok(by_rows, by_heads, end) || !add_ok(*end, dim, end) || *end > INT64_MAX / 4)
        return false;
    return rows <= 1 || heads <= 1 || row >= by_heads + dim || head >= by_rows + dim;
}

}  // namespace

extern "C" int lmc_rotate(const lmc_rotation *r, int32_t dtype, const void *x, int64_t x_row_stride,
                          int64_t x_head_stride, void *out, int64_t out_row_stride, int64_t out_head_stride,
                          int64_t num_rows, void *stream) {
    if (const int rc = check_rotation(r); rc != LMC_OK)
        return rc;
    int64_t x_end, out_end;
    if ((dtype != LMC_E_BF16 && dtype != LMC_E_F16) || num_rows < 0 ||
        !heads_extent(num_rows, x_row_stride, r->num_heads, x_head_stride, r->head_dim, &x_end) ||
        !heads_extent(num_rows, out_row_stride, r->num_heads, out_head_stride, r->head_dim, &out_end) ||
        (num_rows > 0 && (x == nullptr || out == nullptr || (r->rot_dim > 0 && r->positions == nullptr))))
        return LMC_ERR_INVALID_ARG;
    if ((((uintptr_t)x | (uintptr_t)out) & 1) != 0)
        return LMC_ERR_ALIGN;
    if (num_rows == 0)
        return LMC_OK;
    const bool same = x == out && (num_rows == 1 || x_row_stride == out_row_stride) &&
                      (r->num_heads == 1 || x_head_stride == out_head_stride);
    const uint64_t xa = (uint64_t)(uintptr_t)x, oa = (uint64_t)(uintptr_t)out;
    if (!same && std::max(xa, oa) < std::min(xa + 2 * (uint64_t)x_end, oa + 2 * (uint64_t)out_end))
        return LMC_ERR_OVERLAP;
    RotatePlan P = {};
    P.x = static_cast<const uint16_t *>(x);
    P.x_row = x_row_stride;
    P.x_head = x_head_stride;
    P.out = static_cast<uint16_t *>(out);
    P.out_row = out_row_stride;
    P.out_head = out_head_stride;
    P.angles = r->positions;
    P.num_rows = num_rows;
    P.touch_only = same;
    const int width = eights(r, {(int64_t)xa, (int64_t)oa, num_rows > 1 ? 2 * x_row_stride : 0,
                                 r->num_heads > 1 ? 2 * x_head_stride : 0, num_rows > 1 ? 2 * out_row_stride : 0,
                                 r->num_heads > 1 ? 2 * out_head_stride : 0})
                          ? 8
                          : 1;
    plan_heads(P, r, width);
    if (P.items == 0)
        return LMC_OK;  // in place, neither normalised nor turned
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == LMC_E_BF16 ? launch<__nv_bfloat162, kRows>(P, width, s) : launch<__half2, kRows>(P, width, s);
}

extern "C" int lmc_append_rotated(const lmc_layout *L, const lmc_entries *e, const lmc_rotation *r, void *pool,
                                  const int32_t *requests, const int32_t *positions, const void *rows,
                                  int32_t rows_dtype, int64_t row_stride, int64_t num_rows, uint32_t *status,
                                  void *stream) {
    if (const int rc = check_entries(L, e); rc != LMC_OK)
        return rc;
    if (const int rc = check_rotation(r); rc != LMC_OK)
        return rc;
    if (status == nullptr || num_rows < 0 || (rows_dtype != LMC_E_BF16 && rows_dtype != LMC_E_F16) ||
        (e->dtype != LMC_E_E4M3 && e->dtype != rows_dtype) || row_stride < e->entry_dim ||
        row_stride > INT64_MAX / 4 || (int64_t)r->num_heads * r->head_dim > e->entry_dim)
        return LMC_ERR_INVALID_ARG;
    if (num_rows > 0 && (pool == nullptr || requests == nullptr || positions == nullptr || rows == nullptr))
        return LMC_ERR_INVALID_ARG;
    if ((((uintptr_t)status | (uintptr_t)requests | (uintptr_t)positions) & 3) != 0 || ((uintptr_t)rows & 1) != 0)
        return LMC_ERR_ALIGN;
    if (num_rows == 0)
        return LMC_OK;
    const lmc_layer_desc &d = L->desc[e->layer];
    RotatePlan P = {};
    P.x = static_cast<const uint16_t *>(rows);
    P.x_row = row_stride;
    P.x_head = r->head_dim;
    P.angles = r->positions != nullptr ? r->positions : positions;
    P.pages = Pages{d.base, d.stride, L->num_blocks, (int32_t)L->block_size, (int32_t)L->specs[e->layer].token_bytes};
    P.table = token_table(e->table);
    P.requests = requests;
    P.positions = positions;
    P.pool = static_cast<uint8_t *>(pool);
    P.status = status;
    P.num_requests = e->num_requests;
    P.code_scale = e->scale;
    P.code_inverse = inverse_scale(e->scale);
    P.num_rows = num_rows;
    P.rest = e->entry_dim - r->num_heads * r->head_dim;
    const int64_t page = (int64_t)(uintptr_t)pool | d.base | d.stride | P.pages.token_bytes;
    const int width = P.rest % 8 == 0 &&
                              eights(r, {(int64_t)(uintptr_t)rows, 2 * row_stride, e->dtype == LMC_E_E4M3 ? 2 * page : page})
                          ? 8
                          : 1;
    plan_heads(P, r, width);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = rows_dtype == LMC_E_BF16;
    if (e->dtype == LMC_E_E4M3 && !inverse_fits(r, P.code_inverse))
        return bf16 ? launch<__nv_bfloat162, kDivided>(P, width, s) : launch<__half2, kDivided>(P, width, s);
    if (e->dtype == LMC_E_E4M3)
        return bf16 ? launch<__nv_bfloat162, kCodes>(P, width, s) : launch<__half2, kCodes>(P, width, s);
    return bf16 ? launch<__nv_bfloat162, kEntries>(P, width, s) : launch<__half2, kEntries>(P, width, s);
}
