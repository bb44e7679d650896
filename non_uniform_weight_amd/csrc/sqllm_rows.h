// sqllm_rows.h -- what is done with rows of fp16 values on their way into a
// product: the pieces of a row, its sum and largest, and the rounding to 8-bit
// integers; and the quantiser's launch (sqllm_norm.hip), for the calls that
// round their activations inside.
#ifndef SQLLM_ROWS_H
#define SQLLM_ROWS_H

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sqllm_device.h"

namespace sqllm {

// Arguments as checked by sqllm_int8_quantize.
hipError_t launch_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, float *scale,
                                hipStream_t stream);

namespace rows {

using dev::u32x2;
using dev::u32x4;
// fp16 rows begin at any even address: one 16-byte access all the same (global
// memory takes unaligned ones).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

// Eight values of a row from column c on, zeros past its end.
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int c, int cols)
{
    if (c + 8 <= cols) return *(const u32x4_any *)(row + c);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = c + k < cols ? row[c + k] : 0;
    return u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

__device__ __forceinline__ void floats(u32x4 v, float (&y)[8])
{
    const half8_t h = __builtin_bit_cast(half8_t, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (float)h[k];
}

// The largest of sixteen lanes' v, and of a wave's.  In all lanes.
#define SQLLM_ROR(v, n) __builtin_amdgcn_update_dpp(0, (int)(v), 0x120 + n, 0xF, 0xF, true)
__device__ __forceinline__ uint32_t max_of_16(uint32_t v)
{
    v = max(v, (uint32_t)SQLLM_ROR(v, 8));
    v = max(v, (uint32_t)SQLLM_ROR(v, 4));
    v = max(v, (uint32_t)SQLLM_ROR(v, 2));
    return max(v, (uint32_t)SQLLM_ROR(v, 1));
}
#undef SQLLM_ROR

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max_of_16(v);
    return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
               max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// Magnitudes are compared as integers: an infinity or a NaN is the largest.
__device__ __forceinline__ uint32_t magnitude(const float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(y[k]) & 0x7FFFFFFFu);
    return m;
}

constexpr uint32_t kInf = 0x7F800000u;

// The scale of a row whose largest magnitude has these bits.
__device__ __forceinline__ float scale_of(uint32_t top) { return top >= kInf ? NAN : __uint_as_float(top) / 127.f; }

// 127 / m in two parts, so that y * 127 / m is right to a rounding of its own:
// fp16 values lie exactly half way between two integers now and then (m = 381,
// y = 1.5), and with the first part alone some of them land on either side.
struct Inverse {
    float high, low;
};

__device__ __forceinline__ Inverse inverse_of(uint32_t top)
{
    if (top == 0 || top >= kInf) return {0.f, 0.f};
    const float m = __uint_as_float(top);
    const float high = 127.f / m;
    return {high, __builtin_fmaf(-high, m, 127.f) * (high * (1.f / 127.f))};
}

// Eight integers nearest to t, ties to even: added to 1.5 * 2^23, the sum's low
// byte is the integer.
__device__ __forceinline__ u32x2 bytes_of(const float (&t)[8])
{
    uint32_t b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = __float_as_uint(t[k] + 12582912.f);
    auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u),
                                     0x05040100u);
    };
    return u32x2{four(b[0], b[1], b[2], b[3]), four(b[4], b[5], b[6], b[7])};
}

// The same of fp16 values y * inverse: one that is not half way is further from
// it than the rounding here moves it (mantissas of 11 bits).
__device__ __forceinline__ u32x2 integers(const float (&y)[8], Inverse inverse)
{
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = __builtin_fmaf(y[k], inverse.high, y[k] * inverse.low);
    return bytes_of(t);
}

} // namespace rows
} // namespace sqllm

#endif
