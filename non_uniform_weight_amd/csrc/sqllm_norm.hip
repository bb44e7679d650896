// sqllm_norm.hip -- the norm of include/sqllm_norm.h and the quantiser of
// include/sqllm_int8.h: one pass over a row each, so one set of kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sqllm_device.h"
#include "sqllm_fp8.h"
#include "sqllm_int8.h"
#include "sqllm_norm.h"
#include "sqllm_rows.h"

namespace {

using sqllm::dev::u32x2;
using sqllm::dev::u32x4;
using namespace sqllm::rows;
typedef short short2_t __attribute__((ext_vector_type(2)));

// What is done with a row.
enum Form { kNormHalf, kNormInt8, kNormFp8, kQuantize };

struct Rows {
    const uint16_t *x, *residual, *weight;
    uint16_t *sum;
    void *out;   // fp16, int8 or e4m3
    void *scale; // fp32 a row, or bytes: `words` words a row
    int64_t ldx, ldr, ldo;
    int rows, cols;
    int span;    // columns written: `cols` padded as the output form has it
    int words;
    float eps;
    double per_col; // 1 / cols
};

__device__ __forceinline__ void store8(uint16_t *row, int c, int cols, u32x4 v)
{
    if (c + 8 <= cols) {
        *(u32x4_any *)(row + c) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < cols) row[c + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

// The sum of the sixteen lanes' v and then of the wave's four sixteens, in a
// fixed order.  In all lanes.
__device__ __forceinline__ double wave_sum(double v)
{
    auto add = [&](auto turned) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        v += __builtin_bit_cast(double, (uint64_t)(uint32_t)turned((uint32_t)b) | (uint64_t)(uint32_t)turned((uint32_t)(b >> 32)) << 32);
    };
#define SQLLM_TURN(n) add([](uint32_t w) { return __builtin_amdgcn_update_dpp(0, (int)w, 0x120 + n, 0xF, 0xF, true); })
    SQLLM_TURN(8);
    SQLLM_TURN(4);
    SQLLM_TURN(2);
    SQLLM_TURN(1);
#undef SQLLM_TURN
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    auto of = [&](int lane) {
        return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)b, lane) |
                                              (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32);
    };
    return (of(0) + of(16)) + (of(32) + of(48));
}

// The same over a row's threads.  ONE: they are a wave; else the workgroup, of
// up to sixteen, and `red` is sixteen words of LDS of its own.
template <bool ONE>
__device__ __forceinline__ double row_sum(double v, double *red)
{
    v = wave_sum(v);
    if constexpr (!ONE) {
        red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.;
        for (uint32_t k = 0; k < blockDim.x >> 6; ++k) v += red[k];
    }
    return v;
}

template <bool ONE>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *red)
{
    v = wave_max(v);
    if constexpr (!ONE) {
        red[threadIdx.x >> 6] = v;
        __syncthreads();
        for (uint32_t k = 0; k < blockDim.x >> 6; ++k) v = max(v, red[k]);
    }
    return v;
}

__device__ __forceinline__ u32x4 add8(u32x4 a, u32x4 b)
{
    return __builtin_bit_cast(u32x4, (half8_t)(__builtin_bit_cast(half8_t, a) + __builtin_bit_cast(half8_t, b)));
}

// The sum of eight squares in fp32; sums of these are in fp64, so that a row's
// sum is off by 2^-24 over the root of its pieces' number.
__device__ __forceinline__ float squares(u32x4 v)
{
    const half8_t h = __builtin_bit_cast(half8_t, v);
    float s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = (float)h[2 * k], b = (float)h[2 * k + 1];
        s[k] = __builtin_fmaf(a, a, b * b);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// 1 / sqrt(m) in two parts: the reciprocal root r and what one step of
// Newton's method adds to it, r (1 - m r^2) / 2, so that y has no rounding but
// that of its last addition.  (With r alone three times as many of the 8-bit
// codes land on the other side of a border between two.)
struct Root {
    float high, low;
};

__device__ __forceinline__ Root reciprocal_root(double m)
{
    const float f = (float)m, r = rsqrtf(f);
    // not for 0 or infinity, where r says all
    return {r, f > 0.f && f < INFINITY ? 0.5f * r * (float)__builtin_fma(-m * r, (double)r, 1.) : 0.f};
}

// y of eight values: sum * weight is exact in fp32 (two fp16 values).
__device__ __forceinline__ void normalized(u32x4 v, u32x4 w, Root root, float (&y)[8])
{
    const half8_t a = __builtin_bit_cast(half8_t, v), b = __builtin_bit_cast(half8_t, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float p = (float)a[k] * (float)b[k];
        y[k] = __builtin_fmaf(p, root.high, p * root.low);
    }
}

// The int8 form needs no root for its integers: they are nearest to 127 p / the
// largest |p| of the row, p = sum * weight, exact.
__device__ __forceinline__ void products(u32x4 v, u32x4 w, float (&p)[8])
{
    const half8_t a = __builtin_bit_cast(half8_t, v), b = __builtin_bit_cast(half8_t, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = (float)a[k] * (float)b[k];
}

// The integers of p, m its row's largest.  A quotient that has been rounded to
// half way between two goes to its own side: one bit on.
__device__ __forceinline__ u32x2 integers_of(const float (&p)[8], float m, Inverse inverse)
{
    float t[8], off = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        t[k] = __builtin_fmaf(p[k], inverse.high, p[k] * inverse.low);
        off = fmaxf(off, fabsf(t[k] - rintf(t[k])));
    }
    if (off == 0.5f) { // (one wave in two hundred)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double rest = 127. * p[k] - (double)t[k] * m; // exact
            if (fabsf(t[k] - rintf(t[k])) == 0.5f && rest != 0.)
                t[k] = __uint_as_float(__float_as_uint(t[k]) + ((rest > 0.) == (t[k] > 0.f) ? 1 : -1));
        }
    }
    return bytes_of(t);
}

// Before y is rounded again, to e4m3: where it lies on a border between two codes
// (all of those have sixteen low bits of zero) and the exact product does not,
// one bit towards that, or the tie would go to the even code.
__device__ __forceinline__ void off_the_border(u32x4 v, u32x4 w, Root root, float (&y)[8])
{
    uint32_t low = 0xFFFF;
#pragma unroll
    for (int k = 0; k < 8; ++k) low = min(low, __float_as_uint(y[k]) & 0xFFFF);
    if (low) return; // (one wave in a hundred goes on)
    const half8_t a = __builtin_bit_cast(half8_t, v), b = __builtin_bit_cast(half8_t, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float p = (float)a[k] * (float)b[k], rest = __builtin_fmaf(p, root.high, -y[k]) + p * root.low;
        if (rest != 0.f && !(__float_as_uint(y[k]) & 0xFFFF) && fabsf(y[k]) < INFINITY && y[k] != 0.f)
            y[k] = __uint_as_float(__float_as_uint(y[k]) + ((rest > 0.f) == (y[k] > 0.f) ? 1 : -1));
    }
}

// The e4m3 form: a block's exponent from its largest finite magnitude m * 2^p
// (1 <= m < 2): 448 = 1.75 * 2^8, so s = p - 8, one more if m > 1.75.  Shifted
// up by one and raised by 2^24, infinities and NaN wrap to the bottom.
__device__ __forceinline__ uint32_t finite_magnitude(const float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, (__float_as_uint(y[k]) << 1) + 0x01000000u);
    return m;
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t m)
{
    const uint32_t b = m > 0x01000000u ? (m - 0x01000000u) >> 1 : 0;
    if (b == 0) return 127;
    const int s = (int)(b >> 23) - 8 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
    return (uint32_t)max(s, 1); // (below 2^-117: zeros)
}

__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d, float scale)
{
    short2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ void store_half(const Rows &a, int64_t row, int c, const float (&y)[8])
{
    half8_t h;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = (_Float16)y[k];
    store8((uint16_t *)a.out + row * a.ldo, c, a.cols, __builtin_bit_cast(u32x4, h));
}

// The block of these sixteen lanes, and the word of scales of the wave's four.
__device__ __forceinline__ void store_fp8(const Rows &a, int64_t row, int c, const float (&y)[8])
{
    const uint32_t sb = scale_byte(max_of_16(finite_magnitude(y)));
    const float f = __uint_as_float(sb << 23);
    const u32x2 q = {to_e4m3(y[0], y[1], y[2], y[3], f), to_e4m3(y[4], y[5], y[6], y[7], f)};
    if (c < a.ldo) *(u32x2 *)((uint8_t *)a.out + row * a.ldo + c) = q;
    const int s = (int)sb;
    const uint32_t word = (uint32_t)(__builtin_amdgcn_readlane(s, 0) | __builtin_amdgcn_readlane(s, 16) << 8 |
                                     __builtin_amdgcn_readlane(s, 32) << 16) |
                          (uint32_t)__builtin_amdgcn_readlane(s, 48) << 24;
    if ((threadIdx.x & 63) == 0 && c < a.span) ((uint32_t *)a.scale)[row * a.words + (c >> 9)] = word;
}

// What the integers of a row are made with, top: the bits of its largest
// magnitude (of y, or of p with the root that makes y of it).
template <int FORM>
__device__ __forceinline__ Inverse store_scale(const Rows &a, int64_t row, uint32_t top, Root root, bool first)
{
    if (first) {
        const float m = __uint_as_float(top);
        const uint32_t y = FORM == kQuantize ? top : __float_as_uint(fabsf(__builtin_fmaf(m, root.high, m * root.low)));
        ((float *)a.scale)[row] = scale_of(max(top >= kInf ? top : 0, y));
    }
    return inverse_of(top);
}

template <int FORM>
__device__ __forceinline__ void store_integers(const Rows &a, int64_t row, int c, const float (&y)[8], uint32_t top, Inverse inverse)
{
    u32x2 q = {0, 0};
    if (top < kInf) q = FORM == kQuantize ? integers(y, inverse) : integers_of(y, __uint_as_float(top), inverse);
    *(u32x2 *)((int8_t *)a.out + row * a.ldo + c) = q;
}

// A row in the registers of a wave (ONE; four rows a workgroup, no barrier) or
// of a workgroup, V pieces of eight values a thread: read once, written once.
template <int FORM, bool RES, bool ONE, int V>
__global__ void __launch_bounds__(ONE ? 256 : 1024) rows_kernel(Rows a)
{
    __shared__ double sums[16];
    __shared__ uint32_t red[16];
    const int T = ONE ? 64 : blockDim.x, t = ONE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = ONE ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : blockIdx.x;
    if (ONE && row >= a.rows) return;
    const uint16_t *const x = a.x + row * a.ldx;
    u32x4 v[V], r[RES ? V : 1], w[FORM == kQuantize ? 1 : V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = (k * T + t) * 8;
        v[k] = u32x4{0, 0, 0, 0};
        if constexpr (RES) r[k] = v[k];
        if constexpr (FORM != kQuantize) w[k] = v[k];
        if (c < a.cols) {
            v[k] = load8(x, c, a.cols);
            if constexpr (RES) r[k] = load8(a.residual + row * a.ldr, c, a.cols);
            if constexpr (FORM != kQuantize) w[k] = load8(a.weight, c, a.cols);
        }
    }
    if constexpr (RES)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = add8(v[k], r[k]);
    float y[V][8];
    Root root = {};
    if constexpr (FORM != kQuantize) {
        double s = 0.;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (k * T + t) * 8;
            if (RES && a.sum && c < a.cols) store8(a.sum + row * a.cols, c, a.cols, v[k]);
            s += squares(v[k]);
        }
        root = reciprocal_root(row_sum<ONE>(s, sums) * a.per_col + a.eps);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (FORM == kNormInt8) {
                products(v[k], w[k], y[k]);
                continue;
            }
            normalized(v[k], w[k], root, y[k]);
            if constexpr (FORM == kNormFp8) off_the_border(v[k], w[k], root, y[k]);
            // (a root of infinity or NaN turns the zeros past the end into NaN)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((k * T + t) * 8 + j >= a.cols) y[k][j] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            floats(v[k], y[k]);
        }
    }
    if constexpr (FORM == kNormHalf) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (k * T + t) * 8;
            if (c < a.cols) store_half(a, row, c, y[k]);
        }
    } else if constexpr (FORM == kNormFp8) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k * T * 8 < a.span) store_fp8(a, row, (k * T + t) * 8, y[k]); // (whole waves)
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) top = max(top, magnitude(y[k]));
        top = row_max<ONE>(top, red);
        const Inverse inverse = store_scale<FORM>(a, row, top, root, t == 0);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (k * T + t) * 8;
            if (c < a.span) store_integers<FORM>(a, row, c, y[k], top, inverse);
        }
    }
}

// Longer rows: each pass reads the row again, sums of two from `sum` where they
// were kept (it may be x or the residual).
template <int FORM, bool RES>
__global__ void __launch_bounds__(1024) long_rows_kernel(Rows a)
{
    __shared__ double sums[16];
    __shared__ uint32_t red[16];
    const int64_t row = blockIdx.x;
    const uint16_t *const x = a.x + row * a.ldx;
    Root root = {};
    if constexpr (FORM != kQuantize) {
        double s = 0.;
        for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
            u32x4 v = load8(x, c, a.cols);
            if constexpr (RES) {
                v = add8(v, load8(a.residual + row * a.ldr, c, a.cols));
                if (a.sum) store8(a.sum + row * a.cols, c, a.cols, v);
            }
            s += squares(v);
        }
        root = reciprocal_root(row_sum<false>(s, sums) * a.per_col + a.eps);
    }
    auto value = [&](int c, float (&y)[8]) {
        u32x4 v = u32x4{0, 0, 0, 0};
        if (c < a.cols) {
            if (RES && a.sum) {
                v = load8(a.sum + row * a.cols, c, a.cols);
            } else {
                v = load8(x, c, a.cols);
                if constexpr (RES) v = add8(v, load8(a.residual + row * a.ldr, c, a.cols));
            }
        }
        if constexpr (FORM == kQuantize) {
            floats(v, y);
        } else {
            const u32x4 w = c < a.cols ? load8(a.weight, c, a.cols) : u32x4{0, 0, 0, 0};
            if constexpr (FORM == kNormInt8) return products(v, w, y);
            normalized(v, w, root, y);
            if constexpr (FORM == kNormFp8) off_the_border(v, w, root, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j >= a.cols) y[j] = 0.f;
        }
    };
    float y[8];
    if constexpr (FORM == kNormHalf) {
        for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
            value(c, y);
            store_half(a, row, c, y);
        }
    } else if constexpr (FORM == kNormFp8) {
        for (int c0 = 0; c0 < a.span; c0 += 8192) { // (whole waves)
            value(c0 + threadIdx.x * 8, y);
            store_fp8(a, row, c0 + threadIdx.x * 8, y);
        }
    } else {
        uint32_t top = 0;
        for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
            value(c, y);
            top = max(top, magnitude(y));
        }
        top = row_max<false>(top, red);
        const Inverse inverse = store_scale<FORM>(a, row, top, root, threadIdx.x == 0);
        for (int c = threadIdx.x * 8; c < a.span; c += 8192) {
            value(c, y);
            store_integers<FORM>(a, row, c, y, top, inverse);
        }
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

// Threads of a row: as many as leave one piece each up to 512, two up to 1024
// threads, more beyond; shorter rows are a wave's.  us at one, two, three and
// four pieces a thread (with the residual, fp16 out): 1x4096 2.6, 2.9, 3.5, 4.0;
// 16x8192 3.3, 3.2, 3.9, 4.5; 4096x4096 23.2, 23.1, 25.2, 26.2; 4096x8192 44, 42,
// 45, 47 (6.4 TB/s); 1000x24576 at three 39, at four 41 (without a residual 20.4
// and 26).  The quantiser holds less, and where rows are many has room for four:
// 4096x4096 at two and four 11.0 and 10.4, 1024x16384 11.5 and 10.3, 4096x8192
// 18.1 and 17.8 (5.7 TB/s), but 300x5120 3.6 and 3.8, 4096x1024 4.5 at one, 5.3.
template <int FORM, bool RES>
hipError_t launch_rows(const Rows &a, hipStream_t stream)
{
    const int pieces = (a.span + 7) / 8;
    auto launch = [&](auto kern, int v) {
        hipLaunchKernelGGL(kern, dim3(a.rows), dim3((pieces + 64 * v - 1) / (64 * v) * 64), 0, stream, a);
    };
    if (pieces <= 64)
        hipLaunchKernelGGL((rows_kernel<FORM, RES, true, 1>), dim3((a.rows + 3) / 4), dim3(256), 0, stream, a);
    else if (pieces <= 128)
        hipLaunchKernelGGL((rows_kernel<FORM, RES, true, 2>), dim3((a.rows + 3) / 4), dim3(256), 0, stream, a);
    else if (FORM == kQuantize && a.rows >= 1000 && pieces > 256 && pieces <= 4096)
        launch(rows_kernel<FORM, RES, false, 4>, 4);
    else if (pieces <= 512)
        launch(rows_kernel<FORM, RES, false, 1>, 1);
    else if (pieces <= 2 * 1024)
        launch(rows_kernel<FORM, RES, false, 2>, 2);
    else if (pieces <= 3 * 1024)
        launch(rows_kernel<FORM, RES, false, 3>, 3);
    else if (pieces <= 4 * 1024)
        launch(rows_kernel<FORM, RES, false, 4>, 4);
    else
        hipLaunchKernelGGL((long_rows_kernel<FORM, RES>), dim3(a.rows), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A launch takes up to 2^32 - 1 work-items: rows go in pieces of whole rows.
constexpr int64_t kMaxRows = (int64_t)1 << 30, kPiece = (int64_t)1 << 21;

template <int FORM>
hipError_t launch_pieces(Rows a, int64_t rows, hipStream_t stream)
{
    const int width = FORM == kNormHalf ? 2 : 1;
    for (int64_t done = 0; done < rows; done += kPiece) {
        a.rows = (int)(rows - done < kPiece ? rows - done : kPiece);
        const hipError_t e = a.residual ? launch_rows<FORM, FORM != kQuantize>(a, stream) : launch_rows<FORM, false>(a, stream);
        if (e != hipSuccess) return e;
        a.x += kPiece * a.ldx;
        if (a.residual) a.residual += kPiece * a.ldr;
        if (a.sum) a.sum += kPiece * a.cols;
        a.out = (uint8_t *)a.out + kPiece * a.ldo * width;
        if (a.scale) a.scale = (uint32_t *)a.scale + kPiece * (FORM == kNormFp8 ? a.words : 1);
    }
    return hipSuccess;
}

// What the three norms check alike; cols_limit: of the output form.
sqllm_status check_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const uint16_t *weight,
                        int64_t rows, int64_t cols, float eps, const uint16_t *sum, int64_t cols_limit)
{
    if (!x || !weight || (sum && !residual)) return SQLLM_ERR_NULL;
    if (rows < 1 || rows > kMaxRows || cols < 1 || cols > cols_limit || ldx < cols || (residual && ldr < cols))
        return SQLLM_ERR_SHAPE;
    if (!(eps >= 0.f) || eps == INFINITY) return SQLLM_ERR_SHAPE;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(sum, 2)) return SQLLM_ERR_ALIGN;
    return SQLLM_OK;
}

sqllm_status status(hipError_t e) { return e == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP; }

constexpr int64_t kMaxHalfCols = (int64_t)1 << 24, kMaxInt8Cols = 131071;

} // namespace

namespace sqllm {

hipError_t launch_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, float *scale,
                                hipStream_t stream)
{
    const int64_t ld = sqllm_int8_cols(cols);
    return launch_pieces<kQuantize>(
        Rows{x, nullptr, nullptr, nullptr, q, scale, ldx, 0, ld, 0, (int)cols, (int)ld, 0, 0.f, 0.}, rows, stream);
}

} // namespace sqllm

extern "C" int64_t sqllm_int8_cols(int64_t cols)
{
    return cols < 1 || cols > kMaxInt8Cols ? 0 : (cols + 127) / 128 * 128;
}

extern "C" sqllm_status sqllm_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, int8_t *q,
                                            float *scale, hipStream_t stream)
{
    if (!x || !q || !scale) return SQLLM_ERR_NULL;
    if (rows < 1 || rows > kMaxRows || sqllm_int8_cols(cols) == 0 || ldx < cols) return SQLLM_ERR_SHAPE;
    if (!aligned(x, 2) || !aligned(q, 16) || !aligned(scale, 4)) return SQLLM_ERR_ALIGN;
    return status(sqllm::launch_int8_quantize(x, rows, cols, ldx, q, scale, stream));
}

extern "C" sqllm_status sqllm_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                       const uint16_t *weight, int64_t rows, int64_t cols, float eps, uint16_t *sum,
                                       uint16_t *y, hipStream_t stream)
{
    if (!y) return SQLLM_ERR_NULL;
    const sqllm_status st = check_norm(x, ldx, residual, ldr, weight, rows, cols, eps, sum, kMaxHalfCols);
    if (st != SQLLM_OK) return st;
    if (!aligned(y, 2)) return SQLLM_ERR_ALIGN;
    return status(launch_pieces<kNormHalf>(
        Rows{x, residual, weight, sum, y, nullptr, ldx, ldr, cols, 0, (int)cols, (int)cols, 0, eps, 1. / cols}, rows, stream));
}

extern "C" sqllm_status sqllm_rms_norm_int8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                            const uint16_t *weight, int64_t rows, int64_t cols, float eps,
                                            uint16_t *sum, int8_t *q, float *scale, hipStream_t stream)
{
    if (!q || !scale) return SQLLM_ERR_NULL;
    const sqllm_status st = check_norm(x, ldx, residual, ldr, weight, rows, cols, eps, sum, kMaxInt8Cols);
    if (st != SQLLM_OK) return st;
    if (!aligned(q, 16) || !aligned(scale, 4)) return SQLLM_ERR_ALIGN;
    const int64_t ld = sqllm_int8_cols(cols);
    return status(launch_pieces<kNormInt8>(
        Rows{x, residual, weight, sum, q, scale, ldx, ldr, ld, 0, (int)cols, (int)ld, 0, eps, 1. / cols}, rows, stream));
}

extern "C" sqllm_status sqllm_rms_norm_fp8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                           const uint16_t *weight, int64_t rows, int64_t cols, float eps,
                                           uint16_t *sum, uint8_t *q, uint8_t *scale, hipStream_t stream)
{
    if (!q || !scale) return SQLLM_ERR_NULL;
    const sqllm_status st = check_norm(x, ldx, residual, ldr, weight, rows, cols, eps, sum, kMaxHalfCols);
    if (st != SQLLM_OK) return st;
    const int64_t pitch = sqllm_fp8_scale_pitch(cols);
    if (rows * pitch > ((int64_t)1 << 30) - 256) return SQLLM_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(scale, 4)) return SQLLM_ERR_ALIGN;
    return status(launch_pieces<kNormFp8>(Rows{x, residual, weight, sum, q, scale, ldx, ldr, sqllm_fp8_cols(cols), 0,
                                               (int)cols, (int)(pitch * 128), (int)(pitch / 4), eps, 1. / cols},
                                          rows, stream));
}
