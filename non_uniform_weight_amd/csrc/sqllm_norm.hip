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

// The same over a row's threads.  ONE: they are a wave; else the workgroup, of
// up to sixteen, and `red` is sixteen words of LDS of its own.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, uint32_t *red)
{
    v = wave_sum(v);
    if constexpr (!ONE) {
        red[threadIdx.x >> 6] = __float_as_uint(v);
        __syncthreads();
        v = 0.f;
        for (uint32_t k = 0; k < blockDim.x >> 6; ++k) v += __uint_as_float(red[k]);
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

__device__ __forceinline__ float squares(u32x4 v, float sum)
{
    const half8_t h = __builtin_bit_cast(half8_t, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = __builtin_fmaf((float)h[k], (float)h[k], sum);
    return sum;
}

// 1 / sqrt(m) in two parts: the reciprocal root r and what one step of
// Newton's method adds to it, r (1 - m r^2) / 2, so that y has no rounding but
// that of its last addition.  (With r alone one code in a million more lands
// on the other side of a border between two codes.)
struct Root {
    float high, low;
};

__device__ __forceinline__ Root reciprocal_root(float m)
{
    const float r = rsqrtf(m), h = m * r, rest = __builtin_fmaf(m, r, -h);
    const float off = __builtin_fmaf(-rest, r, __builtin_fmaf(-h, r, 1.f));
    // not for m = 0 or infinity, where r says all
    return {r, m > 0.f && m < INFINITY ? 0.5f * r * off : 0.f};
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

__device__ __forceinline__ Inverse store_scale(const Rows &a, int64_t row, uint32_t top, bool first)
{
    if (first) ((float *)a.scale)[row] = scale_of(top);
    return inverse_of(top);
}

// A row in the registers of a wave (ONE; four rows a workgroup, no barrier) or
// of a workgroup, V pieces of eight values a thread: read once, written once.
template <int FORM, bool RES, bool ONE, int V>
__global__ void __launch_bounds__(ONE ? 256 : 1024) rows_kernel(Rows a)
{
    __shared__ uint32_t red[2][16];
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
    if constexpr (FORM != kQuantize) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (k * T + t) * 8;
            if (RES && a.sum && c < a.cols) store8(a.sum + row * a.cols, c, a.cols, v[k]);
            s += squares(v[k], 0.f);
        }
        const Root root = reciprocal_root(row_sum<ONE>(s, red[0]) / (float)a.cols + a.eps);
#pragma unroll
        for (int k = 0; k < V; ++k) normalized(v[k], w[k], root, y[k]);
        // (a root of infinity or NaN turns the zeros past the end into NaN)
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((k * T + t) * 8 + j >= a.cols) y[k][j] = 0.f;
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
        top = row_max<ONE>(top, red[1]);
        const Inverse inverse = store_scale(a, row, top, t == 0);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (k * T + t) * 8;
            if (c < a.span) *(u32x2 *)((int8_t *)a.out + row * a.ldo + c) = top >= kInf ? u32x2{0, 0} : integers(y[k], inverse);
        }
    }
}

// Longer rows: each pass reads the row again, sums of two from `sum` where they
// were kept (it may be x or the residual).
template <int FORM, bool RES>
__global__ void __launch_bounds__(1024) long_rows_kernel(Rows a)
{
    __shared__ uint32_t red[2][16];
    const int64_t row = blockIdx.x;
    const uint16_t *const x = a.x + row * a.ldx;
    Root root = {};
    if constexpr (FORM != kQuantize) {
        float s = 0.f;
        for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
            u32x4 v = load8(x, c, a.cols);
            if constexpr (RES) {
                v = add8(v, load8(a.residual + row * a.ldr, c, a.cols));
                if (a.sum) store8(a.sum + row * a.cols, c, a.cols, v);
            }
            s += squares(v, 0.f);
        }
        root = reciprocal_root(row_sum<false>(s, red[0]) / (float)a.cols + a.eps);
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
            normalized(v, c < a.cols ? load8(a.weight, c, a.cols) : u32x4{0, 0, 0, 0}, root, y);
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
        top = row_max<false>(top, red[1]);
        const Inverse inverse = store_scale(a, row, top, threadIdx.x == 0);
        for (int c = threadIdx.x * 8; c < a.span; c += 8192) {
            value(c, y);
            *(u32x2 *)((int8_t *)a.out + row * a.ldo + c) = top >= kInf ? u32x2{0, 0} : integers(y, inverse);
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
        Rows{x, nullptr, nullptr, nullptr, q, scale, ldx, 0, ld, 0, (int)cols, (int)ld, 0, 0.f}, rows, stream);
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
        Rows{x, residual, weight, sum, y, nullptr, ldx, ldr, cols, 0, (int)cols, (int)cols, 0, eps}, rows, stream));
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
        Rows{x, residual, weight, sum, q, scale, ldx, ldr, ld, 0, (int)cols, (int)ld, 0, eps}, rows, stream));
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
                                               (int)cols, (int)(pitch * 128), (int)(pitch / 4), eps},
                                          rows, stream));
}
