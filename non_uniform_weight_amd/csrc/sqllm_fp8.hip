// sqllm_fp8.hip -- the block-scaled 8-bit floating point calls of
// include/sqllm_fp8.h: argument checks, kernels and launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sqllm_fp8.h"

namespace {

constexpr int kBlock = 128;
constexpr int64_t kMaxCols = (int64_t)1 << 24;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Quantiser.  Sixteen lanes hold a block, eight values each.  The exponent
// comes from the bits of the block's largest magnitude m * 2^p (1 <= m < 2,
// exact in fp32): 448 = 1.75 * 2^8, so s = p - 8, one more if m > 1.75.
// Scaling by 2^-s is exact, and the conversion rounds to nearest even.
// ---------------------------------------------------------------------------

// The block exponent + 127 of its largest finite magnitude.
__device__ __forceinline__ uint32_t scale_byte(float top)
{
    const uint32_t b = __float_as_uint(top);
    if (b == 0) return 127;
    return (b >> 23) - 8 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
}

__device__ __forceinline__ float finite_magnitude(float v)
{
    const float m = fabsf(v);
    return m <= 65504.f ? m : 0.f; // false for NaN too
}

// Four values to e4m3 at 2^-s; infinities become NaN.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d, float inv)
{
    auto fix = [](float v) { return fabsf(v) <= 65504.f ? v : __builtin_nanf(""); };
    uint32_t r = __builtin_amdgcn_cvt_pk_fp8_f32(fix(a) * inv, fix(b) * inv, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(fix(c) * inv, fix(d) * inv, r, true);
}

// One block of 128 columns a sixteen-lane row of the wave, in a loop over the
// grid (row, block) with the pitch's padding among the blocks.
__global__ void __launch_bounds__(256) quantize_kernel(const uint16_t *__restrict__ x, uint32_t total, int cols,
                                                       int64_t ldx, int blocks, uint32_t pitch,
                                                       uint8_t *__restrict__ q, uint8_t *__restrict__ scale)
{
    const int part = threadIdx.x & 15;
    for (uint32_t id = blockIdx.x * 16u + (threadIdx.x >> 4); id < total; id += gridDim.x * 16u) {
        const uint32_t row = id / pitch, b = id - row * pitch;
        if ((int)b >= blocks) {
            if (part == 0) scale[id] = 127;
            continue;
        }
        const int c0 = b * kBlock + part * 8;
        const uint16_t *src = x + (int64_t)row * ldx;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = c0 + k < cols ? (float)__builtin_bit_cast(_Float16, src[c0 + k]) : 0.f;
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, finite_magnitude(v[k]));
#pragma unroll
        for (int m = 8; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
        const uint32_t sb = scale_byte(top);
        const float inv = __uint_as_float((254 - sb) << 23);
        const u32x2 out = {to_e4m3(v[0], v[1], v[2], v[3], inv), to_e4m3(v[4], v[5], v[6], v[7], inv)};
        *(u32x2 *)(q + (int64_t)row * blocks * kBlock + c0) = out;
        if (part == 0) scale[id] = (uint8_t)sb;
    }
}

// ---------------------------------------------------------------------------
// Product.  v_mfma_scale_f32_16x16x128_f8f6f4: lane l gives 32 bytes of row
// l % 16 of A (here W) and of B (here x), and one scale byte for them.  The
// instruction sums over all 128 positions, so any order of a block's columns
// will do as long as A and B agree: quarter l / 16 takes the 16-byte pieces
// l / 16 and 4 + l / 16, which keeps the loads of a row 64 bytes wide.  The
// four quarters of a row pass the block's one scale.  Register i of lane l
// holds the sum of W row 4 (l / 16) + i and x row l % 16.
// ---------------------------------------------------------------------------

__device__ __forceinline__ i32x8 load_piece(const uint8_t *row, int quarter)
{
    const u32x4 lo = *(const u32x4 *)(row + quarter * 16), hi = *(const u32x4 *)(row + 64 + quarter * 16);
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__global__ void __launch_bounds__(64) gemm_simple(const uint8_t *__restrict__ wq, const uint8_t *__restrict__ wscale,
                                                  int rows, const uint8_t *__restrict__ xq,
                                                  const uint8_t *__restrict__ xscale, int batch, int blocks, int pitch,
                                                  uint16_t *__restrict__ y)
{
    const int lane = threadIdx.x, n = lane & 15, quarter = lane >> 4;
    const int r0 = blockIdx.x * 16, b0 = blockIdx.y * 16;
    const int wr = min(r0 + n, rows - 1), xr = min(b0 + n, batch - 1); // rows past the end: copies, not stored
    const uint8_t *wp = wq + (int64_t)wr * blocks * kBlock, *xp = xq + (int64_t)xr * blocks * kBlock;
    const uint8_t *ws = wscale + (int64_t)wr * pitch, *xs = xscale + (int64_t)xr * pitch;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < blocks; ++k)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(load_piece(wp + k * kBlock, quarter),
                                                              load_piece(xp + k * kBlock, quarter), acc, 0, 0, 0,
                                                              (int)ws[k], 0, (int)xs[k]);
    const int b = b0 + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * quarter + i;
        if (b < batch && r < rows) y[(int64_t)b * rows + r] = __builtin_bit_cast(uint16_t, (_Float16)acc[i]);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool good_shape(int64_t rows, int64_t cols)
{
    return rows >= 1 && rows <= INT32_MAX && cols >= 1 && cols <= kMaxCols &&
           rows * sqllm_fp8_scale_pitch(cols) <= INT32_MAX / 2;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

sqllm_status quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, uint8_t *q, uint8_t *scale,
                      hipStream_t stream)
{
    const int blocks = (int)(sqllm_fp8_cols(cols) / kBlock), pitch = (int)sqllm_fp8_scale_pitch(cols);
    const int64_t wgs = (rows * pitch + 15) / 16;
    hipLaunchKernelGGL(quantize_kernel, dim3((unsigned)(wgs < 65536 ? wgs : 65536)), dim3(256), 0, stream, x,
                       (uint32_t)(rows * pitch), (int)cols, ldx, blocks, (uint32_t)pitch, q, scale);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}

} // namespace

extern "C" int64_t sqllm_fp8_cols(int64_t cols)
{
    return cols < 1 || cols > kMaxCols ? 0 : (cols + kBlock - 1) / kBlock * kBlock;
}

extern "C" int64_t sqllm_fp8_scale_pitch(int64_t cols)
{
    return cols < 1 || cols > kMaxCols ? 0 : (cols + 4 * kBlock - 1) / (4 * kBlock) * 4;
}

extern "C" sqllm_status sqllm_fp8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, uint8_t *q,
                                           uint8_t *scale, hipStream_t stream)
{
    if (!x || !q || !scale) return SQLLM_ERR_NULL;
    if (!good_shape(rows, cols) || ldx < cols) return SQLLM_ERR_SHAPE;
    if (!aligned(x, 2) || !aligned(q, 16) || !aligned(scale, 4)) return SQLLM_ERR_ALIGN;
    return quantize(x, rows, cols, ldx, q, scale, stream);
}

extern "C" size_t sqllm_fp8_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    if (!good_shape(rows, cols) || batch < 1 || !good_shape(batch, cols)) return 0;
    return up256((size_t)batch * sqllm_fp8_cols(cols)) + up256((size_t)batch * sqllm_fp8_scale_pitch(cols));
}

extern "C" sqllm_status sqllm_fp8_gemm(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                       const uint16_t *x, int64_t batch, uint16_t *y, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    if (!q || !scale || !x || !y) return SQLLM_ERR_NULL;
    if (!good_shape(rows, cols)) return SQLLM_ERR_SHAPE;
    if (batch < 1 || !good_shape(batch, cols)) return SQLLM_ERR_BATCH;
    if (!aligned(q, 16) || !aligned(scale, 4) || !aligned(x, 2) || !aligned(y, 2)) return SQLLM_ERR_ALIGN;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < sqllm_fp8_workspace_bytes(rows, cols, batch))
        return SQLLM_ERR_WORKSPACE;
    uint8_t *xq = (uint8_t *)workspace, *xs = xq + up256((size_t)batch * sqllm_fp8_cols(cols));
    sqllm_status st = quantize(x, batch, cols, cols, xq, xs, stream);
    if (st != SQLLM_OK) return st;
    hipLaunchKernelGGL(gemm_simple, dim3((unsigned)((rows + 15) / 16), (unsigned)((batch + 15) / 16)), dim3(64), 0,
                       stream, q, scale, (int)rows, xq, xs, (int)batch, (int)(sqllm_fp8_cols(cols) / kBlock),
                       (int)sqllm_fp8_scale_pitch(cols), y);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}
