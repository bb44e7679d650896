// sqllm_fp8.hip -- the block-scaled 8-bit floating point calls of
// include/sqllm_fp8.h: argument checks, kernels and launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "sqllm_device.h"
#include "sqllm_fp8.h"

namespace {

constexpr int kBlock = 128;
constexpr int64_t kMaxCols = (int64_t)1 << 24;

using sqllm::dev::f32x4;
using sqllm::dev::u32x2;
using sqllm::dev::u32x4;
typedef int i32x8 __attribute__((ext_vector_type(8)));

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

// One product: W rows against x rows, both in the stored form.
struct Operands {
    const uint8_t *wq, *wscale, *xq, *xscale;
    uint16_t *y;
    int rows, batch, blocks, pitch;
};

// Four W rows r..r+3 of one x row, rounded once; in one store where the row of
// y is aligned for it.
__device__ __forceinline__ void store4(const Operands &p, int b, int r, f32x4 v)
{
    if (b >= p.batch || r >= p.rows) return;
    uint16_t *y = p.y + (int64_t)b * p.rows + r;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint16_t, (_Float16)v[i]);
    if (r + 4 <= p.rows && ((uintptr_t)y & 7) == 0) {
        *(u32x2 *)y = u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < p.rows) y[i] = h[i];
}

__device__ __forceinline__ void lds_load16(const uint8_t *src, uint8_t *lds_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)src,
                                     (__attribute__((address_space(3))) uint32_t *)lds_base, 16, 0, 0);
}

// Tiled form.  A workgroup computes TM rows of W by TN rows of x, each wave WM
// by WN of them in 16x16 accumulators.  Both operands go through LDS, 128
// columns (one block) at a time, two stages in turn: the loads of the next
// stage go straight from memory into LDS while the matrix cores work on this
// one, and one barrier per stage separates them.  A row's eight 16-byte
// pieces are stored at piece ^ (row % 8), so that the sixteen rows that a
// fragment read takes at one piece lie in different banks; the loads into LDS
// write lane after lane, so the swizzle is in the address they read from.
template <int TM, int TN, int WM, int WN>
__global__ void __launch_bounds__(64 * (TM / WM) * (TN / WN), 2) gemm_tiled(Operands p)
{
    constexpr int W = (TM / WM) * (TN / WN), STAGE = (TM + TN) * kBlock, LOADS = (TM + TN) / 8 / W;
    static_assert((TM + TN) / 8 % W == 0 && TM / 8 % LOADS == 0, "a wave loads rows of one operand");
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quarter = lane >> 4;
    const int mt = (p.rows + TM - 1) / TM, nt = (p.batch + TN - 1) / TN, tiles = mt * nt;
    // Workgroups go round the eight XCDs: give each a run of tiles, four W
    // tiles wide, so that the 32 it works on at once share their rows in its L2.
    constexpr int G = 4;
    const int per = (tiles + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= tiles) return;
    const int group = id / (G * nt), in = id - group * (G * nt), width = min(G, mt - group * G);
    const int r0 = (group * G + in % width) * TM, b0 = (in / width) * TN;

    // this wave's loads: 8 rows each of one operand; lane l reads piece
    // (l % 8) ^ (l / 8) of row l / 8.  Offsets from the tile's first row fit
    // 32 bits (255 rows of at most 2^24 columns).
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    const bool of_w = w * LOADS * 8 < TM;
    const uint8_t *src = of_w ? p.wq + (int64_t)r0 * ld : p.xq + (int64_t)b0 * ld;
    const int most = of_w ? p.rows - 1 - r0 : p.batch - 1 - b0; // rows past the end: copies of the last
    uint32_t from[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = (w * LOADS + i) * 8 + (lane >> 3) - (of_w ? 0 : TM);
        from[i] = (uint32_t)min(row, most) * ld + ((lane & 7) ^ (lane >> 3)) * 16;
    }
    auto load_stage = [&](int k, int half) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            lds_load16(src + (uint32_t)k * kBlock + from[i], lds + half * STAGE + (w * LOADS + i) * 1024);
    };

    constexpr int FM = WM / 16, FN = WN / 16;
    const int wm = (w % (TM / WM)) * WM, wn = (w / (TM / WM)) * WN;
    uint32_t ws[FM], xs[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) ws[i] = (uint32_t)min(r0 + wm + 16 * i + n, p.rows - 1) * p.pitch;
#pragma unroll
    for (int i = 0; i < FN; ++i) xs[i] = (uint32_t)min(b0 + wn + 16 * i + n, p.batch - 1) * p.pitch;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // byte addresses of this lane's two pieces of fragment row 0, per stage
    const int piece = n * kBlock + ((quarter ^ (n & 7)) * 16);
    const uint8_t *a_lo[2], *a_hi[2], *b_lo[2], *b_hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        a_lo[h] = lds + h * STAGE + wm * kBlock + piece;
        a_hi[h] = lds + h * STAGE + wm * kBlock + (piece ^ 64);
        b_lo[h] = lds + h * STAGE + (TM + wn) * kBlock + piece;
        b_hi[h] = lds + h * STAGE + (TM + wn) * kBlock + (piece ^ 64);
    }
    auto fragment = [&](const uint8_t *plo, const uint8_t *phi) {
        const u32x4 lo = *(const u32x4 *)plo, hi = *(const u32x4 *)phi;
        return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    int sw[FM], sx[FN]; // scales of four blocks
    auto stage = [&](int k, auto byte) {
        constexpr int B = decltype(byte)::value, H = B & 1;
        __builtin_amdgcn_s_waitcnt(0x0F70); // vmcnt(0): this wave's part of stage k is in LDS
        __syncthreads();
        if (k + 1 < p.blocks) load_stage(k + 1, H ^ 1);
        i32x8 b[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = fragment(b_lo[H] + j * 16 * kBlock, b_hi[H] + j * 16 * kBlock);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const i32x8 a = fragment(a_lo[H] + i * 16 * kBlock, a_hi[H] + i * 16 * kBlock);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[j], acc[i][j], 0, 0, B, sw[i], B, sx[j]);
        }
    };
    load_stage(0, 0);
    for (int k = 0; k < p.blocks; k += 4) {
#pragma unroll
        for (int i = 0; i < FM; ++i) sw[i] = *(const int *)(p.wscale + ws[i] + k);
#pragma unroll
        for (int i = 0; i < FN; ++i) sx[i] = *(const int *)(p.xscale + xs[i] + k);
        stage(k, std::integral_constant<int, 0>{});
        if (k + 1 < p.blocks) stage(k + 1, std::integral_constant<int, 1>{});
        if (k + 2 < p.blocks) stage(k + 2, std::integral_constant<int, 2>{});
        if (k + 3 < p.blocks) stage(k + 3, std::integral_constant<int, 3>{});
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int b = b0 + wn + 16 * j + n;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int r = r0 + wm + 16 * i + 4 * quarter;
            store4(p, b, r, acc[i][j]);
        }
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

template <int TM, int TN, int WM, int WN>
void launch_tiled(const Operands &p, hipStream_t stream)
{
    auto kern = gemm_tiled<TM, TN, WM, WN>;
    const size_t lds = 2 * (TM + TN) * kBlock;
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)kern, asked, (int)lds);
    const int64_t tiles = (int64_t)((p.rows + TM - 1) / TM) * ((p.batch + TN - 1) / TN);
    hipLaunchKernelGGL(kern, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(64 * (TM / WM) * (TN / WN)), lds, stream, p);
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
    const Operands p = {q, scale, xq, xs, y, (int)rows, (int)batch, (int)(sqllm_fp8_cols(cols) / kBlock),
                        (int)sqllm_fp8_scale_pitch(cols)};
    if (rows >= 512 && batch >= 512)
        launch_tiled<256, 256, 128, 64>(p, stream);
    else
        launch_tiled<128, 128, 64, 64>(p, stream);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}
