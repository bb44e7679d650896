// sqllm_fp8.hip -- the block-scaled 8-bit floating point calls of
// include/sqllm_fp8.h: argument checks, kernels and launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
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
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Quantiser.  The exponent comes from the bits of the block's largest finite
// magnitude m * 2^p (1 <= m < 2, exact in fp32): 448 = 1.75 * 2^8, so s =
// p - 8, one more if m > 1.75.  v_cvt_scalef32_pk_fp8_f16 divides two fp16
// values by a power of two and rounds them to e4m3, ties to even; infinities
// and NaN become NaN.
// ---------------------------------------------------------------------------

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef short short2_t __attribute__((ext_vector_type(2)));
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

// The block exponent + 127 of its largest finite magnitude (fp16 bits).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const uint32_t b = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)top));
    if (b == 0) return 127;
    return (b >> 23) - 8 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
}

__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b)
{
    const ushort2_t m = __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a), __builtin_bit_cast(ushort2_t, b));
    return __builtin_bit_cast(uint32_t, m);
}

// The largest finite magnitude of N pairs of fp16 values.  Magnitudes are
// compared as 16-bit numbers plus 0x8400, which wraps infinities and NaN
// (0x7C00 and up) to the bottom; finite_bits takes it off again.
template <int N>
__device__ __forceinline__ uint32_t magnitude(const uint32_t (&v)[N])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const ushort2_t a = __builtin_bit_cast(ushort2_t, v[k] & 0x7FFF7FFFu) + ushort2_t{0x8400, 0x8400};
        m = max16(m, __builtin_bit_cast(uint32_t, a));
    }
    return max(m & 0xFFFF, m >> 16);
}

__device__ __forceinline__ uint32_t finite_bits(uint32_t m) { return m >= 0x8400 ? m - 0x8400 : 0; }

// Two pairs to four e4m3 codes at 2^-s, scale = 2^s.
__device__ __forceinline__ uint32_t to_e4m3(uint32_t a, uint32_t b, float scale)
{
    short2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(half2_t, a), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(half2_t, b), scale, true);
    return __builtin_bit_cast(uint32_t, r);
}

// The largest v of each sixteen lanes, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
#define SQLLM_ROR(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xF, 0xF, true))
    SQLLM_ROR(8);
    SQLLM_ROR(4);
    SQLLM_ROR(2);
    SQLLM_ROR(1);
#undef SQLLM_ROR
    return v;
}

// Eight values of a row from column c on, zeros past its end.
template <bool VECTOR>
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int c, int cols)
{
    if (VECTOR && c + 8 <= cols) return *(const u32x4 *)(row + c);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = c + k < cols ? row[c + k] : 0;
    return u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

// Sixteen lanes quantise four adjacent blocks of a row (one word of scales),
// eight values a lane and block, all four loads in flight at once.  VECTOR:
// rows are 16-byte aligned.
template <bool VECTOR>
__global__ void __launch_bounds__(256) quantize_kernel(const uint16_t *__restrict__ x, uint32_t total, int cols,
                                                       int64_t ldx, int blocks, uint32_t words,
                                                       uint8_t *__restrict__ q, uint32_t *__restrict__ scale)
{
    const int part = threadIdx.x & 15;
    for (uint32_t id = blockIdx.x * 16u + (threadIdx.x >> 4); id < total; id += gridDim.x * 16u) {
        const uint32_t row = id / words, b0 = (id - row * words) * 4;
        const uint16_t *src = x + (int64_t)row * ldx;
        u32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = u32x4{0, 0, 0, 0};
            if ((int)b0 + k < blocks) v[k] = load8<VECTOR>(src, (b0 + k) * kBlock + part * 8, cols);
        }
        uint32_t word = 0;
        u32x2 *out = (u32x2 *)(q + (int64_t)row * blocks * kBlock + b0 * kBlock) + part;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            const uint32_t sb = scale_byte(finite_bits(row_max(magnitude(w))));
            word |= sb << (8 * k);
            const float f = scale_value(sb);
            if ((int)b0 + k < blocks) out[k * (kBlock / 8)] = u32x2{to_e4m3(w[0], w[1], f), to_e4m3(w[2], w[3], f)};
        }
        if (part == 0) scale[id] = word;
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

// The same of split blockIdx.y, unrounded.
__device__ __forceinline__ void store_partial(const Operands &p, float *partial, int b, int r, f32x4 v)
{
    if (b >= p.batch) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < p.rows) partial[((int64_t)blockIdx.y * p.batch + b) * p.rows + r + i] = v[i];
}

// Each lane's 16 (4) bytes at src to lds_base + 16 (4) * lane.
__device__ __forceinline__ void lds_load16(const uint8_t *src, uint8_t *lds_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)src,
                                     (__attribute__((address_space(3))) uint32_t *)lds_base, 16, 0, 0);
}

__device__ __forceinline__ void lds_load4(const uint8_t *src, uint8_t *lds_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)src,
                                     (__attribute__((address_space(3))) uint32_t *)lds_base, 4, 0, 0);
}

// Tiled form.  A workgroup computes TM rows of W by TN rows of x over the
// blocks of its split, each wave WM by WN of them in 16x16 accumulators.  Both
// operands and their scales go through LDS, 128 columns (one block) a stage,
// S stages in turn: loads go straight from memory into LDS, S - 1 stages
// ahead of the matrix cores, and one barrier a stage separates them.  Every
// wave issues the same number of loads in every stage (past the last block it
// reads that again), so that the count of loads in flight says which stage has
// arrived.  A row's eight 16-byte pieces are stored at piece ^ (row % 8), so
// that the sixteen rows that a fragment read takes at one piece lie in
// different banks; loads into LDS write lane after lane, so the swizzle is in
// the address they read from.
// With splits > 1 the fp32 sums go to partial[split][batch][rows].
template <int TM, int TN, int WM, int WN, int S>
struct Tiling {
    static constexpr int W = (TM / WM) * (TN / WN);
    static constexpr int kData = (TM + TN) * kBlock, kScales = (TM + TN) * 4;
    static constexpr int kLoads = (TM + TN) / 8 / W;                  // 1 KB each
    static constexpr int kScaleWaves = (TM + TN + 63) / 64;            // waves that load scales, 64 rows each
    static constexpr size_t kLds = (size_t)S * (kData + kScaleWaves * 256);
    static_assert((TM + TN) / 8 % W == 0, "as many loads in every wave");
    static_assert(kScaleWaves <= W && TM % 16 == 0, "one load of scales a wave");
};

template <int N>
__device__ __forceinline__ void wait_loads() // until at most N of this wave's loads are in flight
{
    static_assert(N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Barrier after which every wave's loads into LDS but its latest N are there, and
// every wave's reads of LDS from before it are done: what it read may be loaded
// over.  (__syncthreads would wait for those N too: it is a fence for all memory.
// The wait for the reads is in one piece with the barrier, since the matrix steps
// that use them, and with them the compiler's own wait, may be moved past it; at
// present they are not, and it costs nothing.)
template <int N>
__device__ __forceinline__ void stage_barrier()
{
    wait_loads<N>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The tile of this workgroup: its first W row and x row; false if there is
// none.  Workgroups go round the eight XCDs: each gets a run of tiles, four W
// tiles wide, so that the 32 it works on at once share their rows in its L2.
template <int TM, int TN>
__device__ __forceinline__ bool tile_of(const Operands &p, int &r0, int &b0)
{
    constexpr int G = 4;
    const int mt = (p.rows + TM - 1) / TM, nt = (p.batch + TN - 1) / TN, tiles = mt * nt;
    const int per = (tiles + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= tiles) return false;
    const int group = id / (G * nt), in = id - group * (G * nt), width = min(G, mt - group * G);
    r0 = (group * G + in % width) * TM;
    b0 = (in / width) * TN;
    return true;
}

template <int TM, int TN, int WM, int WN, int S>
__global__ void __launch_bounds__(64 * (TM / WM) * (TN / WN), 2) gemm_tiled(Operands p, int splits, float *partial)
{
    using T = Tiling<TM, TN, WM, WN, S>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quarter = lane >> 4;
    int r0, b0;
    if (!tile_of<TM, TN>(p, r0, b0)) return;
    const int share = (p.blocks + splits - 1) / splits, k0 = blockIdx.y * share, k1 = min(k0 + share, p.blocks);
    if (k0 >= k1) return; // (the host leaves no split empty)

    // this wave's loads: 8 rows each of one operand; lane l reads piece
    // (l % 8) ^ (l / 8) of row l / 8.  Offsets from the tile's first row fit
    // 32 bits (255 rows of at most 2^24 columns).
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    const uint8_t *const wsrc = p.wq + (int64_t)r0 * ld, *const xsrc = p.xq + (int64_t)b0 * ld;
    uint32_t from[T::kLoads];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) { // rows past the end: copies of the last
        const int first = (w * T::kLoads + i) * 8, row = first + (lane >> 3);
        const int at = first < TM ? min(row, p.rows - 1 - r0) : min(row - TM, p.batch - 1 - b0);
        from[i] = (uint32_t)at * ld + ((lane & 7) ^ (lane >> 3)) * 16;
    }
    // and one of scales, four blocks of a row a lane (waves past kScaleWaves
    // repeat the last one's)
    const int sr = min(w, T::kScaleWaves - 1) * 64 + lane;
    const uint8_t *srow = sr < TM ? p.wscale + (int64_t)min(r0 + sr, p.rows - 1) * p.pitch
                                  : p.xscale + (int64_t)min(b0 + sr - TM, p.batch - 1) * p.pitch;
    uint8_t *const scales = lds + S * T::kData;
    auto load_stage = [&](int k, int slot) {
        const int at = min(k, k1 - 1);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i)
            lds_load16(((w * T::kLoads + i) * 8 < TM ? wsrc : xsrc) + (uint32_t)at * kBlock + from[i],
                       lds + slot * T::kData + (w * T::kLoads + i) * 1024);
        lds_load4(srow + (at & ~3), scales + (slot * T::kScaleWaves + min(w, T::kScaleWaves - 1)) * 256);
    };

    constexpr int FM = WM / 16, FN = WN / 16;
    const int wm = (w % (TM / WM)) * WM, wn = (w / (TM / WM)) * WN;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int piece = n * kBlock + ((quarter ^ (n & 7)) * 16);
    auto fragment = [&](const uint8_t *lo, const uint8_t *hi) {
        const u32x4 a = *(const u32x4 *)lo, b = *(const u32x4 *)hi;
        return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) load_stage(k0 + s, s);
    int slot = 0;
    for (int k = k0; k < k1; ++k) {
        stage_barrier<(S - 2) * (T::kLoads + 1)>(); // stage k is in LDS
        load_stage(k + S - 1, slot == 0 ? S - 1 : slot - 1); // where stage k - 1 was
        const uint8_t *base = lds + slot * T::kData, *lo = base + piece, *hi = base + (piece ^ 64);
        const int *sc = (const int *)(scales + slot * T::kScaleWaves * 256) + n;
        const int shift = 8 * (k & 3);
        slot = slot == S - 1 ? 0 : slot + 1;
        i32x8 b[FN];
        int sx[FN], sw[FM];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            b[j] = fragment(lo + (TM + wn + 16 * j) * kBlock, hi + (TM + wn + 16 * j) * kBlock);
            sx[j] = sc[TM + wn + 16 * j] >> shift;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) sw[i] = sc[wm + 16 * i] >> shift;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const i32x8 a = fragment(lo + (wm + 16 * i) * kBlock, hi + (wm + 16 * i) * kBlock);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[j], acc[i][j], 0, 0, 0, sw[i], 0, sx[j]);
        }
    }
    wait_loads<0>(); // none may land after the workgroup's LDS is someone else's
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int b = b0 + wn + 16 * j + n;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int r = r0 + wm + 16 * i + 4 * quarter;
            if (splits == 1)
                store4(p, b, r, acc[i][j]);
            else
                store_partial(p, partial, b, r, acc[i][j]);
        }
    }
}

// The tiled form for large products: 256x256 tiles in eight waves of 128x64.
// One stage at a time in flight (64 KB in turn with 64 KB in use) leaves the
// load path idle from a stage's arrival to the next barrier, and a stage takes
// about as long to arrive as to multiply.  Here LDS is a ring of five 32 KB
// units, W and x of a block in turn: W goes out two blocks ahead and x one,
// so that loads are in flight at all times.  The ring takes all of LDS; the
// scales come in registers, a word of four blocks a row, four blocks ahead.
constexpr int kUnit = 256 * kBlock, kUnits = 5;

// The swizzle here: a fragment read takes one piece of 32 rows, in two phases
// (rows 0-3, 12-15, 20-27 and the rest); within each, row % 2 and this number
// put the sixteen rows into the sixteen places of 16 bytes that the 64 banks
// have.
__device__ __forceinline__ int turn(int row) { return ((row >> 1) & 3) | ((row >> 4) & 1) << 2; }

__global__ void __launch_bounds__(512, 2) gemm_large(Operands p)
{
    constexpr int TM = 256, TN = 256, WM = 128, WN = 64, FM = WM / 32, FN = WN / 32;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, half = lane >> 5;
    int r0, b0;
    if (!tile_of<TM, TN>(p, r0, b0)) return;
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    const uint8_t *const wsrc = p.wq + (int64_t)r0 * ld, *const xsrc = p.xq + (int64_t)b0 * ld;
    uint32_t wfrom[4], xfrom[4]; // this wave's loads of a unit: rows 32 w .. 32 w + 31
#pragma unroll
    for (int i = 0; i < 4; ++i) { // rows past the end: copies of the last
        const int row = w * 32 + i * 8 + (lane >> 3), at = ((lane & 7) ^ turn(row)) * 16;
        wfrom[i] = (uint32_t)min(row, p.rows - 1 - r0) * ld + at;
        xfrom[i] = (uint32_t)min(row, p.batch - 1 - b0) * ld + at;
    }
    auto load_unit = [&](const uint8_t *src, const uint32_t (&from)[4], int k, int unit) {
        const uint32_t at = (uint32_t)min(k, p.blocks - 1) * kBlock;
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_load16(src + at + from[i], lds + unit * kUnit + (w * 4 + i) * 1024);
    };
    const int wm = (w & 1) * WM, wn = (w >> 1) * WN;
    uint32_t srow[FM + FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) srow[i] = (uint32_t)min(wm + 32 * i + n, p.rows - 1 - r0) * p.pitch;
#pragma unroll
    for (int i = 0; i < FN; ++i) srow[FM + i] = (uint32_t)min(wn + 32 * i + n, p.batch - 1 - b0) * p.pitch;
    const uint8_t *const wsc = p.wscale + (int64_t)r0 * p.pitch, *const xsc = p.xscale + (int64_t)b0 * p.pitch;
    int sc[FM + FN], next[FM + FN];
    auto load_scale = [&](int i, int k) {
        next[i] = *(const int *)((i < FM ? wsc : xsc) + (uint32_t)min(k & ~3, (p.blocks - 1) & ~3) + srow[i]);
    };
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    // this lane's two pieces of matrix step h (columns 64 h .. 64 h + 63): 4 h +
    // half and 4 h + 2 + half, at their swizzled places
    auto place = [&](int piece) { return n * kBlock + ((piece ^ turn(n)) * 16); };
    const uint8_t *at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = lds + place(2 * q + half);
    auto fragment = [&](int base, int h) {
        const u32x4 a = *(const u32x4 *)(at[2 * h] + base), b = *(const u32x4 *)(at[2 * h + 1] + base);
        return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    };
#pragma unroll
    for (int i = 0; i < FM + FN; ++i) load_scale(i, 0);
    load_unit(wsrc, wfrom, 0, 0);
    load_unit(xsrc, xfrom, 0, 1);
    load_unit(wsrc, wfrom, 1, 2);
    int unit = 0; // of W of block k; x is in the next one
    auto after = [](int u, int by) { return u + by >= kUnits ? u + by - kUnits : u + by; };
    auto step = [&](int k, auto byte) {
        constexpr int B = decltype(byte)::value;
        stage_barrier<4>(); // all but W of block k + 1 is in LDS
        if constexpr (B == 0) {
            // blocks past the last have scales of 2^-127: their products vanish
            const uint32_t keep = p.blocks - k >= 4 ? 0xFFFFFFFFu : (1u << (8 * (p.blocks - k))) - 1;
#pragma unroll
            for (int i = 0; i < FM + FN; ++i) sc[i] = next[i] & keep;
        }
        __builtin_amdgcn_sched_barrier(0);
        const int xu = after(unit, 1), f0 = after(unit, 3), f1 = after(unit, 4);
        const int abase = unit * kUnit + wm * kBlock, bbase = xu * kUnit + wn * kBlock;
        const uint32_t at0 = (uint32_t)min(k + 1, p.blocks - 1) * kBlock, at1 = (uint32_t)min(k + 2, p.blocks - 1) * kBlock;
        i32x8 b[2][FN], a[2];
#pragma unroll
        for (int j = 0; j < FN; ++j) b[0][j] = fragment(bbase + 32 * j * kBlock, 0);
        a[0] = fragment(abase, 0);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[1][j] = fragment(bbase + 32 * j * kBlock, 1);
        if constexpr (2 * B < FM + FN) {
            load_scale(2 * B, k + 4);
            load_scale(2 * B + 1, k + 4);
        }
        // loads go out between the matrix steps, x of the next block first
#pragma unroll
        for (int i = 0; i < 2 * FM; ++i) {
            if (i + 1 < 2 * FM) a[(i + 1) & 1] = fragment(abase + 32 * ((i + 1) % FM) * kBlock, (i + 1) / FM);
            if (i < 4)
                lds_load16(xsrc + at0 + xfrom[i & 3], lds + f0 * kUnit + (w * 4 + i) * 1024);
            else
                lds_load16(wsrc + at1 + wfrom[i & 3], lds + f1 * kUnit + (w * 4 + i - 4) * 1024);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i % FM][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i & 1], b[i / FM][j], acc[i % FM][j], 0, 0,
                                                                                 B, sc[i % FM], B, sc[FM + j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        unit = after(unit, 2);
    };
    for (int k = 0; k < p.blocks; k += 4) {
        step(k, std::integral_constant<int, 0>{});
        step(k + 1, std::integral_constant<int, 1>{});
        step(k + 2, std::integral_constant<int, 2>{});
        step(k + 3, std::integral_constant<int, 3>{});
    }
    wait_loads<0>(); // none may land after the workgroup's LDS is someone else's
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                store4(p, b0 + wn + 32 * j + n, r0 + wm + 32 * i + 8 * g + 4 * half,
                       f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
}

// y = the splits' sums, in order.
__global__ void __launch_bounds__(256) add_splits(const float *partial, int64_t total, int splits, uint16_t *y)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
        for (int s = 0; s < splits; ++s) v += partial[s * total + i];
        y[i] = __builtin_bit_cast(uint16_t, (_Float16)v);
    }
}

// Streaming form, for batches of at most 16: W is read once and the rest hides
// behind that.  A wave takes 16 R rows of W and every waves-th
// block of columns, D steps of loads in flight; the waves' sums are added in
// LDS.  W goes straight into LDS, each wave to a ring of its own (no barrier):
// an instruction reads whole 128-byte lines of eight rows, where loads into
// the matrix cores' register layout read 64 bytes of sixteen, which the memory
// answers a quarter slower (8192x8192: 19 us against 15).  FUSED: x comes in
// fp16 and each wave rounds the block it needs, about 80 vector instructions
// against the 2 R KB of W that the step reads; else in the stored form.  Few
// rows: the columns are split over `splits` workgroups, their sums going to
// partial[split][batch][rows].

// Keeps a uniform address in scalar registers, so that the loads add a 32-bit
// lane offset to it (otherwise each load gets a running 64-bit address of its
// own in vector registers).
typedef const __attribute__((address_space(1))) uint8_t *global_ptr;

__device__ __forceinline__ global_ptr scalar(const void *p)
{
    global_ptr g = (global_ptr)p;
    asm("" : "+s"(g));
    return g;
}

template <typename T>
__device__ __forceinline__ T load_at(global_ptr base, uint32_t offset)
{
    return *(const __attribute__((address_space(1))) T *)(base + offset);
}

constexpr int kStreamWaves = 8;

template <int R>
constexpr int stream_depth() { return R == 1 ? 4 : 3; }

template <int R>
constexpr size_t stream_lds() { return (size_t)kStreamWaves * stream_depth<R>() * R * 2048; }

template <int R, bool FUSED>
struct StreamStep {
    uint32_t ws[R];
    u32x4 x[FUSED ? 4 : 2];
    uint32_t xs;
};

template <int R, bool FUSED>
__global__ void __launch_bounds__(64 * kStreamWaves, 4) gemm_stream(Operands p, const uint16_t *x, int cols, int splits, float *partial)
{
    constexpr int D = stream_depth<R>(), kLoads = 3 * R + (FUSED ? 4 : 3); // loads of a step
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quarter = lane >> 4, r0 = blockIdx.x * 16 * R;
    uint8_t *const own = lds + w * D * R * 2048;
    // lane offsets from the tile's first row and from x fit 32 bits (at most 32
    // rows of 2^24 columns); rows past the last are copies, not stored
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    const uint8_t *wbase = p.wq + (int64_t)r0 * ld, *wsbase = p.wscale + (int64_t)r0 * p.pitch;
    uint32_t from[2 * R], wsp[R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i)
        from[i] = (uint32_t)min(8 * i + (lane >> 3), p.rows - 1 - r0) * ld + ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < R; ++i) wsp[i] = (uint32_t)min(16 * i + n, p.rows - 1 - r0) * p.pitch;
    const uint32_t xr = min(n, p.batch - 1), xf = xr * (uint32_t)cols, xq = xr * ld + quarter * 16, xs = xr * p.pitch;
    const int worker = blockIdx.y * kStreamWaves + w, workers = splits * kStreamWaves;
    const int steps = max(0, (p.blocks - worker + workers - 1) / workers);
    // A wave's i-th block.  Workgroups start at different ones: where the rows
    // are a power of two apart, the same block of all rows would lie in a few
    // of the memory's channels.
    const int turn = (int)(blockIdx.x * (uint32_t)kStreamWaves % (uint32_t)p.blocks);
    auto block_of = [&](int i) {
        const int k = worker + i * workers + turn;
        return k >= p.blocks ? k - p.blocks : k;
    };
    // first column of piece h of block k that this lane quantises
    auto column = [&](int k, int h) { return k * kBlock + (h >> 1) * 64 + (h & 1) * 8 + quarter * 16; };
    StreamStep<R, FUSED> ring[D];
    // every step issues the same loads in the same order, so that their count
    // tells which have arrived; past the wave's last block they read one again
    auto load = [&](int slot, int i) {
        StreamStep<R, FUSED> &s = ring[slot];
        const int k = steps ? block_of(min(i, steps - 1)) : 0;
#pragma unroll
        for (int j = 0; j < 2 * R; ++j)
            lds_load16(wbase + (uint32_t)k * kBlock + from[j], own + slot * R * 2048 + j * 1024);
        const global_ptr wsk = scalar(wsbase + k);
#pragma unroll
        for (int r = 0; r < R; ++r) s.ws[r] = load_at<uint8_t>(wsk, wsp[r]);
        if constexpr (FUSED) {
            // past the row's end (cols is a multiple of 8) its last eight, zeroed at use
#pragma unroll
            for (int h = 0; h < 4; ++h) s.x[h] = load_at<u32x4>(scalar(x), (xf + (uint32_t)min(column(k, h), cols - 8)) * 2);
        } else {
            const global_ptr xk = scalar(p.xq + (uint32_t)k * kBlock), xsk = scalar(p.xscale + k);
            s.x[0] = load_at<u32x4>(xk, xq);
            s.x[1] = load_at<u32x4>(xk, xq + 64);
            s.xs = load_at<uint8_t>(xsk, xs);
        }
        asm volatile("" ::: "memory"); // loads stay in this order
        __builtin_amdgcn_sched_barrier(0);
    };
    const int piece = n * kBlock + ((quarter ^ (n & 7)) * 16);
    f32x4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int slot, int i) {
        const StreamStep<R, FUSED> &s = ring[slot];
        wait_loads<(D - 1) * kLoads>(); // this step's are there
        asm volatile("" ::: "memory");
        i32x8 b;
        uint32_t sb;
        if constexpr (FUSED) {
            const int k = block_of(i);
            uint32_t v[16];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const bool in = column(k, h) < cols;
                v[4 * h] = in ? s.x[h].x : 0, v[4 * h + 1] = in ? s.x[h].y : 0;
                v[4 * h + 2] = in ? s.x[h].z : 0, v[4 * h + 3] = in ? s.x[h].w : 0;
            }
            uint32_t top = magnitude(v); // over the four lanes that hold the block of row n
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            sb = scale_byte(finite_bits(top));
            const float f = scale_value(sb);
#pragma unroll
            for (int h = 0; h < 8; ++h) b[h] = (int)to_e4m3(v[2 * h], v[2 * h + 1], f);
        } else {
            b = i32x8{(int)s.x[0].x, (int)s.x[0].y, (int)s.x[0].z, (int)s.x[0].w,
                      (int)s.x[1].x, (int)s.x[1].y, (int)s.x[1].z, (int)s.x[1].w};
            sb = s.xs;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint8_t *at = own + (slot * R + r) * 2048;
            const u32x4 lo = *(const u32x4 *)(at + piece), hi = *(const u32x4 *)(at + (piece ^ 64));
            const i32x8 a = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            acc[r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[r], 0, 0, 0, (int)s.ws[r], 0, (int)sb);
        }
        __builtin_amdgcn_sched_barrier(0); // the reads of this slot before the loads into it
    };
#pragma unroll
    for (int k = 0; k < D; ++k) load(k, k);
    int i = 0;
    for (; i + D <= steps; i += D) {
#pragma unroll
        for (int k = 0; k < D; ++k) {
            multiply(k, i + k);
            load(k, i + k + D);
        }
    }
    // the last steps issue no loads: fewer are in flight than multiply counts on
    wait_loads<0>();
#pragma unroll
    for (int k = 0; k < D - 1; ++k)
        if (i + k < steps) multiply(k, i + k);
    __syncthreads(); // the rings are done with: their LDS takes the sums
    f32x4 *const red = (f32x4 *)lds;
#pragma unroll
    for (int r = 0; r < R; ++r) red[(w * R + r) * 64 + lane] = acc[r];
    __syncthreads();
    for (int r = w; r < R; r += kStreamWaves) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < kStreamWaves; ++k) v += red[(k * R + r) * 64 + lane];
        if (splits == 1)
            store4(p, n, r0 + 16 * r + 4 * quarter, v);
        else
            store_partial(p, partial, n, r0 + 16 * r + 4 * quarter, v);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Within these, counts of tiles fit 32 bits and so do the work-items of every
// launch (a launch takes no more), and word indices of scales 32 bits.
bool good_shape(int64_t rows, int64_t cols)
{
    return rows >= 1 && rows <= INT32_MAX && cols >= 1 && cols <= kMaxCols &&
           rows * sqllm_fp8_scale_pitch(cols) <= ((int64_t)1 << 30) - 256;
}

bool good_product(int64_t rows, int64_t batch) { return rows * batch <= (int64_t)1 << 38; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

sqllm_status quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, uint8_t *q, uint8_t *scale,
                      hipStream_t stream)
{
    const int blocks = (int)(sqllm_fp8_cols(cols) / kBlock), words = (int)(sqllm_fp8_scale_pitch(cols) / 4);
    const int64_t wgs = (rows * words + 15) / 16;
    auto kern = aligned(x, 16) && ldx % 8 == 0 ? quantize_kernel<true> : quantize_kernel<false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(wgs < 65536 ? wgs : 65536)), dim3(256), 0, stream, x,
                       (uint32_t)(rows * words), (int)cols, ldx, blocks, (uint32_t)words, q, (uint32_t *)scale);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}

void launch_add(const Operands &p, int splits, const float *partial, hipStream_t stream)
{
    const int64_t total = (int64_t)p.batch * p.rows, wgs = (total + 255) / 256;
    hipLaunchKernelGGL(add_splits, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, stream, partial, total, splits,
                       p.y);
}

// The streaming form for larger ones: where a wave has many blocks to read (us
// of the streaming and the tiled form at batch 1 and 16: 8192x22016 38 and 49,
// 45 and 52; 4096x11008 14 and 16, 16 and 17; 8192x8192 22 and 22, 24 and 23;
// 12288x4096 21 and 16, 26 and 16; 16384x2048 13 and 11, 15 and 11).
bool streams(int64_t cols, int64_t batch) { return batch <= 16 && cols > 8192; }

// Splits of a streamed product's columns, up to 256 workgroups in all and two
// blocks a wave at least.  Adding the sums up is a launch more, about 3.6 us of
// the host's time, so only where the rows are few enough for it to save that
// (batch 1 and 16, us at 1, 2, 4 and 8 splits: 256x8192 9.7, 8.8, 7.7, 8.4 and
// 17, 15, 12, 13; 1024x16384 17, 14, 12, 13 and 25, 20, 17, 18; 2048x16384 18,
// 17, 19, 20 and 27, 22, 26, 28; but 2048x8192 11, 11, 12, 17 and 18, 16, 17,
// 26).
int stream_splits(int64_t rows, int64_t blocks)
{
    if (blocks < 64 || rows > 16 * blocks) return 1;
    int s = 1;
    while (s < 8 && rows * s < 16 * 256 && blocks >= 4 * s * kStreamWaves) s *= 2;
    return s;
}

// A small matrix for a few rows of x: the streaming form in one launch that
// rounds x as it goes, while its workgroups fit the compute units at once.
// Every workgroup rounds all of x again, so a wave has at most 60 blocks' rows
// of x to round (or as many as that by compute unit, where there are more
// workgroups than units).  us of this form and of rounding x with tiles or
// streaming after it, replayed from a graph and, in brackets, back to back from
// a host that takes 12 to 13 for two launches:
//   1000x2048, 2 blocks a wave, batch 8 6.2 and 9.3 (7.6 and 10.7), 16 7.5 and
//     9.3 (7.7 and 10.6)
//   4096x4096, 4 blocks, 8 10.3 and 11.3 (10.2 and 12), 12 11.6 and 11.6 (11.5
//     and 12), 16 13.2 and 12.0 (13.1 and 12)
//   512x4096, 4 blocks, 12 10.6 and 10.1 (10.6 and 13), 16 12.2 and 10.5 (12.1
//     and 13)
//   2700x6016, 6 blocks, 8 10.3 and 11.9 (10.2 and 12), 12 12.0 and 12.2 (11.9
//     and 12), 16 13.6 and 12.4 (13.5 and 12)
//   2048x8192, 8 blocks, 1 11.4 and 10.4 (11.2 and 12), 4 12.1 and 10.6 (12.0
//     and 13), 8 13.6 and 10.8 (13.6 and 13), 16 17.8 and 11.4 (17.7 and 13)
//   1300x12800, 4 by compute unit, 8 15.0 and 15.0, 12 16.7 and 16.1, 16 18.6
//     and 17.2
//   28000x512, more rows than units, 1 15.5 and 7.8, 16 31.7 and 8.2
bool fits_one_launch(int64_t rows, int64_t cols, int64_t batch)
{
    if (batch > 16 || rows > 4096 || rows * cols > 1 << 24) return false;
    const int64_t blocks = sqllm_fp8_cols(cols) / kBlock;
    const int64_t units = std::max<int64_t>(rows, 16 * 256 / stream_splits(rows, blocks)); // of 16 x 256
    return batch * blocks * units <= 60 * kStreamWaves * 16 * 256;
}

template <int R, bool FUSED>
void launch_stream(const Operands &p, const uint16_t *x, int cols, float *partial, hipStream_t stream)
{
    auto kern = gemm_stream<R, FUSED>;
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)kern, asked, (int)stream_lds<R>());
    const int splits = stream_splits(p.rows, p.blocks);
    hipLaunchKernelGGL(kern, dim3((p.rows + 16 * R - 1) / (16 * R), splits), dim3(64 * kStreamWaves), stream_lds<R>(),
                       stream, p, x, cols, splits, partial);
    if (splits > 1) launch_add(p, splits, partial, stream);
}

template <int TM, int TN, int WM, int WN, int S>
void launch_tiled(const Operands &p, int splits, float *partial, hipStream_t stream)
{
    using T = Tiling<TM, TN, WM, WN, S>;
    auto kern = gemm_tiled<TM, TN, WM, WN, S>;
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)kern, asked, (int)T::kLds);
    const int64_t tiles = (int64_t)((p.rows + TM - 1) / TM) * ((p.batch + TN - 1) / TN);
    hipLaunchKernelGGL(kern, dim3((unsigned)((tiles + 7) / 8 * 8), splits), dim3(64 * T::W), T::kLds, stream, p, splits,
                       partial);
    if (splits > 1) launch_add(p, splits, partial, stream);
}

void launch_large(const Operands &p, hipStream_t stream)
{
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)gemm_large, asked, kUnits * kUnit);
    const int64_t tiles = (int64_t)((p.rows + 255) / 256) * ((p.batch + 255) / 256);
    hipLaunchKernelGGL(gemm_large, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(512), kUnits * kUnit, stream, p);
}

// The tiling of a product: the largest tile that still gives most compute
// units a workgroup, and splits of the columns where no tile does.  Measured,
// in us:
//   256x256 (gemm_large) against 128x128: 6144x8192 at batch 2048 (192 tiles
//     of 256) 112 and 147, 4096x8192 at 2816 (176) 121 and 132, 8192x8192 at
//     1024 (128) 107 and 100, 4096x4096 at 2048 (128) 62 and 49.
//   128x128 against 64x64: 4096x4096 at 768 (192 tiles of 128) 41 and 42, at
//     512 (128) 41 and 30; 12288x4096 at 256 (192) 41 and 43; 8192x8192 at 512
//     (256) 73 and 101, at 200 (128) 70 and 44.
//   64x64 against 64x32: 4096x4096 at 200 (256 tiles of 64) 17 and 21, at 96
//     (128) 16.4 and 15.3; 8192x8192 at 96 (256) 30 and 45.
//   One, two and four splits of 64x32 tiles: 4096x4096 at 20 (64 tiles) 14.3,
//     13.3, 12.3, at 96 (192) 15, 20, 22; 2048x8192 at 128 (128) 25, 19, 21;
//     1000x2048 at 20 (16) 9.4, 10.0, 9.6.
// From 16384 columns on, a split's sums cost little beside its products, and
// splits of a larger tile read less than small tiles do: 4096x16384 at 256
// 57 us with 128x128 in four splits, 71 with 64x64, 92 with 64x32; at 768 101
// with 128x128 in two splits, 131 in one, 164 with 64x64.
struct Choice {
    int tile; // of launch below
    int splits;
};

Choice choose(int64_t rows, int64_t cols, int64_t batch)
{
    const int64_t blocks = sqllm_fp8_cols(cols) / kBlock;
    auto tiles = [&](int tm, int tn) { return ((rows + tm - 1) / tm) * ((batch + tn - 1) / tn); };
    if (batch > 256 && tiles(256, 256) >= 160) return Choice{0, 1};
    const bool deep = blocks >= 128;
    const int64_t enough = deep ? 256 : 192;
    Choice c;
    int64_t wgs;
    if (batch > 64 && (deep || tiles(128, 128) >= enough))
        c.tile = 1, wgs = tiles(128, 128);
    else if (batch > 32 && (deep || tiles(64, 64) >= enough))
        c.tile = 2, wgs = tiles(64, 64);
    else
        c.tile = 3, wgs = tiles(64, 32);
    int64_t s = 1; // no split below eight blocks
    while (s < 8 && wgs * s < enough && blocks >= 32 && blocks >= 16 * s) s *= 2;
    const int64_t share = (blocks + s - 1) / s;
    c.splits = (int)((blocks + share - 1) / share); // none empty
    return c;
}

void launch_choice(const Choice &c, const Operands &p, float *partial, hipStream_t stream)
{
    if (c.tile == 0)
        launch_large(p, stream);
    else if (c.tile == 1)
        launch_tiled<128, 128, 64, 64, 2>(p, c.splits, partial, stream);
    else if (c.tile == 2)
        launch_tiled<64, 64, 32, 32, 4>(p, c.splits, partial, stream);
    else
        launch_tiled<64, 32, 16, 32, 4>(p, c.splits, partial, stream);
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
    if (!good_shape(rows, cols) || !good_shape(batch, cols) || !good_product(rows, batch)) return 0;
    int splits = streams(cols, batch) ? 1 : choose(rows, cols, batch).splits;
    if (streams(cols, batch) || fits_one_launch(rows, cols, batch))
        splits = std::max(splits, stream_splits(rows, sqllm_fp8_cols(cols) / kBlock));
    return up256((size_t)batch * sqllm_fp8_cols(cols)) + up256((size_t)batch * sqllm_fp8_scale_pitch(cols)) +
           (splits > 1 ? (size_t)splits * batch * rows * 4 : 0);
}

// As launch_product splits.
extern "C" size_t sqllm_fp8_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    if (!good_shape(rows, cols) || !good_shape(batch, cols) || !good_product(rows, batch)) return 0;
    const int splits = streams(cols, batch) ? stream_splits(rows, sqllm_fp8_cols(cols) / kBlock) : choose(rows, cols, batch).splits;
    return std::max<size_t>(splits > 1 ? (size_t)splits * batch * rows * 4 : 0, 256);
}

namespace {

// What both products check alike; x: in either form, aligned to x_align; need: scratch bytes of sizes in range.
sqllm_status check_product(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols, const void *x,
                           uintptr_t x_align, int64_t batch, const uint16_t *y, const void *workspace,
                           size_t workspace_bytes, size_t (*need)(int64_t, int64_t, int64_t))
{
    if (!q || !scale || !x || !y) return SQLLM_ERR_NULL;
    if (!good_shape(rows, cols)) return SQLLM_ERR_SHAPE;
    if (!good_shape(batch, cols)) return SQLLM_ERR_BATCH;
    if (!good_product(rows, batch)) return SQLLM_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(scale, 4) || !aligned(x, x_align) || !aligned(y, 2)) return SQLLM_ERR_ALIGN;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need(rows, cols, batch)) return SQLLM_ERR_WORKSPACE;
    return SQLLM_OK;
}

// The product of operands in the stored form.
sqllm_status launch_product(const Operands &p, int64_t cols, float *partial, hipStream_t stream)
{
    // Two groups of 16 rows a wave halve the reads of x, where there are rows
    // enough (8192x16384 at batch 1 and 16: 31 and 37 us against 40 and 52 with
    // one group; 4096x22016: 28 and 38 against 22 and 28).
    if (streams(cols, p.batch) && p.rows >= 8192)
        launch_stream<2, false>(p, nullptr, (int)cols, partial, stream);
    else if (streams(cols, p.batch))
        launch_stream<1, false>(p, nullptr, (int)cols, partial, stream);
    else
        launch_choice(choose(p.rows, cols, p.batch), p, partial, stream);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}

} // namespace

extern "C" sqllm_status sqllm_fp8_gemm(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                       const uint16_t *x, int64_t batch, uint16_t *y, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    sqllm_status st = check_product(q, scale, rows, cols, x, 2, batch, y, workspace, workspace_bytes,
                                    sqllm_fp8_workspace_bytes);
    if (st != SQLLM_OK) return st;
    uint8_t *xq = (uint8_t *)workspace, *xs = xq + up256((size_t)batch * sqllm_fp8_cols(cols));
    const Operands p = {q, scale, xq, xs, y, (int)rows, (int)batch, (int)(sqllm_fp8_cols(cols) / kBlock),
                        (int)sqllm_fp8_scale_pitch(cols)};
    float *partial = (float *)(xs + up256((size_t)batch * sqllm_fp8_scale_pitch(cols)));
    if (fits_one_launch(rows, cols, batch) && aligned(x, 16) && cols % 8 == 0) {
        launch_stream<1, true>(p, x, (int)cols, partial, stream);
        return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
    }
    st = quantize(x, batch, cols, cols, xq, xs, stream);
    return st != SQLLM_OK ? st : launch_product(p, cols, partial, stream);
}

extern "C" sqllm_status sqllm_fp8_gemm_stored(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                              const uint8_t *xq, const uint8_t *xscale, int64_t batch, uint16_t *y,
                                              void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!xscale) return SQLLM_ERR_NULL;
    const sqllm_status st = check_product(q, scale, rows, cols, xq, 16, batch, y, workspace, workspace_bytes,
                                          sqllm_fp8_stored_workspace_bytes);
    if (st != SQLLM_OK) return st;
    if (!aligned(xscale, 4)) return SQLLM_ERR_ALIGN;
    const Operands p = {q, scale, xq, xscale, y, (int)rows, (int)batch, (int)(sqllm_fp8_cols(cols) / kBlock),
                        (int)sqllm_fp8_scale_pitch(cols)};
    return launch_product(p, cols, (float *)workspace, stream);
}
