// sqllm_int8.hip -- the products of include/sqllm_int8.h: argument checks,
// kernels and launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "sqllm_device.h"
#include "sqllm_int8.h"
#include "sqllm_rows.h"

namespace {

constexpr int kBlock = 128; // columns of a stage
using sqllm::dev::f32x4;
using sqllm::dev::u32x2;
using sqllm::dev::u32x4;
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// v_mfma_i32_16x16x64_i8: lane l gives 16 bytes of row l % 16 of A (here W)
// and of B (here x).  The instruction sums over all 64 positions, so any order
// of the columns will do as long as A and B agree.  Register i of lane l holds
// the sum of W row 4 (l / 16) + i and x row l % 16.  All sums are exact, so
// their order, and how the columns are split, does not show in the result.
// ---------------------------------------------------------------------------

// One product of W rows with x rows, or (gated) two with the same x.
struct Operands {
    const int8_t *wq[2];
    const float *wscale[2];
    const int8_t *xq;
    const float *xscale;
    uint16_t *y;
    int rows, batch, blocks;
};

// Every rounding that the header names is made, in every form of a product: v
// is a number in fp32 before it is rounded to fp16 (the compiler would fuse the
// multiply before it with the rounding in some places and not in others).
__device__ __forceinline__ uint16_t half_of(float v)
{
    asm("" : "+v"(v));
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// A sum as a number; silu(g) u.
__device__ __forceinline__ float scaled(int sum, float xs, float ws) { return (float)sum * (xs * ws); }
__device__ __forceinline__ float gated(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// Four W rows r..r+3 of one x row, rounded once; in one store where the row of
// y is aligned for it.
__device__ __forceinline__ void store4(const Operands &p, int b, int r, const float (&v)[4])
{
    if (b >= p.batch || r >= p.rows) return;
    uint16_t *y = p.y + (int64_t)b * p.rows + r;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = half_of(v[i]);
    if (r + 4 <= p.rows && ((uintptr_t)y & 7) == 0) {
        *(u32x2 *)y = u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < p.rows) y[i] = h[i];
}

// Sums of W rows r..r+3 with x row b, of one or both products, to y.
template <bool GLU>
__device__ __forceinline__ void finish4(const Operands &p, int b, int r, i32x4 g, i32x4 u)
{
    if (b >= p.batch || r >= p.rows) return;
    const float xs = p.xscale[b];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = min(r + i, p.rows - 1);
        v[i] = scaled(g[i], xs, p.wscale[0][at]);
        if constexpr (GLU) v[i] = gated(v[i], scaled(u[i], xs, p.wscale[1][at]));
    }
    store4(p, b, r, v);
}

// The same of split blockIdx.y, as sums: partial[split][product][batch][rows].
template <bool GLU>
__device__ __forceinline__ void store_partial(const Operands &p, int *partial, int b, int r, i32x4 g, i32x4 u)
{
    if (b >= p.batch) return;
    const int64_t size = (int64_t)p.batch * p.rows;
    int *at = partial + blockIdx.y * (GLU ? 2 : 1) * size + (int64_t)b * p.rows + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < p.rows) {
            at[i] = g[i];
            if constexpr (GLU) at[size + i] = u[i];
        }
}

// Each lane's 16 bytes at src to lds_base + 16 * lane.
__device__ __forceinline__ void lds_load16(const int8_t *src, int8_t *lds_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)src,
                                     (__attribute__((address_space(3))) uint32_t *)lds_base, 16, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads() // until at most N of this wave's loads are in flight
{
    static_assert(N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Barrier after which every wave's loads into LDS but its latest N are there, and
// every wave's reads of LDS from before it are done: what it read may be loaded
// over.  (The wait for the reads is in one piece with the barrier, since the
// matrix steps that use them, and with them the compiler's own wait, may be
// moved past it.)
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

// Tiled form.  A workgroup computes TM rows of W (gated: TM / 2 of each matrix)
// by TN rows of x over the blocks of its split, each wave WM by WN of them in
// 16x16 accumulators (gated: WM / 2 rows of gate and the same of up, so that a
// lane holds both sums of a place).  Both operands go through LDS, one block a
// stage, S stages in turn: loads go straight from memory into LDS, S - 1
// stages ahead of the matrix cores, and one barrier a stage separates them.
// Every wave issues the same number of loads in every stage (past the last
// block it reads that again), so that the count of loads in flight says which
// stage has arrived.  A row's eight 16-byte pieces are stored at piece ^
// (row % 8), so that the sixteen rows that a fragment read takes at one piece
// lie in different banks; loads into LDS write lane after lane, so the swizzle
// is in the address they read from.
template <int TM, int TN, int WM, int WN, int S>
struct Tiling {
    static constexpr int W = (TM / WM) * (TN / WN);
    static constexpr int kData = (TM + TN) * kBlock;
    static constexpr int kLoads = (TM + TN) / 8 / W; // 1 KB each
    static constexpr size_t kLds = (size_t)S * kData;
    static_assert((TM + TN) / 8 % W == 0, "as many loads in every wave");
    static_assert(TM % 16 == 0 && WM % 32 == 0, "halves of whole loads and accumulators");
};

template <bool GLU, int TM, int TN, int WM, int WN, int S>
__global__ void __launch_bounds__(64 * (TM / WM) * (TN / WN), 2) gemm_tiled(Operands p, int splits, int *partial)
{
    using T = Tiling<TM, TN, WM, WN, S>;
    constexpr int kRows = GLU ? TM / 2 : TM; // of a matrix
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quarter = lane >> 4;
    int r0, b0;
    if (!tile_of<kRows, TN>(p, r0, b0)) return;
    const int share = (p.blocks + splits - 1) / splits, k0 = blockIdx.y * share, k1 = min(k0 + share, p.blocks);
    if (k0 >= k1) return; // (the host leaves no split empty)

    // this wave's loads: 8 rows each of one operand; lane l reads piece
    // (l % 8) ^ (l / 8) of row l / 8.  Offsets from the tile's first row fit
    // 32 bits (255 rows of at most 2^17 columns).
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    const int8_t *src[T::kLoads];
    uint32_t from[T::kLoads];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) { // rows past the end: copies of the last
        const int first = (w * T::kLoads + i) * 8, row = first + (lane >> 3);
        int at;
        if (first >= TM) {
            src[i] = p.xq + (int64_t)b0 * ld;
            at = min(row - TM, p.batch - 1 - b0);
        } else if constexpr (GLU) {
            src[i] = (first % WM >= WM / 2 ? p.wq[1] : p.wq[0]) + (int64_t)r0 * ld;
            at = min(row / WM * (WM / 2) + row % (WM / 2), p.rows - 1 - r0);
        } else {
            src[i] = p.wq[0] + (int64_t)r0 * ld;
            at = min(row, p.rows - 1 - r0);
        }
        from[i] = (uint32_t)at * ld + ((lane & 7) ^ (lane >> 3)) * 16;
    }
    auto load_stage = [&](int k, int slot) {
        const int at = min(k, k1 - 1);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i)
            lds_load16(src[i] + (uint32_t)at * kBlock + from[i], lds + slot * T::kData + (w * T::kLoads + i) * 1024);
    };

    constexpr int FM = WM / 16, FN = WN / 16;
    const int wm = (w % (TM / WM)) * WM, wn = (w / (TM / WM)) * WN;
    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int piece = n * kBlock + ((quarter ^ (n & 7)) * 16);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) load_stage(k0 + s, s);
    int slot = 0;
    for (int k = k0; k < k1; ++k) {
        stage_barrier<(S - 2) * T::kLoads>(); // stage k is in LDS
        load_stage(k + S - 1, slot == 0 ? S - 1 : slot - 1); // where stage k - 1 was
        const int8_t *base = lds + slot * T::kData;
        slot = slot == S - 1 ? 0 : slot + 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) { // 64 columns: pieces 4 h + quarter
            const int8_t *at = base + (piece ^ (64 * h));
            i32x4 b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = *(const i32x4 *)(at + (TM + wn + 16 * j) * kBlock);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const i32x4 a = *(const i32x4 *)(at + (wm + 16 * i) * kBlock);
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    wait_loads<0>(); // none may land after the workgroup's LDS is someone else's
    constexpr int FR = GLU ? FM / 2 : FM;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int b = b0 + wn + 16 * j + n;
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            const int r = r0 + (GLU ? wm / 2 : wm) + 16 * i + 4 * quarter;
            if (splits == 1)
                finish4<GLU>(p, b, r, acc[i][j], acc[GLU ? i + FR : i][j]);
            else
                store_partial<GLU>(p, partial, b, r, acc[i][j], acc[GLU ? i + FR : i][j]);
        }
    }
}

// The tiled form for large products: 256 rows (gated: 128 of each matrix) by
// 256 rows of x in four waves of 128x128, the largest wave tile that the
// registers hold (256 of sums): LDS is read (128 + 128) / (128 * 128) bytes for
// each product, half of what waves of 64x64 read.  LDS is a ring of five 32 KB
// units, W and x of a block in turn.  A block's four matrix steps (32 columns
// each) read the fragments of the next step while they multiply, so the last
// step of a block reads the first of the next: the barrier that says that the
// next block is there, and that this one has been read, stands before it.  Its
// units are loaded over from there on, four loads a wave and step so that none
// waits for the others to go out: x of the block after the next in that step and
// the one behind it, then W of the block after that.
constexpr int kUnit = 256 * kBlock, kUnits = 5;

// The swizzle here: a fragment read takes one piece of 32 rows, in two phases
// (rows 0-3, 12-15, 20-27 and the rest); within each, row % 2 and this number
// put the sixteen rows into the sixteen places of 16 bytes that the 64 banks
// have.
__device__ __forceinline__ int turn(int row) { return ((row >> 1) & 3) | ((row >> 4) & 1) << 2; }

template <bool GLU>
__global__ void __launch_bounds__(256, 1) gemm_large(Operands p)
{
    constexpr int kRows = GLU ? 128 : 256, F = 4;
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, half = lane >> 5;
    int r0, b0;
    if (!tile_of<kRows, 256>(p, r0, b0)) return;
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    // this wave's loads of a unit: rows 64 w .. 64 w + 63 (gated: of one matrix)
    const int8_t *const wsrc = p.wq[GLU ? w & 1 : 0] + (int64_t)r0 * ld, *const xsrc = p.xq + (int64_t)b0 * ld;
    uint32_t wfrom[8], xfrom[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { // rows past the end: copies of the last
        const int row = w * 64 + i * 8 + (lane >> 3), at = ((lane & 7) ^ turn(row)) * 16;
        wfrom[i] = (uint32_t)min(GLU ? (w >> 1) * 64 + (row & 63) : row, p.rows - 1 - r0) * ld + at;
        xfrom[i] = (uint32_t)min(row, p.batch - 1 - b0) * ld + at;
    }
    auto load_w = [&](int i, int k, int unit) {
        lds_load16(wsrc + (uint32_t)min(k, p.blocks - 1) * kBlock + wfrom[i], lds + unit * kUnit + (w * 8 + i) * 1024);
    };
    auto load_x = [&](int i, int k, int unit) {
        lds_load16(xsrc + (uint32_t)min(k, p.blocks - 1) * kBlock + xfrom[i], lds + unit * kUnit + (w * 8 + i) * 1024);
    };
    const int wm = (w & 1) * 128, wn = (w >> 1) * 128;
    // the scales of this wave's rows, two W rows (gated: one of each matrix) and
    // four of x a lane
    float ws[2], xs[F];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        ws[i] = GLU ? p.wscale[i][min(r0 + wm / 2 + lane, p.rows - 1)] : p.wscale[0][min(r0 + wm + 64 * i + lane, p.rows - 1)];
#pragma unroll
    for (int j = 0; j < F; ++j) xs[j] = p.xscale[min(b0 + wn + 32 * j + n, p.batch - 1)];
    i32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = i32x16{};
    // this lane's piece of matrix step q: 2 q + half, at its swizzled place
    int at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = n * kBlock + (((2 * q + half) ^ turn(n)) * 16);
    auto fragment = [&](int base, int q, int i) { return *(const i32x4 *)(lds + (base + at[q]) + 32 * i * kBlock); };
    i32x4 a[2][F], b[2][F];
    auto after = [](int u, int by) { return u + by >= kUnits ? u + by - kUnits : u + by; };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_w(i, k, 2 * k);
#pragma unroll
        for (int i = 0; i < (k == 0 ? 8 : 4); ++i) load_x(i, k, 2 * k + 1);
    }
    stage_barrier<12>();
#pragma unroll
    for (int i = 0; i < F; ++i) {
        a[0][i] = fragment(wm * kBlock, 0, i);
        b[0][i] = fragment(kUnit + wn * kBlock, 0, i);
    }
    int unit = 0; // of W of block k; x is in the next one
    for (int k = 0; k < p.blocks; ++k) {
        const int next = after(unit, 2), free_x = after(unit, 3), free_w = after(unit, 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q == 3) stage_barrier<8>(); // all but W of block k + 2 is there, block k has been read
            const int wbase = (q == 3 ? next : unit) * kUnit + wm * kBlock, xbase = after(q == 3 ? next : unit, 1) * kUnit + wn * kBlock;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < F; j += 2) {
                    // two matrix steps, in the first half of a step each with a
                    // read of the next behind it, and a load, in this order
                    const int s = i * 2 + j / 2;
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[q & 1][i], b[q & 1][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (s < F) b[(q + 1) & 1][s] = fragment(xbase, (q + 1) & 3, s);
                    if (s % 2 == 1) {
                        if (q == 3) load_x(s / 2, k + 2, unit);
                        if (q == 0) load_x(4 + s / 2, k + 1, free_x);
                        if (q == 1 || q == 2) load_w(q * 4 - 4 + s / 2, k + 2, free_w);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    acc[i][j + 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[q & 1][i], b[q & 1][j + 1], acc[i][j + 1], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (s < F) a[(q + 1) & 1][s] = fragment(wbase, (q + 1) & 3, s);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        unit = next;
    }
    // The sums leave through LDS: a lane holds four rows of y's columns for one of
    // its rows, and stores of those would touch 64 lines each.  Every wave has its
    // own 32 KB: a row of x in 2 kOut bytes, in pieces of 8 bytes at piece ^
    // 2 (row % 16), which keeps pairs of them together.
    constexpr int FR = GLU ? F / 2 : F, kOut = FR * 32; // columns of y of this wave
    wait_loads<0>();
    asm volatile("s_barrier" ::: "memory"); // the units are done with, and no load is on its way into them
    float *const wsc = (float *)(lds + 4 * kUnit) + w * 128;
    wsc[lane] = ws[0], wsc[64 + lane] = ws[1];
    int8_t *const own = lds + w * kUnit;
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int r = 32 * i + 8 * g + 4 * half;
            const f32x4 s0 = *(const f32x4 *)(wsc + r);
            f32x4 s1 = s0;
            if constexpr (GLU) s1 = *(const f32x4 *)(wsc + 64 + r);
#pragma unroll
            for (int j = 0; j < F; ++j) {
                uint16_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = scaled(acc[i][j][4 * g + e], xs[j], s0[e]);
                    if constexpr (GLU) v = gated(v, scaled(acc[i + FR][j][4 * g + e], xs[j], s1[e]));
                    h[e] = half_of(v);
                }
                *(u32x2 *)(own + (32 * j + n) * (2 * kOut) + ((r / 4) ^ ((2 * n) & (kOut / 4 - 1) & 30)) * 8) =
                    u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
            }
        }
    constexpr int kLanes = kOut / 8; // of a row of x, eight columns of y each
    const int c = lane % kLanes, r = r0 + (GLU ? wm / 2 : wm) + 8 * c;
    const bool whole = p.rows % 8 == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll 4
    for (int k = 0; k < 128 / (64 / kLanes); ++k) {
        const int row = k * (64 / kLanes) + lane / kLanes, b = b0 + wn + row;
        const u32x4 v = *(const u32x4 *)(own + row * (2 * kOut) + ((2 * c) ^ ((2 * row) & (kOut / 4 - 1) & 30)) * 8);
        if (b >= p.batch || r >= p.rows) continue;
        uint16_t *const y = p.y + (int64_t)b * p.rows + r;
        if (whole) {
            *(u32x4 *)y = v;
            continue;
        }
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r + e < p.rows) y[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
    }
}

// Keeps a uniform address in scalar registers, so that the loads add a 32-bit
// lane offset to it.
typedef const __attribute__((address_space(1))) int8_t *global_ptr;

__device__ __forceinline__ global_ptr scalar(const void *p)
{
    global_ptr g = (global_ptr)p;
    asm("" : "+s"(g));
    return g;
}

__device__ __forceinline__ u32x4 load_once(global_ptr base, uint32_t offset)
{
    return __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4 *)(base + offset));
}

// The sum over each sixteen lanes, in all of them.
__device__ __forceinline__ int sum_of_16(int v)
{
#define SQLLM_ROR(n) v += __builtin_amdgcn_update_dpp(0, v, 0x120 + n, 0xF, 0xF, true)
    SQLLM_ROR(8);
    SQLLM_ROR(4);
    SQLLM_ROR(2);
    SQLLM_ROR(1);
#undef SQLLM_ROR
    return v;
}

// Streaming form, for few rows of x: W is read once, in whole kilobytes of a
// row, and multiplied in the vector units (v_dot4_i32_i8, four products an
// instruction).  A workgroup holds all of x in its registers: a chunk of 1024
// columns is sixteen of a lane's, and the workgroup's waves share the row's
// chunks, C of them a wave.  So it goes through groups of R rows (gated: R of
// each matrix), chunk c of the next group on its way as soon as chunk c of this
// one is used, and the waves' sums meet in LDS.  HALF: x comes in fp16.  Each
// lane rounds the columns that it holds, once, while the first rows of W are on
// their way; the largest of a row of x comes from all waves through LDS.
constexpr int kChunk = 1024;

template <bool GLU, bool HALF, int B, int C, int R>
__global__ void __launch_bounds__(1024) gemm_dot(Operands p, const uint16_t *x, int cols, int groups)
{
    constexpr int M = GLU ? 2 : 1, V = (R * B + 15) / 16; // sixteens of sums of a group and matrix
    __shared__ int part[2][16][M * V][64];
    __shared__ uint32_t tops[B][16];
    __shared__ float xscale[B];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int ld = p.blocks * kBlock;
    // chunks past the end: the row's last columns, with x of zero
    uint32_t col[C];
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * W + w) * kChunk + lane * 16;
        in[c] = at < ld, col[c] = min(at, ld - 16);
    }
    u32x4 buf[C][M][R];
    // (live: whether there is such a group; without one every lane reads the same)
    auto load = [&](int g, int c, bool live) {
        const uint32_t at = live ? col[c] : 0;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r)
                buf[c][m][r] = load_once(scalar(p.wq[m] + (int64_t)min(g * R + r, p.rows - 1) * ld), at);
        __builtin_amdgcn_sched_barrier(0);
    };
    i32x4 xr[B][C];
    if constexpr (!HALF) {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const i32x4 v = *(const i32x4 *)(p.xq + (uint32_t)min(b, p.batch - 1) * (uint32_t)ld + col[c]);
                xr[b][c] = in[c] ? v : i32x4{0, 0, 0, 0};
            }
        if (threadIdx.x < B) xscale[threadIdx.x] = p.xscale[min((int)threadIdx.x, p.batch - 1)];
    }
    // (x before W, so that it is rounded while W is on its way)
    u32x4 h[HALF ? B : 1][C][2];
    if constexpr (HALF) {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = (int)col[c] + 8 * k;
                    h[b][c][k] = u32x4{0, 0, 0, 0};
                    if (in[c] && at < cols) h[b][c][k] = sqllm::rows::load8(x + (int64_t)min(b, p.batch - 1) * cols, at, cols);
                }
        __builtin_amdgcn_sched_barrier(0);
    }
    int g = blockIdx.x;
#pragma unroll
    for (int c = 0; c < C; ++c) load(g, c, true);
    if constexpr (HALF) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[8];
                    sqllm::rows::floats(h[b][c][k], y);
                    top = max(top, sqllm::rows::magnitude(y));
                }
            top = sqllm::rows::wave_max(top);
            if (lane == 0) tops[b][w] = top;
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int b = 0; b < B; ++b) {
            uint32_t top = 0;
            for (int k = 0; k < W; ++k) top = max(top, tops[b][k]);
            const bool bad = top >= sqllm::rows::kInf;
            const sqllm::rows::Inverse inverse = sqllm::rows::inverse_of(top);
            if (threadIdx.x == 0) xscale[b] = sqllm::rows::scale_of(top);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                u32x2 q[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[8];
                    sqllm::rows::floats(h[b][c][k], y);
                    q[k] = sqllm::rows::integers(y, inverse);
                }
                xr[b][c] = bad ? i32x4{0, 0, 0, 0} : i32x4{(int)q[0].x, (int)q[0].y, (int)q[1].x, (int)q[1].y};
            }
        }
    }
    for (int turn = 0; g < groups; g += gridDim.x, ++turn) {
        const int next = g + gridDim.x;
        // this lane's places: sums (lane % 16) of each sixteen, row i of the group and x row b
        float ws[M][V];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int m = 0; m < M; ++m) ws[m][v] = p.wscale[m][min(g * R + (16 * v + (lane & 15)) / B, p.rows - 1)];
        int acc[M][R][B];
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        const i32x4 v = __builtin_bit_cast(i32x4, buf[c][m][i]);
                        int s = c == 0 ? 0 : acc[m][i][k];
#pragma unroll
                        for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_sdot4(v[e], xr[k][c][e], s, false);
                        asm volatile("" : "+v"(s)); // now, and not after the loads below
                        acc[m][i][k] = s;
                    }
            __builtin_amdgcn_sched_barrier(0);
            load(min(next, groups - 1), c, next < groups);
        }
        // sums over sixteen lanes, each of them in one of the sixteen
        int *const mine = &part[turn & 1][w][0][lane];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                int kept = 0;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (16 * v + k < R * B) {
                        const int s = sum_of_16(acc[m][(16 * v + k) / B][k % B]);
                        kept = (lane & 15) == k ? s : kept;
                    }
                mine[(m * V + v) * 64] = kept;
            }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (w != turn % W) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            int s[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                s[m] = 0;
                for (int k = 0; k < W; ++k) s[m] += part[turn & 1][k][m * V + v][lane];
                s[m] += __shfl_xor(s[m], 16);
                s[m] += __shfl_xor(s[m], 32);
            }
            const int at = 16 * v + lane, b = at % B, row = g * R + at / B;
            float y = scaled(s[0], xscale[b], ws[0][v]);
            if constexpr (GLU) y = gated(y, scaled(s[M - 1], xscale[b], ws[M - 1][v]));
            if (lane < 16 && at < R * B && b < p.batch && row < p.rows) p.y[(int64_t)b * p.rows + row] = half_of(y);
        }
    }
}

// Streaming form, for up to sixteen rows of x: as above on the matrix cores.
// A workgroup holds x in its registers, S blocks of 128 columns a wave (wave w
// those at w, w + W, ...), and goes through groups of 16 rows of W (gated: a
// group of gate, then the same of up).  W comes through LDS, each wave with a
// ring of D blocks of its own, loaded straight from memory, whole lines of eight
// rows an instruction (in the matrix cores' layout it would be 64 bytes of
// sixteen), D blocks ahead and on into the next group.
constexpr int few_waves(int S) { return S > 8 ? 12 : 16; } // most waves of a workgroup

template <bool GLU, int S, int D>
__global__ void __launch_bounds__(64 * few_waves(S)) gemm_few(Operands p, int groups)
{
    static_assert(S % D == 0, "a block's place in the ring is known");
    constexpr int M = GLU ? 2 : 1;
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int n = lane & 15, quarter = lane >> 4;
    int8_t *const ring = lds + w * (D * 2048);
    i32x4 *const part = (i32x4 *)(lds + W * (D * 2048)); // [2][W][64]
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    // This wave's blocks, from another one on in each workgroup: where the rows
    // are a power of two apart, the same block of all rows would lie in a few of
    // the memory's channels.  Past the last it loads block 0, unused.
    uint32_t at[S];
    bool in[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int block = ((s + blockIdx.x) % S) * W + w;
        in[s] = block < p.blocks, at[s] = in[s] ? (uint32_t)block * kBlock : 0;
    }
    i32x4 x[S][2]; // on its way before W, and not waited for before it
    const int8_t *const xrow = p.xq + (uint32_t)min(n, p.batch - 1) * ld + quarter * 16;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[s][h] = *(const i32x4 *)(xrow + at[s] + 64 * h);
    const float xs = p.xscale[min(n, p.batch - 1)];
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // lane l loads piece (l % 8) ^ (l / 8) of row l / 8 of eight
    const int8_t *src[2];
    auto rows_of = [&](int turn) { // of the turn's matrix and group
        const int g = blockIdx.x + turn / M * gridDim.x, m = turn % M;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            src[k] = p.wq[m] + (int64_t)min(min(g, groups - 1) * 16 + 8 * k + (lane >> 3), p.rows - 1) * ld +
                     ((lane & 7) ^ (lane >> 3)) * 16;
    };
    auto load = [&](int s) {
#pragma unroll
        for (int k = 0; k < 2; ++k) lds_load16(src[k] + at[s], ring + (s % D) * 2048 + k * 1024);
        asm volatile("" ::: "memory"); // loads stay in this order
        __builtin_amdgcn_sched_barrier(0);
    };
    const int turns = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * M;
    rows_of(0);
#pragma unroll
    for (int s = 0; s < D; ++s) load(s);
    const int piece = n * kBlock + ((quarter ^ (n & 7)) * 16);
    float ws[M][4] = {};
    i32x4 gate = {0, 0, 0, 0};
    for (int turn = 0; turn < turns; ++turn) {
        const int g = blockIdx.x + turn / M * gridDim.x, m = turn % M;
        // the wave that adds up this group asks for its scales before W of the next
        const bool mine = w == turn / M % W;
        if (mine && m == 0) {
#pragma unroll
            for (int k = 0; k < M; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) ws[k][i] = p.wscale[k][min(g * 16 + 4 * quarter + i, p.rows - 1)];
        }
        i32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            wait_loads<2 * (D - 1)>(); // this block is there (of more loads in flight, more are)
            asm volatile("" ::: "memory");
            const int8_t *const b = ring + (s % D) * 2048;
            const i32x4 lo = *(const i32x4 *)(b + piece), hi = *(const i32x4 *)(b + (piece ^ 64));
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); // read before it is loaded over
            __builtin_amdgcn_sched_barrier(0);
            if (s + D == S) rows_of(turn + 1); // (past the last turn the last rows again)
            load((s + D) % S);
            if (in[s]) {
                acc[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(lo, x[s][0], acc[0], 0, 0, 0);
                acc[1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(hi, x[s][1], acc[1], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        part[((turn & 1) * W + w) * 64 + lane] = acc[0] + acc[1];
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (!mine) continue;
        i32x4 v = {0, 0, 0, 0};
        for (int k = 0; k < W; ++k) v += part[((turn & 1) * W + k) * 64 + lane];
        if (m < M - 1) {
            gate = v;
            continue;
        }
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = GLU ? gated(scaled(gate[i], xs, ws[0][i]), scaled(v[i], xs, ws[M - 1][i])) : scaled(v[i], xs, ws[0][i]);
        store4(p, n, g * 16 + 4 * quarter, y);
    }
    wait_loads<0>(); // none may land after the workgroup's LDS is someone else's
}

// y from the splits' sums.
template <bool GLU>
__global__ void __launch_bounds__(256) add_splits(Operands p, const int *partial, int splits)
{
    const int64_t total = (int64_t)p.batch * p.rows;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        int g = 0, u = 0;
        for (int s = 0; s < splits; ++s) {
            g += partial[s * (GLU ? 2 : 1) * total + i];
            if constexpr (GLU) u += partial[(2 * s + 1) * total + i];
        }
        const int b = (int)(i / p.rows), r = (int)(i - (int64_t)b * p.rows);
        const float xs = p.xscale[b];
        float v = scaled(g, xs, p.wscale[0][r]);
        if constexpr (GLU) v = gated(v, scaled(u, xs, p.wscale[1][r]));
        p.y[i] = half_of(v);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 30;

bool good_sizes(int64_t rows, int64_t cols, int64_t batch)
{
    return rows >= 1 && rows <= kMaxRows && batch >= 1 && batch <= kMaxRows && sqllm_int8_cols(cols) > 0 &&
           rows * batch <= (int64_t)1 << 38;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The columns' splits of a product: `rows` of one matrix.
int splits_of(int64_t rows, int64_t cols, int64_t batch, bool glu)
{
    const int64_t blocks = sqllm_int8_cols(cols) / kBlock, mine = glu ? 32 : 64;
    const int64_t tiles = ((rows + mine - 1) / mine) * ((batch + 63) / 64);
    int64_t s = 1;
    while (s < 8 && tiles * s < 256 && blocks >= 16 * s) s *= 2;
    const int64_t share = (blocks + s - 1) / s;
    return (int)((blocks + share - 1) / share); // none empty
}

size_t workspace_bytes(int64_t rows, int64_t cols, int64_t batch, bool glu)
{
    if (!good_sizes(rows, cols, batch)) return 0;
    const int splits = splits_of(rows, cols, batch, glu);
    return up256((size_t)batch * sqllm_int8_cols(cols)) + up256((size_t)batch * 4) +
           (splits > 1 ? (size_t)splits * batch * rows * (glu ? 8 : 4) : 0);
}

template <bool GLU, int TM, int TN, int WM, int WN, int S>
void launch_tiled(const Operands &p, int splits, int *partial, hipStream_t stream)
{
    using T = Tiling<TM, TN, WM, WN, S>;
    auto kern = gemm_tiled<GLU, TM, TN, WM, WN, S>;
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)kern, asked, (int)T::kLds);
    constexpr int kRows = GLU ? TM / 2 : TM;
    const int64_t tiles = (int64_t)((p.rows + kRows - 1) / kRows) * ((p.batch + TN - 1) / TN);
    hipLaunchKernelGGL(kern, dim3((unsigned)((tiles + 7) / 8 * 8), splits), dim3(64 * T::W), T::kLds, stream, p, splits,
                       partial);
    if (splits > 1) {
        const int64_t wgs = ((int64_t)p.batch * p.rows + 255) / 256;
        hipLaunchKernelGGL(add_splits<GLU>, dim3((unsigned)std::min<int64_t>(wgs, 4096)), dim3(256), 0, stream, p, partial,
                           splits);
    }
}

template <bool GLU, bool HALF, int B, int C, int R>
void launch_dot(const Operands &p, const uint16_t *x, int cols, int waves, hipStream_t stream)
{
    const int groups = (p.rows + R - 1) / R;
    int wgs = 256 * (16 / waves);
    if (wgs > groups) wgs = groups;
    hipLaunchKernelGGL((gemm_dot<GLU, HALF, B, C, R>), dim3(wgs), dim3(64 * waves), 0, stream, p, x, cols, groups);
}

struct Dot {
    int waves, chunks; // of a wave; waves 0: not this form
};

Dot dot_shape(int64_t ld, int64_t batch)
{
    const int total = (int)((ld + kChunk - 1) / kChunk);
    if (batch > 4 || total > 48) return {0, 0};
    if (total <= 8) return {total, 1};
    if (total <= 16) return {(total + 1) / 2, 2};
    return {(total + 2) / 3, 3};
}

template <bool GLU, bool HALF, int B>
void launch_dots(const Operands &p, const uint16_t *x, int cols, Dot d, hipStream_t stream)
{
    if (d.chunks == 1) launch_dot<GLU, HALF, B, 1, 4>(p, x, cols, d.waves, stream);
    if constexpr (!HALF || B < 4)
        if (d.chunks == 2) launch_dot<GLU, HALF, B, 2, B == 1 ? 4 : 2>(p, x, cols, d.waves, stream);
    if constexpr (!HALF || B < 4)
        if (d.chunks == 3) launch_dot<GLU, HALF, B, 3, 2>(p, x, cols, d.waves, stream);
}

template <bool GLU, bool HALF>
void launch_dots(const Operands &p, const uint16_t *x, int cols, Dot d, hipStream_t stream)
{
    if (p.batch == 1)
        launch_dots<GLU, HALF, 1>(p, x, cols, d, stream);
    else if (p.batch == 2)
        launch_dots<GLU, HALF, 2>(p, x, cols, d, stream);
    else
        launch_dots<GLU, HALF, 4>(p, x, cols, d, stream);
}

template <bool GLU, int S, int D>
void launch_few(const Operands &p, hipStream_t stream)
{
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)gemm_few<GLU, S, D>, asked, 160 * 1024);
    const int groups = (p.rows + 15) / 16, waves = (p.blocks + S - 1) / S, lds = waves * (D * 2048 + 2 * 1024);
    const int wgs = std::min(groups, 256 * std::max(1, std::min(16 / waves, 160 * 1024 / lds)));
    hipLaunchKernelGGL((gemm_few<GLU, S, D>), dim3(wgs), dim3(64 * waves), lds, stream, p, groups);
}

template <bool GLU>
void launch_large(const Operands &p, hipStream_t stream)
{
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)gemm_large<GLU>, asked, kUnits * kUnit);
    const int64_t tiles = (int64_t)((p.rows + (GLU ? 127 : 255)) / (GLU ? 128 : 256)) * ((p.batch + 255) / 256);
    hipLaunchKernelGGL(gemm_large<GLU>, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(256), kUnits * kUnit, stream, p);
}

template <bool GLU>
sqllm_status product(const int8_t *const (&q)[2], const float *const (&scale)[2], int64_t rows, int64_t cols,
                     const void *x, const float *xscale, int64_t batch, uint16_t *y, void *workspace,
                     size_t workspace_size, hipStream_t stream)
{
    if (!q[0] || !scale[0] || !q[1] || !scale[1] || !x || !y) return SQLLM_ERR_NULL;
    if (rows < 1 || rows > kMaxRows || sqllm_int8_cols(cols) == 0) return SQLLM_ERR_SHAPE;
    if (batch < 1 || batch > kMaxRows) return SQLLM_ERR_BATCH;
    if (!good_sizes(rows, cols, batch)) return SQLLM_ERR_SHAPE;
    for (int k = 0; k < 2; ++k)
        if (!aligned(q[k], 16) || !aligned(scale[k], 4)) return SQLLM_ERR_ALIGN;
    if (!aligned(x, xscale ? 16 : 2) || !aligned(xscale, 4) || !aligned(y, 2)) return SQLLM_ERR_ALIGN;
    if (!workspace || !aligned(workspace, 256) || workspace_size < workspace_bytes(rows, cols, batch, GLU))
        return SQLLM_ERR_WORKSPACE;
    const int64_t ld = sqllm_int8_cols(cols);
    int8_t *const xq = (int8_t *)workspace;
    float *const xs = (float *)(xq + up256((size_t)batch * ld));
    int *const partial = (int *)((uint8_t *)xs + up256((size_t)batch * 4));
    Operands p = {{q[0], q[1]}, {scale[0], scale[1]}, (const int8_t *)x, xscale, y, (int)rows, (int)batch, (int)(ld / kBlock)};
    const Dot d = dot_shape(ld, batch);
    if (d.waves && !xscale && (batch <= 2 || (batch <= 4 && d.chunks == 1))) {
        launch_dots<GLU, true>(p, (const uint16_t *)x, (int)cols, d, stream);
        return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
    }
    if (!xscale) {
        if (sqllm::launch_int8_quantize((const uint16_t *)x, batch, cols, cols, xq, xs, stream) != hipSuccess)
            return SQLLM_ERR_HIP;
        p.xq = xq, p.xscale = xs;
    }
    if (d.waves) {
        launch_dots<GLU, false>(p, nullptr, (int)cols, d, stream);
    } else if (batch <= 16 && p.blocks <= 192) {
        if (p.blocks <= 32)
            launch_few<GLU, 2, 2>(p, stream);
        else if (p.blocks <= 64)
            launch_few<GLU, 4, 2>(p, stream);
        else if (p.blocks <= 128)
            launch_few<GLU, 8, 4>(p, stream);
        else
            launch_few<GLU, 16, 4>(p, stream);
    } else if (batch > 256 && rows > 2048)
        launch_large<GLU>(p, stream);
    else
        launch_tiled<GLU, 64, 64, 32, 32, 4>(p, splits_of(rows, cols, batch, GLU), partial, stream);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}

} // namespace

extern "C" size_t sqllm_int8_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, false);
}

extern "C" size_t sqllm_int8_glu_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, true);
}

extern "C" sqllm_status sqllm_int8_gemm(const int8_t *q, const float *scale, int64_t rows, int64_t cols, const void *x,
                                        const float *xscale, int64_t batch, uint16_t *y, void *workspace,
                                        size_t workspace_bytes, hipStream_t stream)
{
    return product<false>({q, q}, {scale, scale}, rows, cols, x, xscale, batch, y, workspace, workspace_bytes, stream);
}

extern "C" sqllm_status sqllm_int8_glu(const int8_t *gate, const float *gate_scale, const int8_t *up,
                                       const float *up_scale, int64_t rows, int64_t cols, const void *x,
                                       const float *xscale, int64_t batch, uint16_t *h, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    return product<true>({gate, up}, {gate_scale, up_scale}, rows, cols, x, xscale, batch, h, workspace,
                         workspace_bytes, stream);
}
