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

// A sum as a number; silu(g) u, the quotient by the hardware's reciprocal (a
// step of 2^-23; a division takes ten instructions, 1.5 us of a 256x256 tile).
__device__ __forceinline__ float scaled(int sum, float xs, float ws) { return (float)sum * (xs * ws); }
__device__ __forceinline__ float gated(float g, float u) { return g * __builtin_amdgcn_rcpf(1.f + __expf(-g)) * u; }

// y's rows begin at any even address: stores of 8 and 16 bytes all the same
// (global memory takes unaligned ones; 17700x751 at batch 3320 took 149 us by
// single values, takes 77 this way).
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
using sqllm::rows::u32x4_any;

// Four W rows r..r+3 of one x row, rounded once.
__device__ __forceinline__ void store4(const Operands &p, int b, int r, const float (&v)[4])
{
    if (b >= p.batch || r >= p.rows) return;
    uint16_t *y = p.y + (int64_t)b * p.rows + r;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = half_of(v[i]);
    if (r + 4 <= p.rows) {
        *(u32x2_any *)y = u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
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

// The same of split blockIdx.y, as sums: partial[split][product][batch][rows
// rounded up to four].
__host__ __device__ __forceinline__ int64_t partial_pitch(int64_t rows) { return (rows + 3) / 4 * 4; }

template <bool GLU>
__device__ __forceinline__ void store_partial(const Operands &p, int *partial, int b, int r, i32x4 g, i32x4 u)
{
    if (b >= p.batch || r >= p.rows) return;
    const int64_t pitch = partial_pitch(p.rows), size = p.batch * pitch;
    int *at = partial + blockIdx.y * (GLU ? 2 : 1) * size + b * pitch + r;
    *(i32x4 *)at = g;
    if constexpr (GLU) *(i32x4 *)(at + size) = u;
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
// Tiles `first` to `last` (0: all of them); halves: of tiles of 2 TN rows of x.
template <int TM, int TN>
__device__ __forceinline__ bool tile_of(const Operands &p, int wg, int first, int last, bool halves, int &r0, int &b0)
{
    constexpr int G = 4;
    const int wide = halves ? 2 * TN : TN;
    const int mt = (p.rows + TM - 1) / TM, nt = (p.batch + wide - 1) / wide, mine = ((last ? last : mt * nt) - first) * (halves ? 2 : 1);
    const int per = (mine + 7) / 8, at = (wg & 7) * per + (wg >> 3);
    if (wg >> 3 >= per || at >= mine) return false;
    const int id = first + (halves ? at / 2 : at);
    const int group = id / (G * nt), in = id - group * (G * nt), width = min(G, mt - group * G);
    r0 = (group * G + in % width) * TM;
    b0 = (in / width) * wide + (halves && at % 2 ? TN : 0);
    return b0 < p.batch;
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
// What bounds small tiles is neither memory nor the matrix cores.  By the counters
// W comes from memory once and x once for each XCD (8192x8192 at batch 256 84.0 MB,
// 83.9 needed): workgroups with the same rows of W do share them in their L2.  That
// is 4.1 TB/s at batch 17 and 2.4 at 256, with the matrix cores busy 7 and 23% of
// the time.  Waves stand at a wait for a third to a half of their cycles and before
// the issue of an instruction for a quarter to a third more: a stage is a short
// chain of latencies.  What was tried on it: 64x32 tiles, 8192x8192 at batch 64,
// with four stages 20.6 us, five and six 19.5, twelve 20.4; with every workgroup
// beginning at another block 19.6 to 25; 32 rows of W a tile, at batch 17, 15.4 us,
// in 64x32 tiles 18.2, with split columns 17.6.  So that more chains run side by
// side, a workgroup has G groups of waves: a stage is G blocks, one for each group,
// whose sums are added through LDS at the end.  32x16 tiles, 1024x8192 at batch 32,
// with four groups 7.8 us, with two 9.1; at 256 tiles (4096x4096) 7.2 and 7.0.
template <int TM, int TN, int WM, int WN, int S, int G>
struct Tiling {
    static constexpr int W = (TM / WM) * (TN / WN); // waves of a group
    static constexpr int kData = (TM + TN) * kBlock;
    static constexpr int kLoads = (TM + TN) / 8 / W; // 1 KB each
    static constexpr size_t kLds = (size_t)S * G * kData;
    static_assert((TM + TN) / 8 % W == 0, "as many loads in every wave");
    static_assert(TM % 16 == 0 && WM % 32 == 0, "halves of whole loads and accumulators");
    static_assert(kLds <= 160 * 1024 && (size_t)(G - 1) * TM * TN * 4 <= kLds, "LDS of a compute unit, and the other groups' sums");
};

template <bool GLU, int TM, int TN, int WM, int WN, int S, int G>
__global__ void __launch_bounds__(64 * (TM / WM) * (TN / WN) * G, 2) gemm_tiled(Operands p, int splits, int *partial)
{
    using T = Tiling<TM, TN, WM, WN, S, G>;
    constexpr int kRows = GLU ? TM / 2 : TM; // of a matrix
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = G > 1 ? wave / T::W : 0, w = wave - g * T::W;
    const int n = lane & 15, quarter = lane >> 4;
    int r0, b0;
    if (!tile_of<kRows, TN>(p, blockIdx.x, 0, 0, false, r0, b0)) return;
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
        const int at = min(k + g, k1 - 1);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i)
            lds_load16(src[i] + (uint32_t)at * kBlock + from[i], lds + (slot * G + g) * T::kData + (w * T::kLoads + i) * 1024);
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
    for (int s = 0; s < S - 1; ++s) load_stage(k0 + s * G, s);
    int slot = 0;
    for (int k = k0; k < k1; k += G) {
        stage_barrier<(S - 2) * T::kLoads>(); // stage k is in LDS
        load_stage(k + (S - 1) * G, slot == 0 ? S - 1 : slot - 1); // where the stage before k was
        const int8_t *base = lds + (slot * G + g) * T::kData;
        slot = slot == S - 1 ? 0 : slot + 1;
        if (G > 1 && k + g >= k1) continue; // (a copy of the last)
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
    if constexpr (G > 1) {
        __syncthreads(); // (the stages' reads and loads are done)
        i32x4 *const sums = (i32x4 *)lds + w * FM * FN * 64 + lane;
        if (g) {
#pragma unroll
            for (int i = 0; i < FM * FN; ++i) sums[((g - 1) * T::W * FM * FN + i) * 64] = acc[i / FN][i % FN];
        }
        __syncthreads();
        if (g) return;
#pragma unroll
        for (int i = 0; i < FM * FN; ++i)
#pragma unroll
            for (int k = 0; k < G - 1; ++k) acc[i / FN][i % FN] += sums[(k * T::W * FM * FN + i) * 64];
    }
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

// The tiled form for more rows of x: 64 FM rows (gated: half of them of each
// matrix) by 64 FN rows of x in four waves, each 32 FM by 32 FN of them in 32x32
// accumulators.  FM = FN = 4 is the largest wave tile that the registers hold
// (256 of sums): LDS is read (128 + 128) / (128 * 128) bytes for each product,
// half of what waves of 64x64 read.  LDS holds three blocks of W and two of x in
// turn.  A block's four matrix steps (32 columns each) read the fragments of the
// next step while they multiply, so the last step of a block reads the first of
// the next: the barrier that says that the next block is there, and that this one
// has been read, stands before it.  Its places are loaded over from there on, a
// part in every step so that no load waits for others to go out: x of the block
// after the next in that step and the one behind it, then W of the block after
// that.  SPLIT: a workgroup has a share of the blocks, and the sums go to
// partial[split][product][batch][rows].
// 8192x8192 at batch 4096 takes 205 to 221 us on different cards (2500 TOP/s and
// more; 427 with 64x64 tiles).  Where it took 219, the matrix instructions alone
// took 171 on random operands, 124 on zeros: the clock falls with their power; with
// the reads from LDS 176, with the loads 198.  The rest is a tile's ends: 3 us to
// its first block, 5 from its last to the last store, 3 of those for 256
// conversions a lane.
template <int FM, int FN>
struct Large {
    static constexpr int kW = 64 * FM * kBlock, kX = 64 * FN * kBlock;
    static constexpr size_t kLds = 3 * kW + 2 * kX;
    static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};
constexpr int large_per_unit(int FM, int FN) { return FM * FN <= 4 ? 2 : 1; } // workgroups of a compute unit

// The swizzle here: a fragment read takes one piece of 32 rows, in two phases
// (rows 0-3, 12-15, 20-27 and the rest); within each, row % 2 and this number
// put the sixteen rows into the sixteen places of 16 bytes that the 64 banks
// have.
__device__ __forceinline__ int turn(int row) { return ((row >> 1) & 3) | ((row >> 4) & 1) << 2; }

template <bool GLU, bool SPLIT, int FM, int FN>
__device__ __forceinline__ void large_tile(const Operands &p, int splits, int *partial, int r0, int b0)
{
    using L = Large<FM, FN>;
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, half = lane >> 5;
    const int share = SPLIT ? (p.blocks + splits - 1) / splits : p.blocks; // (the host leaves no split empty)
    const int k0 = SPLIT ? blockIdx.y * share : 0, k1 = SPLIT ? min(k0 + share, p.blocks) : p.blocks;
    const uint32_t ld = (uint32_t)p.blocks * kBlock;
    // this wave's loads of a block: rows 16 FM w and on of W (gated: of one
    // matrix), 16 FN w and on of x, eight a load.  Offsets fit 32 bits (256 rows
    // of at most 2^17 columns).
    const int8_t *const wsrc = p.wq[GLU ? w & 1 : 0] + (int64_t)r0 * ld, *const xsrc = p.xq + (int64_t)b0 * ld;
    uint32_t wfrom[2 * FM], xfrom[2 * FN];
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i) { // rows past the end: copies of the last
        const int row = (GLU ? w >> 1 : w) * 16 * FM + i * 8 + (lane >> 3), place = w * 16 * FM + i * 8 + (lane >> 3);
        wfrom[i] = (uint32_t)min(row, p.rows - 1 - r0) * ld + ((lane & 7) ^ turn(place)) * 16;
    }
#pragma unroll
    for (int i = 0; i < 2 * FN; ++i) {
        const int row = w * 16 * FN + i * 8 + (lane >> 3);
        xfrom[i] = (uint32_t)min(row, p.batch - 1 - b0) * ld + ((lane & 7) ^ turn(row)) * 16;
    }
    int8_t *const xlds = lds + 3 * L::kW;
    auto load_w = [&](int i, int k, int slot) {
        lds_load16(wsrc + (uint32_t)min(k, k1 - 1) * kBlock + wfrom[i], lds + slot * L::kW + (w * 2 * FM + i) * 1024);
    };
    auto load_x = [&](int i, int k, int slot) {
        lds_load16(xsrc + (uint32_t)min(k, k1 - 1) * kBlock + xfrom[i], xlds + slot * L::kX + (w * 2 * FN + i) * 1024);
    };
    const int wm = (w & 1) * 32 * FM, wn = (w >> 1) * 32 * FN;
    // the scales of this wave's rows, FM / 2 W rows (gated: of both matrices) and
    // FN of x a lane
    float ws[FM / 2], xs[FN];
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) {
        const int row = lane + 64 * i, second = GLU && row >= 16 * FM;
        ws[i] = p.wscale[second][min(r0 + (GLU ? wm / 2 : wm) + row - second * 16 * FM, p.rows - 1)];
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) xs[j] = p.xscale[min(b0 + wn + 32 * j + n, p.batch - 1)];
    i32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x16{};
    // this lane's piece of matrix step q: 2 q + half, at its swizzled place
    int at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = n * kBlock + (((2 * q + half) ^ turn(n)) * 16);
    i32x4 a[2][FM], b[2][FN];
    // fragment r of a step: those of x first
    auto read = [&](int to, int r, int q, int wslot, int xslot) {
        if (r < FN)
            b[to][r] = *(const i32x4 *)(xlds + (xslot * L::kX + wn * kBlock + at[q]) + 32 * r * kBlock);
        else
            a[to][r - FN] = *(const i32x4 *)(lds + (wslot * L::kW + wm * kBlock + at[q]) + 32 * (r - FN) * kBlock);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 2 * FM; ++i) load_w(i, k0 + k, k);
#pragma unroll
        for (int i = 0; i < (k == 0 ? 2 * FN : FN); ++i) load_x(i, k0 + k, k);
    }
    stage_barrier<2 * FM + FN>();
#pragma unroll
    for (int r = 0; r < FM + FN; ++r) read(0, r, 0, 0, 0);
    int wslot = 0, xslot = 0; // of block k
    for (int k = k0; k < k1; ++k) {
        const int wnext = wslot == 2 ? 0 : wslot + 1, wfree = wnext == 2 ? 0 : wnext + 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q == 3) stage_barrier<2 * FM>(); // all but W of block k + 2 is there, block k has been read
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < FM * FN; ++m) {
                const int i = m / FN, j = m % FN;
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[q & 1][i], b[q & 1][j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                // a read of the next step, and a load now and then
                if (m < FM + FN) read((q + 1) & 1, m, (q + 1) & 3, q == 3 ? wnext : wslot, q == 3 ? xslot ^ 1 : xslot);
                if ((q & 1 ? q == 3 : q == 0) && m % FM == FM - 1) {
                    if (q == 3)
                        load_x(m / FM, k + 2, xslot);
                    else
                        load_x(FN + m / FM, k + 1, xslot ^ 1);
                }
                if ((q == 1 || q == 2) && m % FN == FN - 1) load_w((q - 1) * FM + m / FN, k + 2, wfree);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        wslot = wnext, xslot ^= 1;
    }
    wait_loads<0>(); // none may land after the workgroup's LDS is someone else's
    constexpr int FR = GLU ? FM / 2 : FM, kOut = FR * 32; // columns of y of this wave
    const int rw = r0 + (GLU ? wm / 2 : wm);
    if constexpr (SPLIT) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    auto four = [&](const i32x16 &v) { return i32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]}; };
                    store_partial<GLU>(p, partial, b0 + wn + 32 * j + n, rw + 32 * i + 8 * g + 4 * half, four(acc[i][j]),
                                       four(acc[GLU ? i + FR : i][j]));
                }
        return;
    }
    // The sums leave through LDS: a lane holds four rows of y's columns for one of
    // its rows, and stores of those would touch 64 lines each.  Every wave has its
    // own part: a row of x in 2 kOut bytes, in pieces of 8 bytes at piece ^
    // 2 (row % 16), which keeps pairs of them together.
    asm volatile("s_barrier" ::: "memory"); // the blocks are done with, and no load is on its way into them
    int8_t *const own = lds + w * (32 * FN * 2 * kOut);
    float *const wsc = (float *)(lds + 4 * (32 * FN * 2 * kOut)) + w * 32 * FM;
    static_assert(4 * 32 * FN * 2 * 32 * FM + 4 * 4 * 32 * FM <= L::kLds, "room for both");
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) wsc[64 * i + lane] = ws[i];
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int r = 32 * i + 8 * g + 4 * half;
            const f32x4 s0 = *(const f32x4 *)(wsc + r);
            f32x4 s1 = s0;
            if constexpr (GLU) s1 = *(const f32x4 *)(wsc + 16 * FM + r);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
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
    const int c = lane % kLanes, r = rw + 8 * c;
#pragma unroll 4
    for (int k = 0; k < 32 * FN * kLanes / 64; ++k) {
        const int row = k * (64 / kLanes) + lane / kLanes, b = b0 + wn + row;
        const u32x4 v = *(const u32x4 *)(own + row * (2 * kOut) + ((2 * c) ^ ((2 * row) & (kOut / 4 - 1) & 30)) * 8);
        if (b >= p.batch || r >= p.rows) continue;
        uint16_t *const y = p.y + (int64_t)b * p.rows + r;
        if (r + 8 <= p.rows) {
            *(u32x4_any *)y = v;
            continue;
        }
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r + e < p.rows) y[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
    }
}

template <bool GLU, bool SPLIT, int FM, int FN>
__global__ void __launch_bounds__(256, large_per_unit(FM, FN)) gemm_large(Operands p, int splits, int *partial)
{
    int r0, b0;
    if (tile_of<GLU ? 32 * FM : 64 * FM, 64 * FN>(p, blockIdx.x, 0, 0, false, r0, b0))
        large_tile<GLU, SPLIT, FM, FN>(p, splits, partial, r0, b0);
}

// Whole rounds of 256x256 tiles, and what is left of them in halves: those begin
// on each compute unit as soon as it is done with its last whole one.
template <bool GLU>
__global__ void __launch_bounds__(256, 1) gemm_large_halves(Operands p, int whole)
{
    constexpr int kRows = GLU ? 128 : 256;
    int r0, b0;
    if ((int)blockIdx.x < whole) {
        if (tile_of<kRows, 256>(p, blockIdx.x, 0, whole, false, r0, b0)) large_tile<GLU, false, 4, 4>(p, 1, nullptr, r0, b0);
    } else {
        if (tile_of<kRows, 128>(p, blockIdx.x - whole, whole, 0, true, r0, b0)) large_tile<GLU, false, 4, 2>(p, 1, nullptr, r0, b0);
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
// Memory bounds it: 8192x22016 at one row 28.4 us (6.4 TB/s), 8192x8192 11.8, gate
// and up of 11008x4096 16.0 and of 22016x8192 55 (6.5 TB/s); tiles took 46, 21 and
// 27.  From matrices that were not read just before, on another card, 35.1 (x in
// fp16 33.2), 14.5 and 19.1.
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
// 8192x8192 at 16 rows takes 16.5 us from memory (12.4 of a matrix that is in the
// 256 MB cache), at one in the form above 11.8: every workgroup reads x first, 33 MB in all out of the second-level caches, and that
// is 3 us before W comes at its rate.  W through registers into LDS in half
// kilobytes of a row took 17.5, x through the ring in turn with the first blocks
// 16.3 and more registers, W asked for before x 16.8 to 17.8.
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

// y from the splits' sums, four rows a thread.
template <bool GLU>
__global__ void __launch_bounds__(256) add_splits(Operands p, const int *partial, int splits)
{
    const int64_t pitch = partial_pitch(p.rows), size = p.batch * pitch;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < size; i += (int64_t)gridDim.x * 1024) {
        i32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
        for (int s = 0; s < splits; ++s) {
            g += *(const i32x4 *)(partial + s * (GLU ? 2 : 1) * size + i);
            if constexpr (GLU) u += *(const i32x4 *)(partial + (2 * s + 1) * size + i);
        }
        const int b = (int)(i / pitch);
        finish4<GLU>(p, b, (int)(i - b * pitch), g, u);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 28; // the work-items of every launch fit 32 bits

bool good_sizes(int64_t rows, int64_t cols, int64_t batch)
{
    return rows >= 1 && rows <= kMaxRows && batch >= 1 && batch <= kMaxRows && sqllm_int8_cols(cols) > 0 &&
           rows * batch <= (int64_t)1 << 38;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Tiled forms: rows of W (gated: of both matrices) and of x, the time of a block
// of 128 columns in us where every compute unit has one workgroup and where it
// has two, and whether it has those at once (else one after the other).  Measured on
// 8192x8192, 64 blocks a tile, at 256 and 512 tiles: 256x256 at batch 2048 118 us
// and at 4096 219; 256x128 at 1024 67, at 2048 132; 128x128 at 512 45, at 1024
// 73; 128x64 at 256 36, at 512 67; 64x64 at 128 25.5, at 256 40; 64x32 at 64
// 19.5, at 128 31.0.  A tile's ends (its first loads, the sums' way out; 10 us of
// a round of 256x256) are in these times as parts of its blocks: where columns are
// few, large tiles take longer than the rule thinks (8192x256 at batch 4096, two
// rounds of two blocks, 27 us for 6.7; 8192x768 40 for 20).
enum Tile { k256x256, k256x128, k128x128, k128x64, k64x64, k64x32, kTiles, k32x16 = kTiles, k32x16x4, k32x32, k32x64, k64x64x3 };
constexpr struct {
    int tm, tn;
    double one, two;
    bool pairs;
} kTile[kTiles] = {{256, 256, 1.68, 3.36, false}, {256, 128, 0.96, 1.92, false}, {128, 128, 0.66, 1.06, true},
                   {128, 64, 0.48, 0.96, false},  {64, 64, 0.34, 0.53, true},    {64, 32, 0.28, 0.42, true}};

// How a product is tiled: what these times make least.  Splitting the columns
// costs a launch (5.5 us) and the sums' way through memory (4 TB/s); what is
// left after whole rounds of 256x256 tiles goes in halves where that is half a
// round or less (gated 13824x5120 at batch 2048, 864 tiles: 262 us, 275 without;
// 5120x5120 at 8192, 640: 188 and 200).  What it weighs, in us at one, two and four
// splits: 8192x8192 at batch 17 64x32 18.2, 19.8, 17.6; at 64 128x64 34, 25, 20.5,
// 64x64 24, 22, 21, 64x32 19.5, 23, 25; at 128 64x64 25.5, 30, 32; at 256 128x64 36, 44, 55, 128x128
// 41, 37, 40; at 512 128x128 45, 58, 73, 256x128 59, 53; 4096x4096 at 32 64x32
// 10.1, 10.0, 9.7; at 128 64x32 10.4, 14, 17, 64x64 13.5, 13.4, 17; at 256 64x64
// 13.6, 20, 23, 128x64 19.5, 19, 21; at 512 128x64 20.5, 29, 128x128 23, 24, 28;
// at 1024 128x128 24.5, 37, 256x128 32, 36.
struct Choice {
    int tile, splits;
    int whole; // 256x256 tiles before the halves, 0: no halves
};

// First, the smallest unsplit tiles of which every compute unit has one at most
// (with more they are slower: 32x32, 11008x4096 at batch 32, 344 tiles, 15.6 us, 64x32
// 13.1).  us, and what the rest of the rule gives: 32x16 4096x4096 at 17 7.0 and 9.5,
// 1024x4096 at 128 6.4 and 8.8, gated at 32 5.7 and 8.8; 32x32 4096x4096 at 64 8.8
// and 10.8, 8192x8192 at 17 15.0 and 17.4, gated 4096x4096 at 32 9.8 and 11.6; 32x64
// 5001x4999 at 40 12.5 and 15.9, 1024x8192 at 400 13.3 and 15.5; 64x64 5001x4999 at
// 128 18.6 and 21.2.  Not where splits of the columns, or two workgroups a unit with
// one group of waves each, are better: 512x13824 at 77, 96 tiles of 32x32, 12.3 and
// 10.6; 8192x22016 at 32 41.8 and 40.3; 32x64, 2000x13824 at 256 25.3 and 22.1; 64x64,
// 3000x1024 at 200 6.6 and 5.8.
Choice choose(int64_t rows, int64_t cols, int64_t batch, bool glu)
{
    const int64_t blocks = sqllm_int8_cols(cols) / kBlock, m = glu ? 2 : 1;
    Choice best = {k256x256, 1, 0};
    double least = 1e30;
    auto tiles = [&](int64_t tm, int64_t tn) { return (rows * m + tm - 1) / tm * ((batch + tn - 1) / tn); };
    auto fits = [&](int64_t n) { return n <= 256 && (blocks <= 64 || (blocks <= 128 && n > 128)); };
    if (fits(tiles(32, 16))) return {tiles(32, 16) <= 128 ? k32x16x4 : k32x16, 1, 0};
    if (fits(tiles(32, 32))) return {k32x32, 1, 0};
    if (blocks <= 64) {
        if (blocks >= 16 && tiles(32, 64) <= 256) return {k32x64, 1, 0};
        if (tiles(64, 32) <= 256) return {k64x32, 1, 0};
        if (blocks > 32 && tiles(64, 64) <= 256) return {k64x64x3, 1, 0};
    }
    for (int t = 0; t < kTiles; ++t) {
        const int64_t of = tiles(kTile[t].tm, kTile[t].tn);
        for (int64_t s = 1; s <= 8 && (s == 1 || (t > k256x256 && blocks >= 8 * s)); s *= 2) {
            const int64_t share = (blocks + s - 1) / s, splits = (blocks + share - 1) / share; // none empty
            const int64_t wgs = of * splits, pairs = wgs / 512, rest = wgs % 512;
            double last = rest > 256 ? kTile[t].two : rest ? kTile[t].one : 0;
            if (rest > 256 && kTile[t].pairs) // some units have one: the loads of the others go faster
                last = kTile[t].one + (kTile[t].two - kTile[t].one) * (rest - 256) / 256;
            double us = share * (pairs * kTile[t].two + last);
            if (splits > 1) us += 5.5 + 2e-6 * splits * batch * rows * m;
            if (us < least) least = us, best = {t, (int)splits, 0};
            const int64_t over = wgs % 256;
            if (t == k256x256 && wgs > 256 && over && over <= 128) {
                us = share * (wgs / 256 * kTile[t].one + kTile[k256x128].one);
                if (us < least) least = us, best = {t, 1, (int)(wgs - over)};
            }
        }
    }
    return best;
}

// The streaming form in the vector units, up to four rows of x: beyond, its
// instructions and the sums' reduction outlast the loads (8192x8192 at four and
// eight rows 13.0 and 18.7 us, the matrix cores' form 16.4 at both; gated
// 11008x4096 18.1 and 24.9, 20.2).  Chunks a wave: few, so that waves are many
// and each has little to add up.  us at one row with 1 and 2 chunks a wave:
// 8192x8192 11.8, 12.0; 5120x5120 6.7, 7.2; with 2 and 3: 8192x22016 29.8, 28.2,
// 4096x11008 10.6, 10.2.
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

int dot_rows(int64_t batch) { return batch > 2 ? 4 : (int)batch; } // rows of x that it is built for

// Whether it rounds x in fp16 itself, which takes registers; those that would
// spill are given rounded x, a launch more.  us inside and after the quantiser:
// 8192x22016, one row 33.2 and 38.1, two 35.7 and 38.7; spilling: at four rows 79
// and 41; gated at two, 12 registers, 512x16500 11.8 and 9.3, 1024x17000 17.1 and
// 12.0, 8192x22016 73.7 and 70.6, 8192x49152 146 and 142, but 8192x16500 55.0 and
// 57.1, 28000x17000 163 and 165.
constexpr bool rounds_inside(bool glu, int held, int chunks)
{
    return chunks == 1 || held == 1 || (held == 2 && (chunks == 2 || !glu));
}

// How a product is computed.  The form on the matrix cores takes up to sixteen
// rows of x whatever W is, one workgroup to 16 rows of W: 8192x8192 at 16 and, in
// tiles, at 17 rows 16.8 and 18.2 us, 1024x8192 7.6 and 7.6, but where rows are
// few and long, split tiles are faster: 256x24576 at 5, 16 and 17 11.0, 16.8 and
// 11.4, 512x16384 8.4, 12.2 and 10.0, 1024x24576 15.7, 21.9 and 13.5.
struct Plan {
    Dot dot;      // the streaming form in the vector units, if it takes the product
    bool inside;  // which rounds x in fp16 itself
    int few;      // else blocks a wave of the one on the matrix cores, 0: not this form
    Choice tiles; // else
};

Plan plan_of(int64_t rows, int64_t cols, int64_t batch, bool glu, bool stored)
{
    const int64_t ld = sqllm_int8_cols(cols), blocks = ld / kBlock;
    Plan p = {dot_shape(ld, batch), false, 0, {k256x256, 1, 0}};
    if (p.dot.waves)
        p.inside = !stored && rounds_inside(glu, dot_rows(batch), p.dot.chunks);
    else if (batch <= 16 && blocks <= 192) // (however few units it fills)
        p.few = blocks <= 32 ? 2 : blocks <= 64 ? 4 : blocks <= 128 ? 8 : 16;
    else
        p.tiles = choose(rows, cols, batch, glu);
    return p;
}

// Scratch of a product: x in integers, unless it comes so, and the sums of splits.
struct Scratch {
    size_t codes, scales, sums;
    size_t bytes() const { return std::max<size_t>(codes + scales + sums, 256); } // (0 says that sizes are out of range)
};

Scratch scratch_of(const Plan &p, int64_t rows, int64_t cols, int64_t batch, bool glu, bool stored)
{
    const int splits = p.tiles.splits;
    return {stored ? 0 : up256((size_t)batch * sqllm_int8_cols(cols)), stored ? 0 : up256((size_t)batch * 4),
            splits > 1 ? (size_t)splits * batch * partial_pitch(rows) * (glu ? 8 : 4) : 0};
}

size_t workspace_bytes(int64_t rows, int64_t cols, int64_t batch, bool glu, bool stored)
{
    if (!good_sizes(rows, cols, batch)) return 0;
    return scratch_of(plan_of(rows, cols, batch, glu, stored), rows, cols, batch, glu, stored).bytes();
}

template <bool GLU>
void launch_add(const Operands &p, int splits, const int *partial, hipStream_t stream)
{
    const int64_t wgs = (p.batch * partial_pitch(p.rows) + 1023) / 1024;
    hipLaunchKernelGGL(add_splits<GLU>, dim3((unsigned)std::min<int64_t>(wgs, 4096)), dim3(256), 0, stream, p, partial,
                       splits);
}

template <bool GLU, int TM, int TN, int WM, int WN, int S, int G>
void launch_tiled(const Operands &p, int splits, int *partial, hipStream_t stream)
{
    using T = Tiling<TM, TN, WM, WN, S, G>;
    auto kern = gemm_tiled<GLU, TM, TN, WM, WN, S, G>;
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)kern, asked, (int)T::kLds);
    constexpr int kRows = GLU ? TM / 2 : TM;
    const int64_t tiles = (int64_t)((p.rows + kRows - 1) / kRows) * ((p.batch + TN - 1) / TN);
    hipLaunchKernelGGL(kern, dim3((unsigned)((tiles + 7) / 8 * 8), splits), dim3(64 * T::W * G), T::kLds, stream, p, splits,
                       partial);
    if (splits > 1) launch_add<GLU>(p, splits, partial, stream);
}

template <bool GLU, bool HALF, int B, int C, int R>
void launch_dot(const Operands &p, const uint16_t *x, int cols, int waves, hipStream_t stream)
{
    const int groups = (p.rows + R - 1) / R;
    int wgs = 256 * (16 / waves);
    if (wgs > groups) wgs = groups;
    hipLaunchKernelGGL((gemm_dot<GLU, HALF, B, C, R>), dim3(wgs), dim3(64 * waves), 0, stream, p, x, cols, groups);
}

// Rows of a group.  us at one row with 2, 4 and 8: 8192x8192, one chunk a wave,
// 12.1, 11.8, 12.4; at four rows 15.7, 14.9, 16.2; 8192x22016, three chunks, 28.2
// and 29.3 with 2 and 4.
template <bool GLU, bool HALF, int B>
void launch_dots(const Operands &p, const uint16_t *x, int cols, Dot d, hipStream_t stream)
{
    if (d.chunks == 1) launch_dot<GLU, HALF, B, 1, 4>(p, x, cols, d.waves, stream);
    if constexpr (!HALF || rounds_inside(GLU, B, 2))
        if (d.chunks == 2) launch_dot<GLU, HALF, B, 2, B == 1 ? 4 : 2>(p, x, cols, d.waves, stream);
    if constexpr (!HALF || rounds_inside(GLU, B, 3))
        if (d.chunks == 3) launch_dot<GLU, HALF, B, 3, 2>(p, x, cols, d.waves, stream);
}

template <bool GLU, bool HALF>
void launch_dots(const Operands &p, const uint16_t *x, int cols, Dot d, hipStream_t stream)
{
    const int held = dot_rows(p.batch);
    if (held == 1)
        launch_dots<GLU, HALF, 1>(p, x, cols, d, stream);
    else if (held == 2)
        launch_dots<GLU, HALF, 2>(p, x, cols, d, stream);
    else
        launch_dots<GLU, HALF, 4>(p, x, cols, d, stream);
}

// Blocks a wave and ring, us at 16 rows.  8192x8192: 4 blocks, ring of 2 16.3, of
// 4 16.5, 8 blocks, 8 17.3, 4 18.8, 16 blocks 23.8; 4096x4096: 2 blocks 6.6, 4
// 7.0, 8 7.3; gated 11008x4096: 18.1, 20.2, 22.1.  Gated with 16 blocks a wave it
// spills ten registers, which do not show: 8192x24576 94 to 96, ungated 50.
template <bool GLU, int S, int D>
void launch_few(const Operands &p, hipStream_t stream)
{
    static std::atomic<uint64_t> asked{0};
    sqllm::dev::raise_lds_limit((const void *)gemm_few<GLU, S, D>, asked, 160 * 1024);
    const int groups = (p.rows + 15) / 16, waves = (p.blocks + S - 1) / S, lds = waves * (D * 2048 + 2 * 1024);
    const int wgs = std::min(groups, 256 * std::max(1, std::min(16 / waves, 160 * 1024 / lds)));
    hipLaunchKernelGGL((gemm_few<GLU, S, D>), dim3(wgs), dim3(64 * waves), lds, stream, p, groups);
}

template <bool GLU, int FM, int FN>
void launch_large(const Operands &p, int splits, int *partial, hipStream_t stream)
{
    using L = Large<FM, FN>;
    auto kern = gemm_large<GLU, false, FM, FN>;
    if constexpr (FM * FN < 16)
        if (splits > 1) kern = gemm_large<GLU, true, FM, FN>;
    static std::atomic<uint64_t> asked[2] = {};
    sqllm::dev::raise_lds_limit((const void *)kern, asked[splits > 1], (int)L::kLds);
    constexpr int kRows = GLU ? 32 * FM : 64 * FM;
    const int64_t tiles = (int64_t)((p.rows + kRows - 1) / kRows) * ((p.batch + 64 * FN - 1) / (64 * FN));
    hipLaunchKernelGGL(kern, dim3((unsigned)((tiles + 7) / 8 * 8), splits), dim3(256), L::kLds, stream, p, splits, partial);
    if (splits > 1) launch_add<GLU>(p, splits, partial, stream);
}

template <bool GLU>
void launch_halves(const Operands &p, int whole, hipStream_t stream)
{
    static std::atomic<uint64_t> asked{0};
    constexpr int kLds = Large<4, 4>::kLds, kRows = GLU ? 128 : 256;
    sqllm::dev::raise_lds_limit((const void *)gemm_large_halves<GLU>, asked, kLds);
    const int64_t tiles = (int64_t)((p.rows + kRows - 1) / kRows) * ((p.batch + 255) / 256);
    const int64_t wgs = whole + ((tiles - whole) * 2 + 7) / 8 * 8;
    hipLaunchKernelGGL(gemm_large_halves<GLU>, dim3((unsigned)wgs), dim3(256), kLds, stream, p, whole);
}

template <bool GLU>
void launch_choice(const Choice &c, const Operands &p, int *partial, hipStream_t stream)
{
    if (c.tile == k256x256 && c.whole) {
        launch_halves<GLU>(p, c.whole, stream);
    } else if (c.tile == k256x256) {
        launch_large<GLU, 4, 4>(p, 1, partial, stream);
    } else if (c.tile == k256x128) {
        launch_large<GLU, 4, 2>(p, c.splits, partial, stream);
    } else if (c.tile == k128x128) {
        launch_large<GLU, 2, 2>(p, c.splits, partial, stream);
    } else if (c.tile == k128x64) {
        launch_tiled<GLU, 128, 64, 32, 64, 4, 1>(p, c.splits, partial, stream);
    } else if (c.tile == k64x64) {
        launch_tiled<GLU, 64, 64, 32, 32, 4, 1>(p, c.splits, partial, stream);
    } else if (c.tile == k64x32) {
        launch_tiled<GLU, 64, 32, 32, 16, 5, 1>(p, c.splits, partial, stream);
    } else if (c.tile == k64x64x3) {
        launch_tiled<GLU, 64, 64, 32, 32, 3, 3>(p, 1, nullptr, stream);
    } else if (c.tile == k32x64) {
        launch_tiled<GLU, 32, 64, 32, 16, 4, 2>(p, 1, nullptr, stream);
    } else if (c.tile == k32x32) {
        launch_tiled<GLU, 32, 32, 32, 16, 5, 2>(p, 1, nullptr, stream);
    } else if (c.tile == k32x16) {
        launch_tiled<GLU, 32, 16, 32, 16, 6, 2>(p, 1, nullptr, stream);
    } else {
        launch_tiled<GLU, 32, 16, 32, 16, 5, 4>(p, 1, nullptr, stream);
    }
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
    const bool stored = xscale != nullptr;
    const Plan plan = plan_of(rows, cols, batch, GLU, stored);
    const Scratch scratch = scratch_of(plan, rows, cols, batch, GLU, stored);
    if (!workspace || !aligned(workspace, 256) || workspace_size < scratch.bytes()) return SQLLM_ERR_WORKSPACE;
    const int64_t ld = sqllm_int8_cols(cols);
    int8_t *const xq = (int8_t *)workspace;
    float *const xs = (float *)(xq + scratch.codes);
    int *const partial = (int *)((uint8_t *)xs + scratch.scales);
    Operands p = {{q[0], q[1]}, {scale[0], scale[1]}, (const int8_t *)x, xscale, y, (int)rows, (int)batch, (int)(ld / kBlock)};
    if (plan.inside) {
        launch_dots<GLU, true>(p, (const uint16_t *)x, (int)cols, plan.dot, stream);
        return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
    }
    if (!stored) {
        if (sqllm::launch_int8_quantize((const uint16_t *)x, batch, cols, cols, xq, xs, stream) != hipSuccess)
            return SQLLM_ERR_HIP;
        p.xq = xq, p.xscale = xs;
    }
    if (plan.dot.waves)
        launch_dots<GLU, false>(p, nullptr, (int)cols, plan.dot, stream);
    else if (plan.few == 2)
        launch_few<GLU, 2, 2>(p, stream);
    else if (plan.few == 4)
        launch_few<GLU, 4, 2>(p, stream);
    else if (plan.few == 8)
        launch_few<GLU, 8, 4>(p, stream);
    else if (plan.few == 16)
        launch_few<GLU, 16, 4>(p, stream);
    else
        launch_choice<GLU>(plan.tiles, p, partial, stream);
    return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP;
}

} // namespace

extern "C" size_t sqllm_int8_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, false, false);
}

extern "C" size_t sqllm_int8_glu_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, true, false);
}

extern "C" size_t sqllm_int8_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, false, true);
}

extern "C" size_t sqllm_int8_glu_stored_workspace_bytes(int64_t rows, int64_t cols, int64_t batch)
{
    return workspace_bytes(rows, cols, batch, true, true);
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

extern "C" sqllm_status sqllm_test_int8_plan(int64_t rows, int64_t cols, int64_t batch, int gated, int stored, int *plan)
{
    if (!plan) return SQLLM_ERR_NULL;
    if (!good_sizes(rows, cols, batch)) return SQLLM_ERR_SHAPE;
    const Plan p = plan_of(rows, cols, batch, gated != 0, stored != 0);
    plan[0] = !stored && !p.inside;
    plan[1] = p.dot.waves ? 0 : p.few ? 1 : 2;
    plan[2] = p.dot.waves ? dot_rows(batch) : p.few ? p.few : p.tiles.tile;
    plan[3] = p.dot.waves ? p.dot.chunks : p.few ? 0 : p.tiles.splits;
    plan[4] = p.dot.waves || p.few ? 0 : p.tiles.whole;
    return SQLLM_OK;
}
