// sqllm_moe.hip -- the mixture-of-experts layer of include/sqllm_moe.h:
// argument checks, workspace layout, kernels and launches.
//
// One call is a chain of small launches on the caller's stream: the router's
// sums and choice, gate and up with the activation, down, and the weighted
// sum over a token's experts.  Nothing is read back by the host: every
// workgroup finds its expert and tokens from ids[] itself.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "sqllm_device.h"
#include "sqllm_internal.h"
#include "sqllm_moe.h"

using namespace sqllm;

namespace {

constexpr int kMaxExperts = SQLLM_MOE_MAX_EXPERTS;
constexpr int kMaxTopk = SQLLM_MOE_MAX_TOPK;
constexpr int kLogWaves = 3;
static_assert(kDefaultWaves == 1 << kLogWaves);
constexpr int64_t kMaxWidth = 65536; // hidden, inter: 16-bit columns of the outliers

// ---------------------------------------------------------------------------
// Router.
// ---------------------------------------------------------------------------

// Sums in 64 bits: a product of two fp16 values is exact in fp32, and 64-bit
// sums of at most 2^16 of them are off by less than 2^-37 of the largest
// partial sum, so the choice does not depend on the order they are taken in.

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

// This lane's part of the sums of R router rows with T tokens' x: 16 bytes of
// each per 512 columns (hidden is a multiple of 256: the last 512 may be half
// there).
template <int R, int T>
__device__ __forceinline__ void row_sums(const uint16_t *const (&w)[R], const uint16_t *const (&x)[T], int hidden,
                                         int lane, double (&sum)[R][T])
{
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) sum[r][t] = 0.0;
    constexpr int kAtOnce = R * T > 1 ? 2 : 4;
#pragma unroll kAtOnce
    for (int c = lane * 8; c < hidden; c += 512) {
        half8_t wv[R], xv[T];
#pragma unroll
        for (int r = 0; r < R; ++r) wv[r] = *(const half8_t *)(w[r] + c);
#pragma unroll
        for (int t = 0; t < T; ++t) xv[t] = *(const half8_t *)(x[t] + c);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[r][t] += (double)((float)wv[r][i] * (float)xv[t][i]);
    }
}

// v of lane l - N of the same row of 16, or of the last lane of the rows before
// (DPP row_shr, row_bcast); 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_double(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, true);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// The sum over the wave's lanes, in every lane: a prefix sum by DPP shifts
// within rows of 16 and broadcasts across them, of which lane 63 has the last.
__device__ __forceinline__ double wave_sum(double v)
{
    v += dpp_double<0x111, 0xF>(v); // row_shr 1, 2, 4, 8
    v += dpp_double<0x112, 0xF>(v);
    v += dpp_double<0x114, 0xF>(v);
    v += dpp_double<0x118, 0xF>(v);
    v += dpp_double<0x142, 0xA>(v); // row_bcast 15, 31
    v += dpp_double<0x143, 0xC>(v);
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, 63), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), 63);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// A double's place in ascending order as an unsigned number; NaN is 0, below
// -infinity, and -0 counts as +0.
__device__ __forceinline__ uint64_t order_key(double v)
{
    if (v != v) return 0;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// The largest v of the wave, in every lane: DPP shifts within rows of 16 and
// broadcasts across them leave it in lane 63.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#define SQLLM_MAX_STEP(ctrl, rows) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, true))
    SQLLM_MAX_STEP(0x111, 0xF); // row_shr 1, 2, 4, 8
    SQLLM_MAX_STEP(0x112, 0xF);
    SQLLM_MAX_STEP(0x114, 0xF);
    SQLLM_MAX_STEP(0x118, 0xF);
    SQLLM_MAX_STEP(0x142, 0xA); // row_bcast 15, 31
    SQLLM_MAX_STEP(0x143, 0xC);
#undef SQLLM_MAX_STEP
    return __builtin_amdgcn_readlane(v, 63);
}

// The bits of all lanes' v, in every lane: the same.
__device__ __forceinline__ uint32_t wave_or(uint32_t v)
{
#define SQLLM_OR_STEP(ctrl, rows) v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, true)
    SQLLM_OR_STEP(0x111, 0xF); // row_shr 1, 2, 4, 8
    SQLLM_OR_STEP(0x112, 0xF);
    SQLLM_OR_STEP(0x114, 0xF);
    SQLLM_OR_STEP(0x118, 0xF);
    SQLLM_OR_STEP(0x142, 0xA); // row_bcast 15, 31
    SQLLM_OR_STEP(0x143, 0xC);
#undef SQLLM_OR_STEP
    return __builtin_amdgcn_readlane(v, 63);
}

// One wave's choice for one token; lane l holds experts l, l + 64, ... (N of
// them; logit(e) is expert e's sum).  Each of the topk rounds takes the
// largest key left, by its upper and then its lower half (ties: the lowest
// expert).
template <int N, typename L>
__device__ __forceinline__ void choose(L logit, const float *bias, int experts, int topk, int flags, float scale,
                                       int32_t *ids, float *weights)
{
    const int lane = threadIdx.x & 63;
    double s[N];
    uint64_t key[N];
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = lane + 64 * j < experts ? logit(lane + 64 * j) : -__builtin_inf();
    if (flags & SQLLM_MOE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = 1.0 / (1.0 + exp(-s[j]));
    } else {
        // the largest sum, exactly: its key's upper half, then the lower one among
        // those (the upper half alone is off by up to 2^-20 of a sum, which from
        // 2^30 on takes exponentials out of range)
        uint64_t most = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) most = max(most, order_key(s[j]));
        const uint32_t hi = wave_max((uint32_t)(most >> 32));
        const uint32_t lo = wave_max((uint32_t)(most >> 32) == hi ? (uint32_t)most : 0);
        most = (uint64_t)hi << 32 | lo;
        const double top = __longlong_as_double((long long)(most >> 63 ? most ^ 0x8000000000000000ull : ~most));
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            s[j] = lane + 64 * j < experts ? exp(s[j] - top) : 0.0;
            sum += s[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] /= sum;
    }
    // bit j of left: expert lane + 64 j can still be chosen
    uint32_t left = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 64 * j;
        if (e < experts) left |= 1u << j;
        key[j] = e < experts ? order_key(bias ? s[j] + (double)bias[e] : s[j]) : 0;
    }
    double kept = 0.0, sum = 0.0; // lane k ends with the k-th score
    int mine = 0;
    for (int k = 0; k < topk; ++k) {
        uint64_t best = 0;
        int at = -1;
        double sc = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (((left >> j) & 1) && (at < 0 || key[j] > best)) best = key[j], at = j, sc = s[j];
        uint64_t with = __ballot(at >= 0);
        const uint32_t hi = wave_max(at >= 0 ? (uint32_t)(best >> 32) : 0);
        with &= __ballot((uint32_t)(best >> 32) == hi);
        if (with & (with - 1)) { // several: the lower half decides, then the lowest expert
            const bool in = (with >> lane) & 1;
            const uint32_t lo = wave_max(in ? (uint32_t)best : 0);
            with &= __ballot((uint32_t)best == lo);
            if (with & (with - 1)) {
                const uint32_t first = ~wave_max((with >> lane) & 1 ? ~(uint32_t)(lane + 64 * at) : 0);
                with = 1ull << (first & 63);
            }
        }
        const int owner = __builtin_ctzll(with), e = owner + 64 * __builtin_amdgcn_readlane(at, owner);
        const double got = __shfl(sc, owner);
        if (lane == owner) left &= ~(1u << at);
        if (lane == k) kept = got, mine = e;
        sum += got;
    }
    if (lane < topk) {
        ids[lane] = mine;
        // the quotient first: 1 / sum is infinite where all scores are tiny
        weights[lane] = (float)((flags & SQLLM_MOE_KEEP_SUM ? kept : kept / sum) * (double)scale);
    }
}

// Small routers in one launch: a workgroup of sixteen waves does all of one
// token.
constexpr int kRouteWaves = 16;

template <int N>
__global__ void __launch_bounds__(64 * kRouteWaves) route_small(const uint16_t *__restrict__ x,
                                                                const uint16_t *__restrict__ router,
                                                                const float *__restrict__ bias, int hidden, int experts,
                                                                int topk, int flags, float scale,
                                                                int32_t *__restrict__ ids, float *__restrict__ weights)
{
    __shared__ double logits[64 * N];
    const int t = blockIdx.x, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint16_t *const xt[1] = {x + (int64_t)t * hidden};
    constexpr int R = 4; // rows at a time, so that their loads and sums over the wave overlap
    for (int e = w * R; e < experts; e += kRouteWaves * R) {
        const uint16_t *row[R];
#pragma unroll
        for (int r = 0; r < R; ++r) row[r] = router + (int64_t)min(e + r, experts - 1) * hidden;
        double sum[R][1];
        row_sums(row, xt, hidden, lane, sum);
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r][0] = wave_sum(sum[r][0]);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane == 0 && e + r < experts) logits[e + r] = sum[r][0];
    }
    __syncthreads();
    if (w == 0)
        choose<N>([&](int e) { return logits[e]; }, bias, experts, topk, flags, scale, ids + t * topk, weights + t * topk);
}

// Larger ones in two: logits[t][e], a wave for one expert and T tokens, then
// the choice.
template <int T>
__global__ void __launch_bounds__(256) route_logits(const uint16_t *__restrict__ x, const uint16_t *__restrict__ router,
                                                    int hidden, int experts, int batch, double *__restrict__ logits)
{
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6), t0 = blockIdx.y * T, lane = threadIdx.x & 63;
    if (e >= experts) return;
    const uint16_t *xt[T];
#pragma unroll
    for (int t = 0; t < T; ++t) xt[t] = x + (int64_t)min(t0 + t, batch - 1) * hidden;
    const uint16_t *const row[1] = {router + (int64_t)e * hidden};
    double sum[1][T];
    row_sums(row, xt, hidden, lane, sum);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const double v = wave_sum(sum[0][t]);
        if (lane == 0 && t0 + t < batch) logits[(int64_t)(t0 + t) * experts + e] = v;
    }
}

template <int N>
__global__ void __launch_bounds__(64) route_choose(const double *__restrict__ logits, const float *__restrict__ bias,
                                                   int experts, int topk, int flags, float scale,
                                                   int32_t *__restrict__ ids, float *__restrict__ weights)
{
    const int t = blockIdx.x;
    choose<N>([&](int e) { return logits[(int64_t)t * experts + e]; }, bias, experts, topk, flags, scale, ids + t * topk,
              weights + t * topk);
}

// ---------------------------------------------------------------------------
// Experts.  A workgroup owns 64 rows (a tile of the packed layout, lane = row)
// of one expert in use and all the tokens that chose it; its waves share the
// columns in half groups of 128 and add up their fp32 sums in LDS.
//
// Two decodes.  Without a table in memory: a row's centroids stay in registers
// as bytes, the low bytes of the fp16 values in one set and the high bytes in
// another, and v_perm_b32 picks four of them at once by four codes.  Or with a
// table of pairs of centroids in LDS (below), which a workgroup has to write
// first; it pays where a tile has many columns, and the more the wider the
// codes (gate_by_table and down_by_table).
//
// Products: v_mfma_f32_4x4x4f16 with CBSZ = 4 multiplies each lane's own four
// weights (B: lane = row) by the four activations of four tokens that block
// ABID of lanes holds (A): register i of lane r ends with row r's sum for
// token i of the quad.
// ---------------------------------------------------------------------------

using dev::f32x4;
using dev::half4_t;
using dev::u32x2;
using dev::u32x4;

struct Projection {
    const uint8_t *packed;
    const uint16_t *lut;
    const int32_t *row_ptr;
    const uint16_t *col;
    const uint16_t *val;
    int64_t nnz;
};

// v_perm_b32: result byte k is byte sel[k] of lo (0..3) or hi (4..7); 8, 9, 10
// and 11 repeat the top bit of bytes 1 and 3 of lo and of hi.
__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }

// A row's centroids, split into low and high bytes, four to a register.
template <int BITS>
struct Table {
    static constexpr int N = BITS == 2 ? 1 : (1 << BITS) / 4;
    uint32_t lo[N], hi[N];

    __device__ __forceinline__ void load(const uint16_t *row)
    {
        uint32_t w[2 * N];
        if constexpr (BITS == 2) {
            const u32x2 v = *(const u32x2 *)row;
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int q = 0; q < N / 2; ++q) {
                const u32x4 v = ((const u32x4 *)row)[q];
                w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            lo[k] = perm(w[2 * k + 1], w[2 * k], 0x06040200);
            hi[k] = perm(w[2 * k + 1], w[2 * k], 0x07050301);
        }
    }

    // The centroids of four codes, one a byte of `sel` (the low three bits);
    // at 4 bits `upper` has 0xFF in the bytes of the codes from 8 on.
    __device__ __forceinline__ half4_t pick(uint32_t sel, uint32_t upper) const
    {
        uint32_t l, h;
        if constexpr (BITS == 2) {
            l = perm(lo[0], lo[0], sel);
            h = perm(hi[0], hi[0], sel);
        } else if constexpr (BITS == 3) {
            l = perm(lo[1], lo[0], sel);
            h = perm(hi[1], hi[0], sel);
        } else {
            const uint32_t l0 = perm(lo[1], lo[0], sel), l1 = perm(lo[3], lo[2], sel);
            const uint32_t h0 = perm(hi[1], hi[0], sel), h1 = perm(hi[3], hi[2], sel);
            l = (l1 & upper) | (l0 & ~upper);
            h = (h1 & upper) | (h0 & ~upper);
        }
        return __builtin_bit_cast(half4_t, u32x2{perm(h, l, 0x05010400), perm(h, l, 0x07030602)});
    }
};

// The codes of one half group (128 columns) of a lane's row, and the order in
// which its matrix steps take the columns.  A step takes four columns; steps
// 2n and 2n + 1 take the eight columns that lane block n holds of the
// activations:
//   3 and 4 bits: dword n holds columns 8n..8n+7 as four bytes of two codes;
//     step 2n takes the first codes (columns 0, 2, 4, 6), 2n + 1 the others.
//   2 bits: dword m holds columns 16m..16m+15 as four bytes of four codes;
//     step 4m + i takes columns i, 4 + i, 8 + i, 12 + i.
template <int BITS>
struct Half {
    uint32_t d[4 * BITS];

    __device__ __forceinline__ void load(const uint8_t *src) // src: this lane's bytes of the half group's first piece
    {
#pragma unroll
        for (int q = 0; q < BITS; ++q) {
            const u32x4 v = __builtin_nontemporal_load((const u32x4 *)(src + q * 1024));
            d[4 * q] = v.x, d[4 * q + 1] = v.y, d[4 * q + 2] = v.z, d[4 * q + 3] = v.w;
        }
    }

    // Four bytes of two codes: pairs 4n..4n+3 of the half group (3, 4 bits).
    template <int N>
    __device__ __forceinline__ uint32_t pairs() const
    {
        if constexpr (BITS == 4) return d[N];
        constexpr int u = 3 * (N / 4), q = N % 4;
        if constexpr (q < 3) return d[u + q];
        // the unit's last four pairs lie in the top two bits of its 12 bytes
        return ((d[u] >> 6) & 0x03030303) | ((d[u + 1] >> 4) & 0x0C0C0C0C) | ((d[u + 2] >> 2) & 0x30303030);
    }

    template <int STEP>
    __device__ __forceinline__ half4_t weights(const Table<BITS> &t) const
    {
        if constexpr (BITS == 2) {
            return t.pick((d[STEP / 4] >> (2 * (STEP % 4))) & 0x03030303, 0);
        } else {
            const uint32_t v = pairs<STEP / 2>();
            // the codes' bit 3 to every bit of their bytes: perm's selectors 8
            // to 11 repeat the top bit of the operands' bytes 1 and 3
            uint32_t upper = 0;
            if constexpr (BITS == 4) upper = STEP % 2 ? perm(v, v << 8, 0x0B090A08) : perm(v << 4, v << 12, 0x0B090A08);
            return t.pick((v >> (BITS * (STEP % 2))) & 0x07070707, upper);
        }
    }
};

// A half group's activations of a quad of tokens: lane 4n + i loads what
// token i has for steps 2n and 2n + 1 (at 2 bits the two lane blocks of 16
// columns load all of them), put into the order above when it is used.
template <int BITS>
struct QuadX {
    u32x4 raw[BITS == 2 ? 2 : 1];

    __device__ __forceinline__ void load(const uint16_t *x, int block) // x: the token's 128 columns
    {
        if constexpr (BITS == 2) {
            const u32x4 *p = (const u32x4 *)(x + 16 * (block >> 1));
            raw[0] = p[0], raw[1] = p[1];
        } else {
            raw[0] = *(const u32x4 *)(x + 8 * block);
        }
    }

    __device__ __forceinline__ u32x4 ordered(int block) const // x, y: step 2n; z, w: step 2n + 1
    {
        uint32_t a0 = raw[0].x, a1 = raw[0].y, b0 = raw[0].z, b1 = raw[0].w;
        if constexpr (BITS == 2) {
            const bool odd = block & 1; // columns 2, 3 of each four instead of 0, 1
            a0 = odd ? raw[0].y : raw[0].x, a1 = odd ? raw[0].w : raw[0].z;
            b0 = odd ? raw[1].y : raw[1].x, b1 = odd ? raw[1].w : raw[1].z;
        }
        return u32x4{perm(a1, a0, 0x05040100), perm(b1, b0, 0x05040100), perm(a1, a0, 0x07060302),
                     perm(b1, b0, 0x07060302)};
    }
};

// The experts in use, each once and in ascending order, are the launch's grid
// rows: which expert row `slot` is, and which tokens chose it.  Every wave
// works it out for itself from ids[] (at most 128), without a barrier: a
// bitmap of the experts, its running count, and two ballots.
// Orders a wave's own LDS accesses (its LDS instructions run in order; the
// compiler may not move them across this).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct Chosen {
    int expert; // -1: fewer experts are in use
    int count;  // tokens that chose it
};

struct ChosenLds {
    uint32_t bitmap[kMaxExperts / 32];
    uint32_t list[kMaxBatch]; // token | first of its choices << 8
};

__device__ __forceinline__ Chosen find_chosen(const int32_t *ids, int pairs, int topk, int batch, int experts, int slot,
                                              ChosenLds &lds)
{
    const int lane = threadIdx.x & 63;
    auto id_of = [&](int p) {
        const int e = p < pairs ? ids[p] : -1;
        return e < experts ? e : -1;
    };
    const int e0 = id_of(lane), e1 = id_of(lane + 64);
    if (lane < kMaxExperts / 32) lds.bitmap[lane] = 0;
    wave_sync();
    if (e0 >= 0) atomicOr(&lds.bitmap[e0 >> 5], 1u << (e0 & 31));
    if (e1 >= 0) atomicOr(&lds.bitmap[e1 >> 5], 1u << (e1 & 31));
    wave_sync();
    const uint32_t word = lane < kMaxExperts / 32 ? lds.bitmap[lane] : 0;
    int before = __popc(word); // running count over the sixteen words, in one row of lanes
    static_assert(kMaxExperts / 32 == 16, "one row of lanes");
    before += __builtin_amdgcn_update_dpp(0, before, 0x111, 0xF, 0xF, true); // row_shr 1, 2, 4, 8
    before += __builtin_amdgcn_update_dpp(0, before, 0x112, 0xF, 0xF, true);
    before += __builtin_amdgcn_update_dpp(0, before, 0x114, 0xF, 0xF, true);
    before += __builtin_amdgcn_update_dpp(0, before, 0x118, 0xF, 0xF, true);
    const uint64_t past = __ballot(lane < kMaxExperts / 32 && before > slot);
    if (past == 0) return {-1, 0};
    const int at = __builtin_ctzll(past);
    uint32_t w = __builtin_amdgcn_readlane(word, at);
    for (int skip = slot - (__builtin_amdgcn_readlane(before, at) - __popc(w)); skip > 0; --skip) w &= w - 1;
    const int e = 32 * at + __builtin_ctz(w);
    const uint64_t m0 = __ballot(e0 == e), m1 = __ballot(e1 == e);
    // lane t: token t's choices are bits t * topk .. of the 128
    const int sh = lane * topk;
    uint64_t bits = 0;
    if (lane < batch) bits = sh >= 64 ? m1 >> (sh - 64) : (m0 >> sh) | (sh ? m1 << (64 - sh) : 0);
    bits &= (1ull << topk) - 1;
    const uint64_t tokens = __ballot(bits != 0);
    if (bits) lds.list[__popcll(tokens & ((1ull << lane) - 1))] = lane | (__builtin_ctzll(bits) << 8);
    wave_sync();
    return {e, (int)__popcll(tokens)};
}

// The pair (token, first choice) of an expert's token j, j the same in all
// lanes: in scalar registers, where the addresses of sixteen tokens fit.
__device__ __forceinline__ int64_t same_pair(const ChosenLds &lds, int j, int topk)
{
    const int at = __builtin_amdgcn_readfirstlane(lds.list[j]);
    return (at & 255) * topk + (at >> 8);
}

// One chunk of 64 nonzeros [cb, min(cb + 64, v1)) of a tile: a nonzero per lane,
// rows non-decreasing over the lanes, lanes past the end of no row; lane = row
// has its row's entries [rp_lo, rp_hi).
struct Chunk {
    int back; // lanes before this one with nonzeros of the same row
    int last; // lane of the last nonzero of this lane's row, -1 if it has none here

    __device__ __forceinline__ void set(int cb, int v1, int lane, int rp_lo, int rp_hi)
    {
        const int first = max(rp_lo, cb) - cb, end = min(min(rp_hi, cb + 64), v1) - 1 - cb;
        last = first <= end ? end : -1;
        const uint64_t head = first <= end ? 1ull << first : 0; // first lanes of the rows here
        const uint64_t heads = (uint64_t)wave_or((uint32_t)(head >> 32)) << 32 | wave_or((uint32_t)head);
        back = lane - (63 - __clzll(heads & ((2ull << lane) - 1)));
    }

    // Adds the chunk (lane's product v) to the row lanes' sums: an
    // inclusive scan over the wave that starts anew at each row, of which a row
    // takes its last lane.  (The difference of an unbroken scan at a row's ends
    // is two instructions a step less, but has the rounding errors of all rows
    // before it in the chunk, and NaN after an infinity.)
    __device__ __forceinline__ void add(float v, int lane, float &sum) const
    {
        int n = back;
        asm("" : "+v"(n)); // compared anew for each token: the comparisons' masks do not fit the scalar registers
        // (the shifts are calls, made by all lanes before any is chosen)
        auto step = [&](bool same, float before) { v += same ? before : 0.f; };
        step(n >= 1, dev::row_shr<1>(v));
        step(n >= 2, dev::row_shr<2>(v));
        step(n >= 4, dev::row_shr<4>(v));
        step(n >= 8, dev::row_shr<8>(v));
        step(n > (lane & 15), dev::row_bcast15(v));
        step(n > (lane & 31), dev::row_bcast31(v));
        const float top = dev::lane_read(max(last, 0), v);
        sum += last >= 0 ? top : 0.f;
    }
};

// A wave's share of a tile's outliers, in one of two forms.
//   By rows: lane = row takes entries 4 share .. 4 share + 3 of its row, then
//     those 4 `shares` further, four at a load.  About 30 vector instructions
//     a step and 12 a token.
//   By chunks: an even part [v0, v1) of the tile's nonzeros, 64 at a time, a
//     nonzero per lane (Chunk): about 40 vector instructions a chunk and 35 a
//     token, whatever the rows hold.
// By rows unless the fullest row would take more than twice as many steps as
// there are chunks (us of a call by rows and by chunks, replayed from a graph:
// 16 tokens, 128 experts 4096x1536 at 0.45% 148 and 159, at 2% 211 and 231; 8
// experts 4096x3584, 4 bits, 58 and 62, 71 and 96, at 5% 96 and 172; 8 tokens,
// 128 experts 2048x768, 4 bits, 57 and 57, 61 and 68).
struct Outliers {
    const uint16_t *cols, *vals; // the tile's
    int lo, count;               // this lane's row: entries [lo, lo + count)
    int len;                     // the tile's
    int share, shares, log; // log2 of shares
    int64_t left;                // entries from the tile's first to the arrays' end

    __device__ __forceinline__ void set(const Projection &p, int rp_lo, int rp_hi, int worker, int log_workers)
    {
        const int nz0 = __builtin_amdgcn_readfirstlane(rp_lo); // all else relative to the tile's first
        lo = rp_lo - nz0, count = rp_hi - rp_lo;
        len = __builtin_amdgcn_readlane(rp_hi, 63) - nz0;
        cols = p.col + nz0, vals = p.val + nz0;
        share = worker, shares = 1 << log_workers, log = log_workers;
        left = p.nnz - nz0;
    }

    // Their products with the tokens' activations value(j, c), into sum[j].
    template <int T, int N, typename V>
    __device__ __forceinline__ void add(int tokens, V value, float (&sum)[N]) const
    {
        const int steps = ((int)wave_max((uint32_t)count) + 4 * shares - 1) >> (log + 2);
        const int chunks = (len + 64 * shares - 1) >> (log + 6);
        if (left >= 4 && steps <= 2 * chunks)
            by_rows<T>(tokens, value, sum, steps);
        else
            by_chunks<T>(tokens, value, sum);
    }

    template <int T, int N, typename V>
    __device__ __forceinline__ void by_rows(int tokens, V value, float (&sum)[N], int steps) const
    {
        for (int n = 0; n < steps; ++n) {
            const int first = 4 * (share + n * shares); // of the row
            // four entries at once, from further left at the end of the arrays
            const int64_t at = min(lo + (int64_t)min(first, max(count - 1, 0)), left - 1), from = min(at, left - 4);
            const int skip = 16 * (int)(at - from);
            uint64_t c, v;
            __builtin_memcpy(&c, cols + from, 8);
            __builtin_memcpy(&v, vals + from, 8);
            c >>= skip, v >>= skip;
            float w[4];
            int col[4];
            // Entries past the row's count are other rows' or, at the arrays' end,
            // nobody's: they read x in column 0 and add nothing, whatever it holds.
            bool own[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                own[k] = first + k < count;
                col[k] = own[k] ? (int)(c >> (16 * k)) & 0xFFFF : 0;
                w[k] = dev::f16_to_f32((uint16_t)(v >> (16 * k)));
            }
#pragma unroll
            for (int j = 0; j < T; ++j)
                if (j < tokens) {
                    float xv[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) xv[k] = value(j, col[k]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum[j] += own[k] ? w[k] * xv[k] : 0.f;
                }
        }
    }

    template <int T, int N, typename V>
    __device__ __forceinline__ void by_chunks(int tokens, V value, float (&sum)[N]) const
    {
        const int lane = threadIdx.x & 63, per = len >> log, extra = len - per * shares;
        const int v0 = share * per + min(share, extra), v1 = v0 + per + (share < extra ? 1 : 0);
        constexpr int kAtOnce = 2;
        for (int base = v0; base < v1; base += 64 * kAtOnce) {
            int col[kAtOnce];
            float val[kAtOnce];
            Chunk chunk[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) { // past the last: that one again, of no row
                const int at = min(base + 64 * k + lane, v1 - 1);
                col[k] = cols[at];
                val[k] = dev::f16_to_f32(vals[at]);
                chunk[k].set(base + 64 * k, v1, lane, lo, lo + count);
            }
#pragma unroll
            for (int j = 0; j < T; ++j)
                if (j < tokens) {
                    float xv[kAtOnce];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) xv[k] = value(j, col[k]);
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
                        if (base + 64 * k < v1) chunk[k].add(val[k] * xv[k], lane, sum[j]);
                    __builtin_amdgcn_sched_barrier(0); // (tokens interleaved do not fit the registers)
                }
        }
    }
};

// This wave's share (worker `worker` of 2^log_workers) of one matrix for one
// tile: every so many half groups; its share of the outliers is left in `out`.
// x(j) is the fp16 row of matrix column j.
// Column 4h + i of the matrix steps ends in sum[4h + i].
template <int BITS, int NQ, typename X>
__device__ __forceinline__ void tile_product(const Projection &p, int64_t tile, int groups, int worker, int log_workers, X x,
                                             float (&sum)[4 * NQ], Outliers &out)
{
    // half groups in flight, as many as fit 128 registers (with sums of sixteen
    // tokens, NQ = 8, even one spills four to seven of them)
    constexpr int D = NQ == 1 ? (BITS == 2 ? 3 : 4) : (NQ == 2 ? (BITS == 2 ? 2 : 3) : (NQ == 4 && BITS == 3 ? 2 : 1));
    constexpr int C = NQ == 1 ? 2 : 1; // accumulator chains: a step does not wait for the one before it
    const int lane = threadIdx.x & 63, block = lane >> 2;
    const int64_t row = tile * 64 + lane;
    Table<BITS> table;
    table.load(p.lut + (row << BITS));
    const int32_t *rp = p.nnz ? p.row_ptr + row : (const int32_t *)dev::g_placeholder;
    const int rp_lo = rp[0], rp_hi = rp[1];
    const int workers = 1 << log_workers;
    const int n = (2 * groups - worker + workers - 1) >> log_workers; // half groups of this wave
    const uint8_t *codes = p.packed + tile * groups * (2 * BITS * 1024);
    const uint16_t *xr[NQ];
#pragma unroll
    for (int h = 0; h < NQ; ++h) xr[h] = x(4 * h + (lane & 3));
    Half<BITS> ring[D];
    QuadX<BITS> xq[D][NQ];
    // The same loads in every step, so that the waits before a step leave the
    // ring's other loads in flight: past the wave's last half group they read
    // a few cached zeros.
    auto load = [&](int k, int i) {
        const int g = worker + i * workers;
        ring[k].load((i < n ? codes + (int64_t)g * (BITS * 1024) : (const uint8_t *)dev::g_placeholder) + lane * 16);
#pragma unroll
        for (int h = 0; h < NQ; ++h)
            xq[k][h].load(i < n ? xr[h] + 128 * g : (const uint16_t *)dev::g_placeholder, block);
    };
    f32x4 acc[NQ][C];
#pragma unroll
    for (int h = 0; h < NQ; ++h)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[h][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int k) {
        u32x4 xs[NQ];
#pragma unroll
        for (int h = 0; h < NQ; ++h) xs[h] = xq[k][h].ordered(block);
        [&]<int... Ns>(std::integer_sequence<int, Ns...>) {
            (
                [&] {
                    const half4_t we = ring[k].template weights<2 * Ns>(table);
                    const half4_t wo = ring[k].template weights<2 * Ns + 1>(table);
#pragma unroll
                    for (int h = 0; h < NQ; ++h)
                        acc[h][0] = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(half4_t, u32x2{xs[h].x, xs[h].y}),
                                                                      we, acc[h][0], 4, Ns, 0);
#pragma unroll
                    for (int h = 0; h < NQ; ++h)
                        acc[h][C - 1] = __builtin_amdgcn_mfma_f32_4x4x4f16(
                            __builtin_bit_cast(half4_t, u32x2{xs[h].z, xs[h].w}), wo, acc[h][C - 1], 4, Ns, 0);
                }(),
                ...);
        }(std::make_integer_sequence<int, 16>{});
    };
#pragma unroll
    for (int k = 0; k < D; ++k) load(k, k);
    out.set(p, rp_lo, rp_hi, worker, log_workers);
    int i = 0;
    for (; i + D <= n; i += D) {
#pragma unroll
        for (int k = 0; k < D; ++k) {
            multiply(k);
            load(k, i + k + D);
        }
    }
#pragma unroll
    for (int k = 0; k < D - 1; ++k)
        if (i + k < n) multiply(k);
#pragma unroll
    for (int h = 0; h < NQ; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[4 * h + r] = C == 2 ? acc[h][0][r] + acc[h][C - 1][r] : acc[h][0][r];
}

// The other decode, at 3 and 4 bits: a table in LDS of the tile's pairs of
// centroids, entry [second code][first code][row] of two fp16 values (16 or 64
// KB; a row's entries share a bank of its own).  A pair of codes is a byte, and
// the address of its entry that byte above the row's: one v_perm_b32 and one LDS
// read for two weights, in the order of their columns, where the decode from
// registers takes six vector instructions at 4 bits and three at 3.
template <int BITS>
constexpr int kPairTable = (1 << 2 * BITS) * 64 * 4;
template <int BITS>
constexpr int kBuilders = 1 << (BITS - 1); // waves that write a table, two second codes each

// A row's centroids, and those of the two second codes whose entries this wave
// writes.
template <int BITS>
struct PairRow {
    uint32_t first[1 << (BITS - 1)], second;

    __device__ __forceinline__ void load(const uint16_t *row, int builder)
    {
#pragma unroll
        for (int q = 0; q < (1 << BITS) / 8; ++q) {
            const u32x4 v = ((const u32x4 *)row)[q];
            first[4 * q] = v.x, first[4 * q + 1] = v.y, first[4 * q + 2] = v.z, first[4 * q + 3] = v.w;
        }
        second = ((const uint32_t *)row)[builder];
    }

    __device__ __forceinline__ void store(uint8_t *table, int builder) const
    {
        uint32_t *to = (uint32_t *)table + (builder << (BITS + 7)) + (threadIdx.x & 63);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < 1 << BITS; ++c)
                to[((s << BITS) + c) * 64] =
                    perm(second, first[c / 2], (c & 1 ? 0x0302 : 0x0100) | (s ? 0x07060000 : 0x05040000));
    }
};

// The half group that a wave has on its way, codes and activations, and the
// sums of one matrix.  (One is enough with sixteen waves a compute unit: with
// two or three the registers do not hold the table's answers too, 4 tokens, 8
// experts 4096x14336 at 4 bits 132 and 152 us a call against 114.)
template <int BITS, int NQ>
struct TableProduct {
    static constexpr int C = NQ == 1 ? 2 : 1; // accumulator chains, as in tile_product
    Half<BITS> codes;
    u32x4 x[NQ];
    f32x4 acc[NQ][C];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int h = 0; h < NQ; ++h)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[h][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // Half group g (128 columns) of a tile.
    __device__ __forceinline__ void load(const uint8_t *tile, const uint16_t *const (&rows)[NQ], int g)
    {
        const int lane = threadIdx.x & 63;
        codes.load(tile + (int64_t)g * (BITS * 1024) + lane * 16);
#pragma unroll
        for (int h = 0; h < NQ; ++h) x[h] = *(const u32x4 *)(rows[h] + 128 * g + 8 * (lane >> 2));
    }

    __device__ __forceinline__ void multiply(const uint8_t *table)
    {
        const uint32_t row = (threadIdx.x & 63) * 4; // of an entry, below the pair's byte
        [&]<int... Ns>(std::integer_sequence<int, Ns...>) {
            (
                [&] {
                    uint32_t v = codes.template pairs<Ns>();
                    if constexpr (BITS == 3) v &= 0x3F3F3F3F;
                    const uint32_t e0 = *(const uint32_t *)(table + perm(v, row, 0x0C0C0400));
                    const uint32_t e1 = *(const uint32_t *)(table + perm(v, row, 0x0C0C0500));
                    const uint32_t e2 = *(const uint32_t *)(table + perm(v, row, 0x0C0C0600));
                    const uint32_t e3 = *(const uint32_t *)(table + perm(v, row, 0x0C0C0700));
#pragma unroll
                    for (int h = 0; h < NQ; ++h)
                        acc[h][0] = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(half4_t, u32x2{x[h].x, x[h].y}),
                                                                      __builtin_bit_cast(half4_t, u32x2{e0, e1}), acc[h][0], 4,
                                                                      Ns, 0);
#pragma unroll
                    for (int h = 0; h < NQ; ++h)
                        acc[h][C - 1] = __builtin_amdgcn_mfma_f32_4x4x4f16(
                            __builtin_bit_cast(half4_t, u32x2{x[h].z, x[h].w}),
                            __builtin_bit_cast(half4_t, u32x2{e2, e3}), acc[h][C - 1], 4, Ns, 0);
                }(),
                ...);
        }(std::make_integer_sequence<int, 16>{});
    }

    __device__ __forceinline__ void sums(float (&sum)[4 * NQ]) const
    {
#pragma unroll
        for (int h = 0; h < NQ; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[4 * h + r] = C == 2 ? acc[h][0][r] + acc[h][C - 1][r] : acc[h][0][r];
    }
};

// Every wave's loads into LDS have arrived.
__device__ __forceinline__ void all_loads_done()
{
    __builtin_amdgcn_s_waitcnt(0x0F70); // vmcnt(0)
    __syncthreads();
}

// Copies `rows` rows of `bytes` (a multiple of 512) into LDS, row j from
// source(j), 1 KB or the rest of a row per instruction, straight from memory;
// they are there once the caller's later loads are and all waves have met.
template <typename S>
__device__ __forceinline__ void stage_rows(int rows, int bytes, S source, uint8_t *lds)
{
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    for (int j = 0; j < rows; ++j) {
        const uint8_t *src = source(j);
        for (int at = w * 1024; at < bytes; at += kDefaultWaves * 1024)
            if (at + lane * 16 < bytes)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t *)(src + at + lane * 16),
                                                 (__attribute__((address_space(3))) uint32_t *)(lds + j * bytes + at), 16,
                                                 0, 0);
    }
}

// ---------------------------------------------------------------------------
// a = silu(gate x) * (up x), split into two fp16 values per entry for the
// matrix steps of down, hi + lo * 2^-11 (one fp16 value would double the error
// of y; without the factor lo would have no bits left where a is small), and
// whole for its outliers.
// The even waves of a workgroup have the gate's tile, the odd ones the up's.
// (Two or four tiles to a workgroup, with two or four of its waves each,
// measured no faster anywhere: 16 tokens, 128 experts 1536x4096 103 and 92 us
// against 90; one token, 6 experts 1280x2048 22 and 14 us against 10.)
// Grid (inter / 64, experts in use at most).
// ---------------------------------------------------------------------------
struct Activations { // [pair][inter]
    uint16_t *hi, *lo;
    float *whole;
};

__device__ __forceinline__ void store_activation(const Activations &a, const ChosenLds &lds, int j, int topk, int inter,
                                                 int tile, float g, float u)
{
    const float v = g / (1.f + expf(-g)) * u;
    const _Float16 hi = (_Float16)v;
    const float rest = fabsf(v) < 65520.f ? (v - (float)hi) * 2048.f : 0.f; // beyond, hi is infinite or NaN
    const int64_t pair = (int64_t)(lds.list[j] & 255) * topk + (lds.list[j] >> 8);
    const int64_t at = pair * inter + tile * 64 + (threadIdx.x & 63);
    a.hi[at] = __builtin_bit_cast(uint16_t, hi);
    a.lo[at] = __builtin_bit_cast(uint16_t, (_Float16)rest);
    a.whole[at] = v;
}

template <int BITS, int NQ>
__device__ __forceinline__ void gate_up_body(const Projection &gate, const Projection &up, const uint16_t *x,
                                             const ChosenLds &lds, Chosen c, int topk, int hidden, int inter,
                                             int room, Activations a, uint8_t *space)
{
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x;
    const int64_t tile = (int64_t)c.expert * (inter >> 6) + t;
    auto row_of = [&](int j) { return x + (int64_t)(lds.list[j] & 255) * hidden; };
    const int64_t own_nnz = w & 1 ? up.nnz : gate.nnz;
    const bool staged = c.count * hidden * 2 <= room && gate.nnz + up.nnz > 0;
    if (staged)
        stage_rows(c.count, hidden * 2, [&](int j) { return (const uint8_t *)row_of(j); }, space);
    float sum[4 * NQ];
    Outliers out;
    tile_product<BITS, NQ>(w & 1 ? up : gate, tile, hidden >> 8, w >> 1, kLogWaves - 1,
                           [&](int j) { return row_of(min(j, c.count - 1)); }, // past the last: a copy, dropped
                           sum, out);
    if (staged) {
        all_loads_done();
        const uint16_t *xs = (const uint16_t *)space;
        if (own_nnz) out.add<4 * NQ>(c.count, [&](int j, int col) { return dev::f16_to_f32(xs[j * hidden + col]); }, sum);
        __syncthreads(); // the space is used again below
    } else if (own_nnz) {
        out.add<4 * NQ>(c.count, [&](int j, int col) { return dev::f16_to_f32(row_of(j)[col]); }, sum);
    }
    float *const red = (float *)space;
#pragma unroll
    for (int j = 0; j < 4 * NQ; ++j) red[(w * 4 * NQ + j) * 64 + lane] = sum[j];
    __syncthreads();
    for (int j = w; j < c.count; j += kDefaultWaves) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < kDefaultWaves; k += 2) {
            g += red[(k * 4 * NQ + j) * 64 + lane];
            u += red[((k + 1) * 4 * NQ + j) * 64 + lane];
        }
        store_activation(a, lds, j, topk, inter, t, g, u);
    }
}

// The same at 4 bits by pair tables: all waves have the gate's tile, then the
// up's, each at every eighth half group, in one stream of loads.  The up's
// table takes the gate's place, so that two workgroups share a compute unit.
template <int NQ>
__device__ __forceinline__ void gate_up_table_body(const Projection &gate, const Projection &up, const uint16_t *x,
                                                   const ChosenLds &lds, Chosen c, int topk, int hidden, int inter,
                                                   int room, Activations a, uint8_t *space)
{
    constexpr int BITS = 4;
    static_assert(kBuilders<BITS> == kDefaultWaves);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x;
    const int64_t tile = (int64_t)c.expert * (inter >> 6) + t, row = tile * 64 + lane;
    auto row_of = [&](int j) { return x + (int64_t)(lds.list[j] & 255) * hidden; };
    PairRow<BITS> entries, next;
    entries.load(gate.lut + (row << BITS), w);
    next.load(up.lut + (row << BITS), w);
    const int32_t *grp = gate.nnz ? gate.row_ptr + row : (const int32_t *)dev::g_placeholder;
    const int32_t *urp = up.nnz ? up.row_ptr + row : (const int32_t *)dev::g_placeholder;
    const int g_lo = grp[0], g_hi = grp[1], u_lo = urp[0], u_hi = urp[1];
    const int halves = hidden >> 7, n = (halves - w + kDefaultWaves - 1) >> kLogWaves; // of this wave
    const int64_t from = tile * halves * (BITS * 1024);
    const uint16_t *xr[NQ];
#pragma unroll
    for (int h = 0; h < NQ; ++h) xr[h] = row_of(min(4 * h + (lane & 3), c.count - 1)); // past the last: a copy, dropped
    TableProduct<BITS, NQ> p;
    auto load = [&](int i) { // gate's n, then up's
        if (i < 2 * n) p.load((i < n ? gate : up).packed + from, xr, w + (i < n ? i : i - n) * kDefaultWaves);
    };
    auto run = [&](int first, float (&to)[4 * NQ]) {
        p.clear();
        for (int i = first; i < first + n; ++i) {
            p.multiply(space);
            load(i + 1);
        }
        p.sums(to);
    };
    float sum[2][4 * NQ];
    load(0);
    entries.store(space, w);
    dev::lds_barrier();
    run(0, sum[0]);
    dev::lds_barrier(); // the gate's table is done with
    next.store(space, w);
    dev::lds_barrier();
    run(n, sum[1]);
    __syncthreads(); // the up's too
    if (gate.nnz + up.nnz > 0) {
        const bool staged = c.count * hidden * 2 <= room;
        if (staged) {
            stage_rows(c.count, hidden * 2, [&](int j) { return (const uint8_t *)row_of(j); }, space);
            all_loads_done();
        }
        const uint16_t *xs = (const uint16_t *)space;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Projection &q = s ? up : gate;
            if (q.nnz == 0) continue;
            Outliers out;
            out.set(q, s ? u_lo : g_lo, s ? u_hi : g_hi, w, kLogWaves);
            if (staged)
                out.add<4 * NQ>(c.count, [&](int j, int col) { return dev::f16_to_f32(xs[j * hidden + col]); }, sum[s]);
            else
                out.add<4 * NQ>(c.count, [&](int j, int col) { return dev::f16_to_f32(row_of(j)[col]); }, sum[s]);
        }
        __syncthreads(); // the space is used again below
    }
    float *const red = (float *)space;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4 * NQ; ++j) red[((s * kDefaultWaves + w) * 4 * NQ + j) * 64 + lane] = sum[s][j];
    __syncthreads();
    for (int j = w; j < c.count; j += kDefaultWaves) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < kDefaultWaves; ++k) {
            g += red[(k * 4 * NQ + j) * 64 + lane];
            u += red[((kDefaultWaves + k) * 4 * NQ + j) * 64 + lane];
        }
        store_activation(a, lds, j, topk, inter, t, g, u);
    }
}

template <int MAXQ>
__global__ void __launch_bounds__(kDefaultWaves * 64, 4) experts_gate_up_table(Projection gate, Projection up,
                                                                        const uint16_t *x, const int32_t *ids, int batch,
                                                                        int experts, int topk, int hidden, int inter,
                                                                        int room, Activations a)
{
    __shared__ ChosenLds chosen[kDefaultWaves];
    extern __shared__ __align__(16) uint8_t space[];
    ChosenLds &lds = chosen[threadIdx.x >> 6];
    const Chosen c = find_chosen(ids, batch * topk, topk, batch, experts, blockIdx.y, lds);
    if (c.expert < 0) return;
    // above eight tokens the table's answers and the sums do not fit the
    // registers (16 tokens, 2 experts 4096x4096: 78 us a call, from registers 71)
    if (MAXQ >= 4 && c.count > 8)
        gate_up_body<4, MAXQ >= 4 ? 4 : 1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
    else if (MAXQ >= 2 && c.count > 4)
        gate_up_table_body<MAXQ >= 2 ? 2 : 1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
    else
        gate_up_table_body<1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
}

template <int BITS, int MAXQ>
__global__ void __launch_bounds__(kDefaultWaves * 64, 4) experts_gate_up(Projection gate, Projection up, const uint16_t *x,
                                                                  const int32_t *ids, int batch, int experts, int topk,
                                                                  int hidden, int inter, int room, Activations a)
{
    __shared__ ChosenLds chosen[kDefaultWaves];
    extern __shared__ __align__(16) uint8_t space[];
    ChosenLds &lds = chosen[threadIdx.x >> 6];
    const Chosen c = find_chosen(ids, batch * topk, topk, batch, experts, blockIdx.y, lds);
    if (c.expert < 0) return;
    if (MAXQ >= 4 && c.count > 8)
        gate_up_body<BITS, MAXQ >= 4 ? 4 : 1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
    else if (MAXQ >= 2 && c.count > 4)
        gate_up_body<BITS, MAXQ >= 2 ? 2 : 1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
    else
        gate_up_body<BITS, 1>(gate, up, x, lds, c, topk, hidden, inter, room, a, space);
}

// ---------------------------------------------------------------------------
// part[split][pair][hidden] = down a, fp32, over the split's columns.  A
// token j's two fp16 values stand in columns j and 2 NQ + j.
// Grid (workgroups for hidden / 64 tiles, experts in use at most, splits).
// ---------------------------------------------------------------------------
// By pair tables: eight waves share a tile.
template <int BITS, int NQ>
__device__ __forceinline__ void down_table_body(const Projection &down, Activations a, const ChosenLds &lds, Chosen c,
                                                int topk, int hidden, int inter, int room, int64_t pairs,
                                                float *partial, uint8_t *space)
{
    constexpr int T = 2 * NQ;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x;
    const int64_t tile = (int64_t)c.expert * (hidden >> 6) + t, row = tile * 64 + lane;
    auto pair_of = [&](int j) { return (int64_t)(lds.list[j] & 255) * topk + (lds.list[j] >> 8); };
    const int log_workers = kLogWaves + __builtin_ctz(gridDim.z), workers = 1 << log_workers; // splits: a power of two
    const int worker = blockIdx.z * kDefaultWaves + w;
    const int64_t lo_from_hi = a.lo - a.hi; // (a choice between the pointers puts them in scratch memory)
    PairRow<BITS> entries;
    entries.load(down.lut + (row << BITS), w % kBuilders<BITS>);
    const int32_t *rp = down.nnz ? down.row_ptr + row : (const int32_t *)dev::g_placeholder;
    const int lo = rp[0], hi = rp[1];
    const int halves = inter >> 7, n = (halves - worker + workers - 1) >> log_workers; // of this wave
    const uint16_t *xr[NQ];
#pragma unroll
    for (int h = 0; h < NQ; ++h) {
        const int j = 4 * h + (lane & 3);
        xr[h] = a.hi + (j < T ? 0 : lo_from_hi) + pair_of(min(j & (T - 1), c.count - 1)) * inter;
    }
    TableProduct<BITS, NQ> p;
    auto load = [&](int i) {
        if (i < n) p.load(down.packed + tile * halves * (BITS * 1024), xr, worker + i * workers);
    };
    load(0);
    if (w < kBuilders<BITS>) entries.store(space, w);
    dev::lds_barrier();
    p.clear();
    for (int i = 0; i < n; ++i) {
        p.multiply(space);
        load(i + 1);
    }
    float sum[4 * NQ];
    p.sums(sum);
    __syncthreads(); // the table is done with
    if (down.nnz > 0) { // (staged now, the table had the space)
        auto whole_of = [&](int j) { return a.whole + same_pair(lds, j, topk) * inter; };
        const bool staged = c.count * inter * 4 <= room;
        if (staged) {
            stage_rows(c.count, inter * 4, [&](int j) { return (const uint8_t *)whole_of(j); }, space);
            all_loads_done();
        }
        Outliers out;
        out.set(down, lo, hi, worker, log_workers);
        const float *xs = (const float *)space;
        if (staged)
            out.add<T>(c.count, [&](int j, int col) { return xs[j * inter + col]; }, sum);
        else
            out.add<T>(c.count, [&](int j, int col) { return whole_of(j)[col]; }, sum);
        __syncthreads(); // the space is used again below
    }
    float *const red = (float *)space;
#pragma unroll
    for (int j = 0; j < T; ++j) red[(w * T + j) * 64 + lane] = sum[j] + sum[T + j] * 0x1p-11f;
    __syncthreads();
    for (int j = w; j < c.count; j += kDefaultWaves) {
        float v = 0.f;
        for (int k = 0; k < kDefaultWaves; ++k) v += red[(k * T + j) * 64 + lane];
        partial[(blockIdx.z * pairs + pair_of(j)) * hidden + t * 64 + lane] = v;
    }
}

template <int BITS, int MAXQ>
__global__ void __launch_bounds__(kDefaultWaves * 64, 4) experts_down_table(Projection down, Activations a,
                                                                     const int32_t *ids, int batch, int experts, int topk,
                                                                     int hidden, int inter, int room, float *partial)
{
    __shared__ ChosenLds chosen[kDefaultWaves];
    extern __shared__ __align__(16) uint8_t space[];
    ChosenLds &lds = chosen[threadIdx.x >> 6];
    const Chosen c = find_chosen(ids, batch * topk, topk, batch, experts, blockIdx.y, lds);
    if (c.expert < 0) return;
    const int64_t pairs = batch * topk;
    if (MAXQ >= 4 && c.count > 8)
        down_table_body<BITS, MAXQ >= 4 ? 8 : 1>(down, a, lds, c, topk, hidden, inter, room, pairs, partial, space);
    else if (MAXQ >= 2 && c.count > 4)
        down_table_body<BITS, MAXQ >= 2 ? 4 : 1>(down, a, lds, c, topk, hidden, inter, room, pairs, partial, space);
    else if (c.count > 2)
        down_table_body<BITS, 2>(down, a, lds, c, topk, hidden, inter, room, pairs, partial, space);
    else
        down_table_body<BITS, 1>(down, a, lds, c, topk, hidden, inter, room, pairs, partial, space);
}

// From registers: `parts` waves share a tile, so that a workgroup has 8 / parts.
template <int BITS, int NQ>
__device__ __forceinline__ void down_body(const Projection &down, Activations a, const ChosenLds &lds, Chosen c,
                                          int topk, int hidden, int inter, int log_parts, int room, int64_t pairs,
                                          float *partial, uint8_t *space)
{
    constexpr int T = 2 * NQ; // tokens
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int parts = 1 << log_parts, tiles = hidden >> 6, part = w & (parts - 1);
    const int t = (blockIdx.x << (kLogWaves - log_parts)) + (w >> log_parts);
    const bool owns = t < tiles; // the last workgroup may have waves too many
    const int64_t tile = (int64_t)c.expert * tiles + min(t, tiles - 1);
    auto pair_of = [&](int j) { return (int64_t)(lds.list[j] & 255) * topk + (lds.list[j] >> 8); };
    float *const to = partial + blockIdx.z * pairs * hidden + t * 64 + lane;
    float sum[4 * NQ];
    const int log_workers = log_parts + __builtin_ctz(gridDim.z), worker = blockIdx.z * parts + part;
    const int64_t lo_from_hi = a.lo - a.hi; // (a choice between the pointers puts them in scratch memory)
    auto whole_of = [&](int j) { return a.whole + same_pair(lds, j, topk) * inter; };
    const bool staged = c.count * inter * 4 <= room && down.nnz > 0;
    if (staged) stage_rows(c.count, inter * 4, [&](int j) { return (const uint8_t *)whole_of(j); }, space);
    Outliers out;
    tile_product<BITS, NQ>(down, tile, inter >> 8, worker, log_workers,
                           [&](int j) { return a.hi + (j < T ? 0 : lo_from_hi) + pair_of(min(j & (T - 1), c.count - 1)) * inter; },
                           sum, out);
    if (staged) {
        all_loads_done();
        const float *xs = (const float *)space;
        out.add<T>(c.count, [&](int j, int col) { return xs[j * inter + col]; }, sum);
        __syncthreads(); // the space is used again below
    } else if (down.nnz > 0) {
        out.add<T>(c.count, [&](int j, int col) { return whole_of(j)[col]; }, sum);
    }
    auto whole = [&](int j) { return sum[j] + sum[T + j] * 0x1p-11f; };
    float *const red = (float *)space;
    if (parts == 1) {
#pragma unroll
        for (int j = 0; j < T; ++j)
            if (owns && j < c.count) to[pair_of(j) * hidden] = whole(j);
        return;
    }
#pragma unroll
    for (int j = 0; j < T; ++j) red[(w * T + j) * 64 + lane] = whole(j);
    __syncthreads();
    const int w0 = w - part;
    for (int j = part; j < c.count; j += parts) {
        float v = 0.f;
        for (int k = w0; k < w0 + parts; ++k) v += red[(k * T + j) * 64 + lane];
        if (owns) to[pair_of(j) * hidden] = v;
    }
}

template <int BITS, int MAXQ>
__global__ void __launch_bounds__(kDefaultWaves * 64, 4) experts_down(Projection down, Activations a,
                                                                      const int32_t *ids, int batch, int experts,
                                                                      int topk, int hidden, int inter, int log_parts,
                                                                      int room, float *partial)
{
    __shared__ ChosenLds chosen[kDefaultWaves];
    extern __shared__ __align__(16) uint8_t space[];
    ChosenLds &lds = chosen[threadIdx.x >> 6];
    const Chosen c = find_chosen(ids, batch * topk, topk, batch, experts, blockIdx.y, lds);
    if (c.expert < 0) return;
    const int64_t pairs = batch * topk;
    if (MAXQ >= 4 && c.count > 8)
        down_body<BITS, MAXQ >= 4 ? 8 : 1>(down, a, lds, c, topk, hidden, inter, log_parts, room, pairs, partial, space);
    else if (MAXQ >= 2 && c.count > 4)
        down_body<BITS, MAXQ >= 2 ? 4 : 1>(down, a, lds, c, topk, hidden, inter, log_parts, room, pairs, partial, space);
    else if (MAXQ >= 1 && c.count > 2)
        down_body<BITS, MAXQ >= 1 ? 2 : 1>(down, a, lds, c, topk, hidden, inter, log_parts, room, pairs, partial, space);
    else
        down_body<BITS, 1>(down, a, lds, c, topk, hidden, inter, log_parts, room, pairs, partial, space);
}

// y = the weighted sum of a token's partial sums, its choices in order; a
// repeated id's partial sums stand at its first choice.  All of them are loaded
// before the first is used.  (Adding them up in the down launch instead, by the
// last workgroup of each 64 to 512 rows to arrive, measured slower at every
// size: 14.4 us against 6.7 + 4.8 for one token and 6 experts of 2048x1280, 107
// against 65 + 6 for 16 tokens and 128 experts.)
__global__ void __launch_bounds__(256) experts_combine(const float *__restrict__ partial, const int32_t *__restrict__ ids,
                                                       const float *__restrict__ weights, int batch, int experts,
                                                       int topk, int hidden, int splits, uint16_t *__restrict__ y)
{
    const int t = blockIdx.y, row = blockIdx.x * 256 + threadIdx.x, lane = threadIdx.x & 63;
    const int64_t pairs = batch * topk;
    const float *p = partial + (int64_t)t * topk * hidden + row;
    const int id = lane < topk ? ids[t * topk + lane] : -1; // lane k: choice k
    const int weight = lane < topk ? __float_as_int(weights[t * topk + lane]) : 0;
    float w[kMaxTopk], sum[kMaxTopk];
#pragma unroll
    for (int k = 0; k < kMaxTopk; ++k) {
        const int e = __builtin_amdgcn_readlane(id, k);
        uint64_t same = __ballot(id == e);
        w[k] = sum[k] = 0.f;
        if (e >= 0 && e < experts && __builtin_ctzll(same) == k) {
            for (int s = 0; s < splits; ++s) sum[k] += p[(s * pairs + k) * hidden];
            for (; same; same &= same - 1) w[k] += __int_as_float(__builtin_amdgcn_readlane(weight, __builtin_ctzll(same)));
        }
    }
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxTopk; ++k) v += w[k] * sum[k];
    y[(int64_t)t * hidden + row] = __builtin_bit_cast(uint16_t, (_Float16)v);
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

sqllm_status check_sizes(int batch, int experts, int topk, int64_t hidden, int64_t inter)
{
    auto width = [](int64_t v) { return v >= kGroupCols && v <= kMaxWidth && v % kGroupCols == 0; };
    if (!width(hidden) || !width(inter)) return SQLLM_ERR_SHAPE;
    if (experts < 1 || experts > kMaxExperts || topk < 1 || topk > kMaxTopk || topk > experts) return SQLLM_ERR_SHAPE;
    if ((int64_t)experts * (hidden > inter ? hidden : inter) >= (int64_t)1 << 30) return SQLLM_ERR_SHAPE;
    if (batch < 1 || batch > kMaxBatch) return SQLLM_ERR_BATCH;
    return SQLLM_OK;
}

int64_t used_at_most(int batch, int experts, int topk) { return batch * topk < experts ? batch * topk : experts; }

// Waves that share a down tile (8 waves to a workgroup): all eight while the
// launch then fits the compute units at once (20 waves each).  Beyond that a
// wave keeps at least three half groups, and fewer waves share a tile while
// there are more than 40 a unit, since each has its expert to find, its table to
// load and its sums to join (us of a call at 8, 4, 2 and 1: 16 tokens, 128
// experts 4096x1536, 3 bits, 173, 151, 145, 139; 8 tokens, 128 experts 2048x768
// 50, 45, 41, 44; 16 tokens, 64 experts 2048x2048, 2 bits, 51, 50, 52, 54; 8
// experts 4096x3584 54, 55, 69, 98).
int down_parts_for(int64_t tiles, int64_t inter)
{
    int p = kDefaultWaves;
    if (tiles * p > 256 * 20)
        while (p > 1 && (inter / 128 < 3 * p || tiles * p > 256 * 40)) p /= 2;
    return p;
}

// Workgroups that share a down tile's columns: more than one only while the
// launch would leave compute units without work and every wave keeps at
// least two half groups (one, two and four splits, us of the whole call: one
// token, 2 of 8 experts 2048x5632 at 4 bits 29.8, 25.3, 24.9; 4 of 60 experts
// 2048x1536 15.9, 16.5, 20.4).
int down_splits(int batch, int experts, int topk, int64_t hidden, int64_t inter)
{
    int s = 1;
    while (s < 8 && used_at_most(batch, experts, topk) * (hidden / 64) * s < 256 && inter / 128 >= 4 * kDefaultWaves * s) s *= 2;
    return s;
}

// Scratch of one call, in this order.
struct Layout {
    size_t logits, act, part, end;
    Layout(int batch, int experts, int topk, int64_t hidden, int64_t inter)
    {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        const size_t pairs = (size_t)batch * topk;
        logits = 0;
        act = up((size_t)batch * experts * 8);
        part = act + up(pairs * inter * 8);
        end = part + up(pairs * hidden * 4 * down_splits(batch, experts, topk, hidden, inter));
    }
};

sqllm_status check_workspace(const void *ws, size_t bytes, size_t need)
{
    return !ws || !aligned(ws, 256) || bytes < need ? SQLLM_ERR_WORKSPACE : SQLLM_OK;
}

sqllm_status check_experts(const sqllm_experts *p)
{
    if (!p || !p->packed || !p->lut) return SQLLM_ERR_NULL;
    if (p->nnz < 0 || p->nnz > INT32_MAX) return SQLLM_ERR_SHAPE;
    if (p->nnz > 0 && (!p->row_ptr || !p->col_idx || !p->val)) return SQLLM_ERR_NULL;
    if (!aligned(p->packed, 16) || !aligned(p->lut, 16)) return SQLLM_ERR_ALIGN;
    if (p->nnz > 0 && (!aligned(p->row_ptr, 4) || !aligned(p->col_idx, 2) || !aligned(p->val, 2))) return SQLLM_ERR_ALIGN;
    return SQLLM_OK;
}

sqllm_status check_route(const uint16_t *x, const uint16_t *router, const float *bias, int flags, const int32_t *ids,
                         const float *weights)
{
    if (!x || !router || !ids || !weights) return SQLLM_ERR_NULL;
    if (flags & ~(SQLLM_MOE_SIGMOID | SQLLM_MOE_KEEP_SUM)) return SQLLM_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return SQLLM_ERR_ALIGN;
    return SQLLM_OK;
}

sqllm_status check_products(const uint16_t *x, const int32_t *ids, const float *weights, const sqllm_experts *gate,
                            const sqllm_experts *up, const sqllm_experts *down, int bits, const uint16_t *y)
{
    if (!x || !ids || !weights || !y) return SQLLM_ERR_NULL;
    if (bits < 2 || bits > 4) return SQLLM_ERR_BITS;
    for (const sqllm_experts *p : {gate, up, down}) {
        const sqllm_status st = check_experts(p);
        if (st != SQLLM_OK) return st;
    }
    if (!aligned(x, 16) || !aligned(y, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return SQLLM_ERR_ALIGN;
    return SQLLM_OK;
}

// experts * hidden up to which one launch routes.  On the GPU one launch takes
// longer, since a token's workgroup reads the whole router through one compute
// unit's loads (8 experts of 4096: 5.3 us against 4.9 in two launches, 64 of
// 2048 7.3 against 4.2, 64 of 4096 11.6 against 5.0), but the second launch
// costs the host about 3.6 us, which is what bounds small layers.
constexpr int64_t kRouteSmall = 131072;

sqllm_status launched() { return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP; }

sqllm_status route(const uint16_t *x, const uint16_t *router, const float *bias, int batch, int experts,
                   int64_t hidden, int topk, int flags, float scale, int32_t *ids, float *weights, const Layout &at,
                   char *ws, hipStream_t stream)
{
    const int n = (experts + 63) / 64; // experts per lane of the choosing wave
    if ((int64_t)experts * hidden <= kRouteSmall) {
        auto kern = n == 1 ? route_small<1> : n == 2 ? route_small<2> : n <= 4 ? route_small<4> : route_small<8>;
        hipLaunchKernelGGL(kern, dim3(batch), dim3(64 * kRouteWaves), 0, stream, x, router, bias, (int)hidden, experts,
                           topk, flags, scale, ids, weights);
        return launched();
    }
    double *logits = (double *)(ws + at.logits);
    if (batch == 1)
        hipLaunchKernelGGL((route_logits<1>), dim3((experts + 3) / 4, 1), dim3(256), 0, stream, x, router, (int)hidden,
                           experts, batch, logits);
    else
        hipLaunchKernelGGL((route_logits<2>), dim3((experts + 3) / 4, (batch + 1) / 2), dim3(256), 0, stream, x, router,
                           (int)hidden, experts, batch, logits);
    auto kern = n == 1 ? route_choose<1> : n == 2 ? route_choose<2> : n <= 4 ? route_choose<4> : route_choose<8>;
    hipLaunchKernelGGL(kern, dim3(batch), dim3(64), 0, stream, logits, bias, experts, topk, flags, scale, ids, weights);
    return launched();
}

Projection projection(const sqllm_experts &p)
{
    return {(const uint8_t *)p.packed, p.lut, p.row_ptr, p.col_idx, p.val, p.nnz};
}

// 64 KB (16 tokens, 8 experts 4096x3584 at 4 bits: 70 us a call against 75
// with 32 KB, where fewer experts' tokens fit, and 76 gathering from memory;
// 16 tokens, 128 experts 4096x1536: 146, 147 and 150).
constexpr int64_t kStageRoom = 64 << 10;

// Which decode the products take: pair tables for gate and up at 4 bits from
// 1024 columns on (us of a call with registers and with tables: 8 tokens, 128
// experts 2048x768 52 and 44, 64 experts 1024x2048 41.4 and 40.5, 512x2048 28.6
// and 29.0; one token, 2 of 8 experts 4096x11008 60 and 47; at 3 bits 42 and
// 42, 16 tokens, 128 experts 4096x1536 161 and 162, one token 4096x2048 23 and
// 26) ...
bool gate_by_table(int hidden) { return hidden >= 1024; }

// ... and for down at 3 and 4 bits where eight waves share a tile anyway or
// have 2048 columns (one token, 6 of 64 experts 2048x1280 at 3 bits 20.1 and
// 18.7, 4 of 64 1024x2048 34 and 31 with 8 tokens, 8 of 8 4096x14336 108 and
// 101, at 4 bits 141 and 116; but 128 experts 4096x1536 161 and 172, 2048x768
// 36 and 39, at 4 bits 190 and 192, 44 and 46).
bool down_by_table(int parts, int cols) { return parts == kDefaultWaves || cols >= 2048; }

template <int BITS, int MAXQ>
sqllm_status products(const uint16_t *x, const int32_t *ids, const float *weights, const Projection &gate,
                      const Projection &up, const Projection &down, int batch, int experts, int topk, int hidden,
                      int inter, uint16_t *y, const Layout &at, char *ws, hipStream_t stream)
{
    const size_t entries = (size_t)batch * topk * inter;
    const Activations a = {(uint16_t *)(ws + at.act), (uint16_t *)(ws + at.act) + entries,
                           (float *)(ws + at.act + 4 * entries)};
    float *part = (float *)(ws + at.part);
    const int used = (int)used_at_most(batch, experts, topk), splits = down_splits(batch, experts, topk, hidden, inter);
    // LDS of a workgroup: the waves' sums, or before that its tokens' activations
    // for the outliers to gather from, if these take at most kStageRoom (two
    // workgroups share a compute unit)
    const size_t red = (size_t)kDefaultWaves * 4 * MAXQ * 64 * sizeof(float);
    auto space = [&](int64_t stage) { return std::max(red, (size_t)std::min(stage, kStageRoom)); };
    const size_t gate_lds = space(gate.nnz + up.nnz > 0 ? (int64_t)batch * hidden * 2 : 0);
    const size_t down_lds = space(down.nnz > 0 ? (int64_t)batch * inter * 4 : 0);
    const int down_parts = down_parts_for((int64_t)used * (hidden / 64) * splits, inter / splits);
    const int down_wgs = (hidden / 64 * down_parts + kDefaultWaves - 1) / kDefaultWaves;
    const dim3 threads(64 * kDefaultWaves);
    bool by_table = false;
    if constexpr (BITS == 4) {
        if ((by_table = gate_by_table(hidden))) {
            const int lds = (int)std::max((size_t)kPairTable<BITS>, gate_lds);
            static std::atomic<uint64_t> asked{0};
            dev::raise_lds_limit((const void *)experts_gate_up_table<MAXQ>, asked, (int)kStageRoom);
            hipLaunchKernelGGL((experts_gate_up_table<MAXQ>), dim3(inter / 64, used), threads, lds, stream, gate, up, x,
                               ids, batch, experts, topk, hidden, inter, lds, a);
        }
    }
    if (!by_table) {
        static std::atomic<uint64_t> asked{0};
        dev::raise_lds_limit((const void *)experts_gate_up<BITS, MAXQ>, asked, (int)kStageRoom);
        hipLaunchKernelGGL((experts_gate_up<BITS, MAXQ>), dim3(inter / 64, used), threads, gate_lds, stream, gate, up, x, ids,
                           batch, experts, topk, hidden, inter, (int)gate_lds, a);
    }
    by_table = false;
    if constexpr (BITS > 2) {
        if ((by_table = down_by_table(down_parts, inter / splits))) {
            const int lds = (int)std::max((size_t)kPairTable<BITS>, down_lds);
            static std::atomic<uint64_t> asked{0};
            dev::raise_lds_limit((const void *)experts_down_table<BITS, MAXQ>, asked, (int)kStageRoom);
            hipLaunchKernelGGL((experts_down_table<BITS, MAXQ>), dim3(hidden / 64, used, splits), threads, lds, stream, down, a,
                               ids, batch, experts, topk, hidden, inter, lds, part);
        }
    }
    if (!by_table) {
        static std::atomic<uint64_t> asked{0};
        dev::raise_lds_limit((const void *)experts_down<BITS, MAXQ>, asked, (int)kStageRoom);
        hipLaunchKernelGGL((experts_down<BITS, MAXQ>), dim3(down_wgs, used, splits), threads, down_lds, stream, down, a, ids,
                           batch, experts, topk, hidden, inter, __builtin_ctz(down_parts), (int)down_lds, part);
    }
    hipLaunchKernelGGL(experts_combine, dim3(hidden / 256, batch), dim3(256), 0, stream, part, ids, weights, batch,
                       experts, topk, hidden, splits, y);
    return launched();
}

sqllm_status products_of(int bits, const uint16_t *x, const int32_t *ids, const float *weights,
                         const sqllm_experts *gate, const sqllm_experts *up, const sqllm_experts *down, int batch,
                         int experts, int topk, int64_t hidden, int64_t inter, uint16_t *y, const Layout &at, char *ws,
                         hipStream_t stream)
{
    const int q = batch > 8 ? 2 : batch > 4 ? 1 : 0;
    decltype(&products<2, 1>) of[3][3] = {{products<2, 1>, products<2, 2>, products<2, 4>},
                                          {products<3, 1>, products<3, 2>, products<3, 4>},
                                          {products<4, 1>, products<4, 2>, products<4, 4>}};
    auto run = of[bits - 2][q];
    return run(x, ids, weights, projection(*gate), projection(*up), projection(*down), batch, experts, topk,
               (int)hidden, (int)inter, y, at, ws, stream);
}

} // namespace

extern "C" size_t sqllm_moe_workspace_bytes(int batch, int experts, int topk, int64_t hidden, int64_t inter)
{
    if (check_sizes(batch, experts, topk, hidden, inter) != SQLLM_OK) return 0;
    return Layout(batch, experts, topk, hidden, inter).end;
}

extern "C" sqllm_status sqllm_moe_route(const uint16_t *x, const uint16_t *router, const float *bias, int batch,
                                        int experts, int64_t hidden, int topk, int flags, float scale, int32_t *ids,
                                        float *weights, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    sqllm_status st = check_route(x, router, bias, flags, ids, weights);
    if (st == SQLLM_OK) st = check_sizes(batch, experts, topk, hidden, kGroupCols);
    if (st != SQLLM_OK) return st;
    const Layout at(batch, experts, topk, hidden, kGroupCols);
    st = check_workspace(workspace, workspace_bytes, at.end);
    if (st != SQLLM_OK) return st;
    return route(x, router, bias, batch, experts, hidden, topk, flags, scale, ids, weights, at, (char *)workspace,
                 stream);
}

extern "C" sqllm_status sqllm_moe_experts(const uint16_t *x, const int32_t *ids, const float *weights,
                                          const sqllm_experts *gate, const sqllm_experts *up,
                                          const sqllm_experts *down, int bits, int batch, int experts, int topk,
                                          int64_t hidden, int64_t inter, uint16_t *y, void *workspace,
                                          size_t workspace_bytes, hipStream_t stream)
{
    sqllm_status st = check_products(x, ids, weights, gate, up, down, bits, y);
    if (st == SQLLM_OK) st = check_sizes(batch, experts, topk, hidden, inter);
    if (st != SQLLM_OK) return st;
    const Layout at(batch, experts, topk, hidden, inter);
    st = check_workspace(workspace, workspace_bytes, at.end);
    if (st != SQLLM_OK) return st;
    return products_of(bits, x, ids, weights, gate, up, down, batch, experts, topk, hidden, inter, y, at,
                       (char *)workspace, stream);
}

extern "C" sqllm_status sqllm_moe_layer(const uint16_t *x, const uint16_t *router, const float *bias, int flags,
                                        float scale, const sqllm_experts *gate, const sqllm_experts *up,
                                        const sqllm_experts *down, int bits, int batch, int experts, int topk,
                                        int64_t hidden, int64_t inter, int32_t *ids, float *weights, uint16_t *y,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    sqllm_status st = check_route(x, router, bias, flags, ids, weights);
    if (st == SQLLM_OK) st = check_products(x, ids, weights, gate, up, down, bits, y);
    if (st == SQLLM_OK) st = check_sizes(batch, experts, topk, hidden, inter);
    if (st != SQLLM_OK) return st;
    const Layout at(batch, experts, topk, hidden, inter);
    st = check_workspace(workspace, workspace_bytes, at.end);
    if (st != SQLLM_OK) return st;
    st = route(x, router, bias, batch, experts, hidden, topk, flags, scale, ids, weights, at, (char *)workspace, stream);
    if (st != SQLLM_OK) return st;
    return products_of(bits, x, ids, weights, gate, up, down, batch, experts, topk, hidden, inter, y, at,
                       (char *)workspace, stream);
}
