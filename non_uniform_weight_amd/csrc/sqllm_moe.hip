// sqllm_moe.hip -- the mixture-of-experts layer of include/sqllm_moe.h:
// argument checks, workspace layout, kernels and launches.
//
// One call is a chain of small launches on the caller's stream: the router's
// sums and choice, gate and up with the activation, down, and the weighted
// sum over a token's experts.  Nothing is read back by the host: every
// workgroup finds its expert and tokens from ids[] itself.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sqllm_internal.h"
#include "sqllm_moe.h"

using namespace sqllm;

namespace {

constexpr int kMaxExperts = SQLLM_MOE_MAX_EXPERTS;
constexpr int kMaxTopk = SQLLM_MOE_MAX_TOPK;
constexpr int64_t kMaxWidth = 65536; // hidden, inter: 16-bit columns of the outliers

// ---------------------------------------------------------------------------
// Router.
// ---------------------------------------------------------------------------

// logits[t][e], one wave each, in 64 bits: a product of two fp16 values is
// exact in fp32, and 64-bit sums of at most 2^16 of them are off by less
// than 2^-37 of the largest partial sum, so the choice below does not
// depend on the order they are taken in.
__global__ void __launch_bounds__(64) route_logits(const uint16_t *__restrict__ x, const uint16_t *__restrict__ router,
                                                   int hidden, int experts, double *__restrict__ logits)
{
    const int e = blockIdx.x, t = blockIdx.y, lane = threadIdx.x;
    const _Float16 *xr = (const _Float16 *)x + (int64_t)t * hidden, *wr = (const _Float16 *)router + (int64_t)e * hidden;
    double acc = 0.0;
    for (int c = lane; c < hidden; c += 64) acc += (double)((float)xr[c] * (float)wr[c]);
    for (int m = 32; m; m >>= 1) acc += __shfl_xor(acc, m);
    if (lane == 0) logits[(int64_t)t * experts + e] = acc;
}

// A double's place in ascending order as an unsigned number; NaN is 0, below
// -infinity, and -0 counts as +0.
__device__ __forceinline__ uint64_t order_key(double v)
{
    if (v != v) return 0;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// One wave per token; lane l holds experts l, l + 64, ...  Each of the topk
// rounds takes the largest key left (ties: the lowest expert).
__global__ void __launch_bounds__(64) route_select(const double *__restrict__ logits, const float *__restrict__ bias,
                                                   int experts, int topk, int flags, float scale,
                                                   int32_t *__restrict__ ids, float *__restrict__ weights)
{
    constexpr int N = kMaxExperts / 64;
    const int t = blockIdx.x, lane = threadIdx.x;
    double s[N];
    uint64_t key[N];
    if (flags & SQLLM_MOE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 64 * j;
            s[j] = e < experts ? 1.0 / (1.0 + exp(-logits[(int64_t)t * experts + e])) : 0.0;
        }
    } else {
        double top = -__builtin_inf(), sum = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 64 * j;
            s[j] = e < experts ? logits[(int64_t)t * experts + e] : -__builtin_inf();
            top = fmax(top, s[j]);
        }
        for (int m = 32; m; m >>= 1) top = fmax(top, __shfl_xor(top, m));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            s[j] = lane + 64 * j < experts ? exp(s[j] - top) : 0.0;
            sum += s[j];
        }
        for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] /= sum;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 64 * j;
        key[j] = e < experts ? order_key(bias ? s[j] + (double)bias[e] : s[j]) : 0;
    }
    int taken = 0; // bit j: this lane's expert j is chosen already
    double kept[kMaxTopk], sum = 0.0;
    for (int k = 0; k < topk; ++k) {
        uint64_t best = 0;
        int at = INT32_MAX;
        double sc = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 64 * j;
            if (e < experts && !((taken >> j) & 1) && (at == INT32_MAX || key[j] > best)) best = key[j], at = e, sc = s[j];
        }
        for (int m = 32; m; m >>= 1) {
            const uint64_t ob = __shfl_xor((unsigned long long)best, m);
            const int oa = __shfl_xor(at, m);
            const double os = __shfl_xor(sc, m);
            if (oa != INT32_MAX && (at == INT32_MAX || ob > best || (ob == best && oa < at))) best = ob, at = oa, sc = os;
        }
        if ((at & 63) == lane) taken |= 1 << (at >> 6);
#pragma unroll
        for (int q = 0; q < kMaxTopk; ++q)
            if (q == k) kept[q] = sc;
        sum += sc;
        if (lane == 0) ids[t * topk + k] = at;
    }
    if (lane == 0) {
        const double f = flags & SQLLM_MOE_KEEP_SUM ? (double)scale : (double)scale / sum;
#pragma unroll
        for (int k = 0; k < kMaxTopk; ++k)
            if (k < topk) weights[t * topk + k] = (float)(kept[k] * f);
    }
}

// ---------------------------------------------------------------------------
// Experts.
// ---------------------------------------------------------------------------

struct Projection {
    const uint8_t *packed;
    const uint16_t *lut;
    const int32_t *row_ptr;
    const uint16_t *col;
    const uint16_t *val;
    int64_t nnz;
};

template <int BITS>
__device__ __forceinline__ int code_of(const uint8_t *s, int c) // code c (0..255) of a group whose piece q is at s + 1024 q
{
    auto byte = [&](int i) { return (int)s[(i >> 4) * 1024 + (i & 15)]; };
    const int p = c >> 1, hi = c & 1;
    if constexpr (BITS == 4) return (byte(p) >> (4 * hi)) & 15;
    if constexpr (BITS == 2) return (byte(p >> 1) >> (4 * (p & 1) + 2 * hi)) & 3;
    const int u = p >> 4, q = p & 15;
    int v;
    if (q < 12)
        v = byte(12 * u + q) & 63;
    else
        v = (byte(12 * u + q - 12) >> 6) | (byte(12 * u + 4 + q - 12) >> 6) << 2 | (byte(12 * u + 8 + q - 12) >> 6) << 4;
    return (v >> (3 * hi)) & 7;
}

// Row `row` of expert e's matrix times v (fp16 or fp32), fp32.
template <int BITS, typename V>
__device__ __forceinline__ float row_product(const Projection &p, int e, int row, int rows, int cols, const V *v)
{
    const int lane = row & 63, groups = cols >> 8;
    const int64_t at = (int64_t)e * rows + row;
    const uint16_t *lut = p.lut + (at << BITS);
    const uint8_t *base = p.packed + ((int64_t)e * (rows >> 6) + (row >> 6)) * groups * (2 * BITS * 1024) + lane * 16;
    float acc = 0.f;
    for (int g = 0; g < groups; ++g)
        for (int c = 0; c < 256; ++c) {
            const int k = code_of<BITS>(base + (int64_t)g * (2 * BITS * 1024), c);
            acc += (float)__builtin_bit_cast(_Float16, lut[k]) * (float)v[g * 256 + c];
        }
    if (p.nnz)
        for (int i = p.row_ptr[at]; i < p.row_ptr[at + 1]; ++i)
            acc += (float)__builtin_bit_cast(_Float16, p.val[i]) * (float)v[p.col[i]];
    return acc;
}

// a[pair][inter]: gate and up of one 64-row tile for one (token, choice).
template <int BITS>
__global__ void __launch_bounds__(64) experts_gate_up(Projection gate, Projection up, const uint16_t *x,
                                                      const int32_t *ids, int experts, int topk, int hidden, int inter,
                                                      float *a)
{
    const int pair = blockIdx.y, row = blockIdx.x * 64 + threadIdx.x, e = ids[pair];
    if (e < 0 || e >= experts) return;
    const _Float16 *v = (const _Float16 *)x + (int64_t)(pair / topk) * hidden;
    const float g = row_product<BITS>(gate, e, row, inter, hidden, v);
    const float u = row_product<BITS>(up, e, row, inter, hidden, v);
    a[(int64_t)pair * inter + row] = g / (1.f + __expf(-g)) * u;
}

template <int BITS>
__global__ void __launch_bounds__(64) experts_down(Projection down, const float *a, const int32_t *ids,
                                                   const float *weights, int experts, int topk, int hidden, int inter,
                                                   uint16_t *y)
{
    const int t = blockIdx.y, row = blockIdx.x * 64 + threadIdx.x;
    float sum = 0.f;
    for (int k = 0; k < topk; ++k) {
        const int pair = t * topk + k, e = ids[pair];
        if (e < 0 || e >= experts) continue;
        sum += weights[pair] * row_product<BITS>(down, e, row, hidden, inter, a + (int64_t)pair * inter);
    }
    y[(int64_t)t * hidden + row] = __builtin_bit_cast(uint16_t, (_Float16)sum);
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

// Scratch of one call, in this order.
struct Layout {
    size_t logits, act, end;
    Layout(int batch, int experts, int topk, int64_t inter)
    {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        logits = 0;
        act = up((size_t)batch * experts * 8);
        end = act + up((size_t)batch * topk * inter * 4);
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

sqllm_status launched() { return hipGetLastError() == hipSuccess ? SQLLM_OK : SQLLM_ERR_HIP; }

sqllm_status route(const uint16_t *x, const uint16_t *router, const float *bias, int batch, int experts,
                   int64_t hidden, int topk, int flags, float scale, int32_t *ids, float *weights, const Layout &at,
                   char *ws, hipStream_t stream)
{
    double *logits = (double *)(ws + at.logits);
    hipLaunchKernelGGL(route_logits, dim3(experts, batch), dim3(64), 0, stream, x, router, (int)hidden, experts, logits);
    hipLaunchKernelGGL(route_select, dim3(batch), dim3(64), 0, stream, logits, bias, experts, topk, flags, scale, ids,
                       weights);
    return launched();
}

Projection projection(const sqllm_experts &p)
{
    return {(const uint8_t *)p.packed, p.lut, p.row_ptr, p.col_idx, p.val, p.nnz};
}

template <int BITS>
sqllm_status products(const uint16_t *x, const int32_t *ids, const float *weights, const Projection &gate,
                      const Projection &up, const Projection &down, int batch, int experts, int topk, int hidden,
                      int inter, uint16_t *y, const Layout &at, char *ws, hipStream_t stream)
{
    float *a = (float *)(ws + at.act);
    hipLaunchKernelGGL((experts_gate_up<BITS>), dim3(inter / 64, batch * topk), dim3(64), 0, stream, gate, up, x, ids,
                       experts, topk, hidden, inter, a);
    hipLaunchKernelGGL((experts_down<BITS>), dim3(hidden / 64, batch), dim3(64), 0, stream, down, a, ids, weights,
                       experts, topk, hidden, inter, y);
    return launched();
}

sqllm_status products_of(int bits, const uint16_t *x, const int32_t *ids, const float *weights,
                         const sqllm_experts *gate, const sqllm_experts *up, const sqllm_experts *down, int batch,
                         int experts, int topk, int64_t hidden, int64_t inter, uint16_t *y, const Layout &at, char *ws,
                         hipStream_t stream)
{
    auto run = bits == 2 ? products<2> : bits == 3 ? products<3> : products<4>;
    return run(x, ids, weights, projection(*gate), projection(*up), projection(*down), batch, experts, topk,
               (int)hidden, (int)inter, y, at, ws, stream);
}

} // namespace

extern "C" size_t sqllm_moe_workspace_bytes(int batch, int experts, int topk, int64_t hidden, int64_t inter)
{
    if (check_sizes(batch, experts, topk, hidden, inter) != SQLLM_OK) return 0;
    return Layout(batch, experts, topk, inter).end;
}

extern "C" sqllm_status sqllm_moe_route(const uint16_t *x, const uint16_t *router, const float *bias, int batch,
                                        int experts, int64_t hidden, int topk, int flags, float scale, int32_t *ids,
                                        float *weights, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    sqllm_status st = check_route(x, router, bias, flags, ids, weights);
    if (st == SQLLM_OK) st = check_sizes(batch, experts, topk, hidden, kGroupCols);
    if (st != SQLLM_OK) return st;
    const Layout at(batch, experts, topk, kGroupCols);
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
    const Layout at(batch, experts, topk, inter);
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
    const Layout at(batch, experts, topk, inter);
    st = check_workspace(workspace, workspace_bytes, at.end);
    if (st != SQLLM_OK) return st;
    st = route(x, router, bias, batch, experts, hidden, topk, flags, scale, ids, weights, at, (char *)workspace, stream);
    if (st != SQLLM_OK) return st;
    return products_of(bits, x, ids, weights, gate, up, down, batch, experts, topk, hidden, inter, y, at,
                       (char *)workspace, stream);
}
