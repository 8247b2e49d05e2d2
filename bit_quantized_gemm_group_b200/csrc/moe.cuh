// moe.cuh -- around the experts' products: the router, the slot maps it makes for them and
// the weighted sum that brings their outputs back to the tokens.
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"

namespace qg {

constexpr int kMaxExperts = 512, kMaxTopk = 32, kMaxExpertGroups = 32;

struct RouteParams {
    const void* logits;  // [M][E]
    const float* bias;   // [E] or NULL
    int32_t* idx;        // [M][topk]
    float* weights;      // [M][topk]
    int M, E, topk, n_group, topk_group, group_top;
    bool sigmoid, renorm;
    float scale;
};

template <int T>
QG_DEV_INLINE float load_logit(const void* p, int64_t at)
{
    if (T == IN_F32) return static_cast<const float*>(p)[at];
    const uint32_t b = static_cast<const uint16_t*>(p)[at];
    return half_word<T>(b, 0);
}

// (key, index) order: larger key first, then lower index
QG_DEV_INLINE bool before(double a, int i, double b, int j) { return a > b || (a == b && i < j); }

// One warp per token; lane l holds experts l, l + 32, ..  Scores and keys in binary64: which
// of two nearly equal experts comes first is decided by the formula and not by rounding.
template <int T, int VPL>
__global__ void __launch_bounds__(128) route_topk_kernel(const RouteParams p)
{
    __shared__ double skey[4][kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.x * 4 + warp;
    if (m >= p.M) return;
    const int E = p.E;
    double score[VPL], key[VPL];
    bool bad = false, any = false;
    float mx = -__int_as_float(0x7f800000);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane + 32 * v;
        const float x = e < E ? load_logit<T>(p.logits, (int64_t)m * E + e) : -__int_as_float(0x7f800000);
        bad |= !(x < __int_as_float(0x7f800000));
        any |= x > -__int_as_float(0x7f800000);
        mx = fmaxf(mx, x);
        score[v] = x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    any = __any_sync(0xffffffffu, any);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const double x = score[v];
        key[v] = x;   // -inf stays -inf: not available
        score[v] = !any ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)mx);
        sum += score[v];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const double lowest = -__longlong_as_double(0x7ff0000000000000ll);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane + 32 * v;
        if (!p.sigmoid && any) score[v] /= sum;
        const bool there = key[v] > lowest;
        const double b = p.bias && e < E ? (double)p.bias[e] : 0.0;
        key[v] = there ? score[v] + b : lowest;
        bad |= there && !(key[v] < -lowest);
    }
    if (__any_sync(0xffffffffu, bad)) {   // the token goes nowhere
        if (lane == 0) set_status(5u);
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = lowest;
    }
    if (p.n_group > 1) {
        const int size = E / p.n_group;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v < E) skey[warp][lane + 32 * v] = key[v];
        __syncwarp();
        double top = lowest;   // of group `lane`
        if (lane < p.n_group) {
            double a = lowest, b = lowest;
            for (int i = 0; i < size; ++i) {
                const double x = skey[warp][lane * size + i];
                if (x > a) { b = a; a = x; }
                else if (x > b) b = x;
            }
            top = p.group_top == 2 && size > 1 ? a + b : a;
        }
        int rank = 0;   // groups that come before this one
        for (int g = 0; g < p.n_group; ++g) {
            const double t = __shfl_sync(0xffffffffu, top, g);
            rank += before(t, g, top, lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane + 32 * v;
            if (e < E && !(kept >> (e / size) & 1u)) key[v] = lowest;
        }
    }
    double total = 0.0, wj = 0.0;
    int ej = -1;   // lane j keeps choice j
    for (int j = 0; j < p.topk; ++j) {
        double k = lowest, sc = 0.0;
        int i = kMaxExperts;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (before(key[v], lane + 32 * v, k, i)) { k = key[v]; i = lane + 32 * v; sc = score[v]; }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double k2 = __shfl_xor_sync(0xffffffffu, k, o), s2 = __shfl_xor_sync(0xffffffffu, sc, o);
            const int i2 = __shfl_xor_sync(0xffffffffu, i, o);
            if (before(k2, i2, k, i)) { k = k2; i = i2; sc = s2; }
        }
        const bool there = k > lowest;
        if (!there) { i = -1; sc = 0.0; }
        total += sc;
        if (lane == j) { ej = i; wj = sc; }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v == i) key[v] = lowest;
    }
    if (lane < p.topk) {
        if (p.renorm) wj = total > 0.0 ? wj / total : 0.0;
        p.idx[(int64_t)m * p.topk + lane] = ej;
        p.weights[(int64_t)m * p.topk + lane] = (float)(wj * (double)p.scale);
    }
}

// Slot maps: a counting sort of the M * topk choices by expert, then by token.  Blocks of
// kSlotBlock choices; count: each block's choices per expert (a NULL hist: only block 0's,
// kept in shared memory by place).
constexpr int kSlotBlock = 1024;

struct SlotParams {
    const int32_t* idx;   // [n]
    int32_t* offsets;     // [E + 1]
    int32_t* slot_token;  // [n]
    int32_t* token_slot;  // [n]
    int32_t* hist;        // [blocks][E]
    int n, topk, E, blocks;
};

__global__ void __launch_bounds__(256) slot_count_kernel(const SlotParams p)
{
    __shared__ int cnt[kMaxExperts];
    for (int e = threadIdx.x; e < p.E; e += 256) cnt[e] = 0;
    __syncthreads();
    const int end = min(p.n, ((int)blockIdx.x + 1) * kSlotBlock);
    for (int i = blockIdx.x * kSlotBlock + threadIdx.x; i < end; i += 256) {
        const int e = p.idx[i];
        if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
        else if (e != -1) set_status(6u);   // not an expert: left out, like -1
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += 256) p.hist[blockIdx.x * p.E + e] = cnt[e];
}

__global__ void __launch_bounds__(256) slot_place_kernel(const SlotParams p)
{
    __shared__ int base[kMaxExperts];    // slots before this block's first of each expert
    __shared__ int total[kMaxExperts];
    __shared__ int chunk[kSlotBlock];
    for (int e = threadIdx.x; e < p.E; e += 256) {
        int b = 0, t = 0;
        for (int k = 0; k < p.blocks; ++k) {
            const int c = p.hist[k * p.E + e];
            b += k < (int)blockIdx.x ? c : 0;
            t += c;
        }
        base[e] = b;
        total[e] = t;
    }
    const int i0 = blockIdx.x * kSlotBlock, cnt = min(kSlotBlock, p.n - i0);
    for (int i = threadIdx.x; i < cnt; i += 256) chunk[i] = p.idx[i0 + i];
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        for (int e = 0; e < p.E; ++e) {
            base[e] += at;
            if (blockIdx.x == 0) p.offsets[e] = at;
            at += total[e];
        }
        if (blockIdx.x == 0) p.offsets[p.E] = at;
        total[0] = at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cnt; i += 256) {
        const int e = chunk[i];
        int slot = -1;
        if (e >= 0 && e < p.E) {
            slot = base[e];
            for (int j = 0; j < i; ++j) slot += chunk[j] == e;
            p.slot_token[slot] = (i0 + i) / p.topk;
        }
        p.token_slot[i0 + i] = slot;
    }
    const int used = total[0];   // entries without a choice
    for (int i = i0 + threadIdx.x; i < i0 + cnt; i += 256)
        if (i >= used) p.slot_token[i] = -1;
}

// Y[m] = rn( sum_j weights[m][j] D[token_slot[m][j]] ), j in order, fp32.  One thread per 8
// columns of a token.  HBM-bound: every slot's row is read once.
template <bool BF16>
__global__ void __launch_bounds__(256) combine_experts_kernel(const uint16_t* __restrict__ D, int S, int N, int M,
                                                              int topk, const int32_t* __restrict__ token_slot,
                                                              const float* __restrict__ weights,
                                                              uint16_t* __restrict__ Y)
{
    const int chunks = N / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (int64_t)M * chunks) return;
    const int64_t m = id / chunks;
    const int c = (int)(id - m * chunks) * 8;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j = 0; j < topk; ++j) {
        const int s = token_slot[m * topk + j];
        if (s < 0 || s >= S) {
            if (s != -1 && c == 0) set_status(6u);
            continue;
        }
        const float w = weights[m * topk + j];
        const uint4 x = ldg_stream_v4(D + (int64_t)s * N + c);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = fmaf(w, half_word<BF16 ? IN_BF16 : IN_F16>(u[i], 0), acc[2 * i]);
            acc[2 * i + 1] = fmaf(w, half_word<BF16 ? IN_BF16 : IN_F16>(u[i], 1), acc[2 * i + 1]);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = BF16 ? pack_bf16x2_rn(acc[2 * i], acc[2 * i + 1]) : pack_f16x2_rn(acc[2 * i], acc[2 * i + 1]);
    *reinterpret_cast<uint4*>(Y + m * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace qg
