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
template <typename T>
QG_DEV_INLINE bool before(T a, int i, T b, int j) { return a > b || (a == b && i < j); }

constexpr float kInf = __builtin_huge_valf();

// The groups that stay, from the keys of the warp's token in shared memory (an expert that is not
// available: -inf): a bit each.  `margin`: the least value that stays less the largest that goes.
template <typename T>
QG_DEV_INLINE uint32_t kept_groups(const T* key, const RouteParams& p, int lane, T* margin)
{
    const int size = p.E / p.n_group;
    // `sub` lanes a group (32 over n_group rounded up to a power of two), each every sub-th
    // expert; the lanes start apart, so that groups of 32 do not meet in a bank
    const int log = p.n_group > 1 ? 32 - __clz(p.n_group - 1) : 0, sub = 32 >> log, g = lane >> (5 - log);
    T a = -kInf, b = -kInf;
    if (g < p.n_group) {
        int i = lane % size;
        const int own = lane & (sub - 1);
        for (int n = own; n < size; n += sub) {
            const T x = key[g * size + i];
            if (x > a) { b = a; a = x; }
            else if (x > b) b = x;
            i += sub;
            while (i >= size) i -= size;
        }
    }
    for (int o = 1; o < sub; o <<= 1) {
        const T a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
        b = a > a2 ? (b > a2 ? b : a2) : (a > b2 ? a : b2);
        a = a > a2 ? a : a2;
    }
    T top = p.group_top == 2 && size > 1 ? a + b : a;
    top = __shfl_sync(0xffffffffu, top, (lane << (5 - log)) & 31);   // lane g: group g's value
    if (lane >= p.n_group) top = -kInf;
    int rank = 0;   // groups that come before this one
    for (int g = 0; g < p.n_group; ++g) rank += before(__shfl_sync(0xffffffffu, top, g), g, top, lane);
    const bool in = lane < p.n_group && rank < p.topk_group;
    const uint32_t last = __ballot_sync(0xffffffffu, lane < p.n_group && rank == p.topk_group - 1);
    const uint32_t next = __ballot_sync(0xffffffffu, lane < p.n_group && rank == p.topk_group);
    const T lo = __shfl_sync(0xffffffffu, top, __ffs(last) - 1);
    *margin = next ? lo - __shfl_sync(0xffffffffu, top, __ffs(next) - 1) : (T)kInf;
    if (*margin != *margin) *margin = 0;   // both -inf
    return __ballot_sync(0xffffffffu, in);
}

// One token by one warp, straight from the definition: scores and keys in binary64 (which of
// two nearly equal experts comes first is decided by the formula and not by rounding).  Lane l
// holds experts l, l + 32, ..  mx: the largest logit; `bad`: the token goes nowhere.
template <int T, int VPL>
__device__ __noinline__ void route_exact(const RouteParams& p, float mx, bool bad, double* skey, int m, int lane)
{
    const int E = p.E;
    const bool any = mx > -kInf;
    float x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] = lane + 32 * v < E ? load_logit<T>(p.logits, (int64_t)m * E + lane + 32 * v) : -kInf;
    double score[VPL], key[VPL], sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        score[v] = !any ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[v])) : exp((double)x[v] - (double)mx);
        sum += score[v];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane + 32 * v;
        if (!p.sigmoid && any) score[v] /= sum;
        key[v] = bad || !(x[v] > -kInf) ? -kInf : score[v] + (p.bias && e < E ? (double)p.bias[e] : 0.0);
    }
    if (p.n_group > 1) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v < E) skey[lane + 32 * v] = key[v];
        __syncwarp();
        double margin;
        const uint32_t kept = kept_groups(skey, p, lane, &margin);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane + 32 * v;
            if (e < E && !(kept >> (e / (E / p.n_group)) & 1u)) key[v] = -kInf;
        }
        __syncwarp();
    }
    unsigned long long u[VPL];   // the keys as integers of the same order; 0: not available
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const unsigned long long bits = __double_as_longlong(key[v] + 0.0);   // -0 is 0
        u[v] = key[v] > -kInf ? bits ^ ((bits >> 63) ? ~0ull : 1ull << 63) : 0ull;
    }
    double total = 0.0, wj = 0.0;
    int ej = -1;   // lane j keeps choice j
    for (int j = 0; j < p.topk; ++j) {
        unsigned long long best = u[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) best = max(best, u[v]);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        best = (unsigned long long)hi << 32 | lo;
        if (best == 0ull) break;
        int i = kMaxExperts;   // the lowest expert of that key
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v)
            if (u[v] == best) i = lane + 32 * v;
        i = __reduce_min_sync(0xffffffffu, i);
        double sc = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v == i) {
                sc = score[v];
                u[v] = 0ull;
            }
        sc = __shfl_sync(0xffffffffu, sc, i & 31);
        total += sc;
        if (lane == j) { ej = i; wj = sc; }
    }
    if (lane < p.topk) {
        if (p.renorm) wj = total > 0.0 ? wj / total : 0.0;
        p.idx[(int64_t)m * p.topk + lane] = ej;
        p.weights[(int64_t)m * p.topk + lane] = (float)(wj * (double)p.scale);
    }
}

// fp32 keys as integers of the same order; 0: not available
QG_DEV_INLINE uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 is 0
    return x > -kInf ? b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
}
QG_DEV_INLINE float unordered(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// One warp per token.  Without a bias the choice is by the logits (both scores rise with them);
// with one, and for groups, by fp32 keys.  Where fp32 cannot tell an order that binary64 decides
// -- two keys, or the last group kept and the first dropped, nearer than the keys' error;
// logits that binary64 scores cannot tell apart (saturated, or nearer than 2^-40) -- the token
// is done again by route_exact: about one in two hundred of 256 experts with a bias.
// The weights of the chosen are binary64 values, one lane each, rounded once (0.2 to 1 us of the times below).
// Bound by the choice: 8 + 1 dependent rounds of a maximum over the warp (16384 x 256, top 8: 25 us
// plain softmax, 46 us with bias and groups, of which 11 us for the second looks; the logits
// alone take 1.3 us of HBM).
template <int T, int VPL>
__global__ void __launch_bounds__(128) route_topk_kernel(const RouteParams p)
{
    __shared__ double skey[4][kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.x * 4 + warp;
    if (m >= p.M) return;
    const int E = p.E;
    float x[VPL], key[VPL], mx = -kInf;
    bool bad = false;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = lane + 32 * v;
        x[v] = e < E ? load_logit<T>(p.logits, (int64_t)m * E + e) : -kInf;
        bad |= !(x[v] < kInf);
        mx = fmaxf(mx, x[v]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (p.bias) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane + 32 * v;
            const float b = e < E ? __ldg(p.bias + e) : 0.0f;
            bad |= x[v] > -kInf && !(b < kInf);
            key[v] = b;
        }
    }
    if (__any_sync(0xffffffffu, bad)) {   // the token goes nowhere
        if (lane == 0) set_status(5u);
        route_exact<T, VPL>(p, -kInf, true, skey[warp], m, lane);
        return;
    }
    // fp32 scores, where they are needed: each is within 2^-20 of its value
    const bool scores = p.bias || p.n_group > 1;
    if (scores) {
        float sc[VPL];
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            sc[v] = p.sigmoid ? __frcp_rn(1.0f + expf(-x[v])) : mx > -kInf ? expf(x[v] - mx) : 0.0f;
            if (!p.sigmoid) sum += sc[v];
        }
        float inv = 1.0f;
        if (!p.sigmoid) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            inv = sum > 0.0 ? 1.0f / (float)sum : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = fmaf(sc[v], inv, p.bias ? key[v] : 0.0f);
    }
    float far = 1.0f;   // the keys' largest magnitude
    if (scores) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            if (!(x[v] > -kInf)) key[v] = -kInf;
            if (key[v] > -kInf) far = fmaxf(far, fabsf(key[v]));
        }
        far = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(far)));
    }
    // two keys nearer than this may be the other way round: a score is within 2^-21 (expf, the sum
    // and the quotient, each a few 2^-24 of at most 1), a key within 2^-24 of itself more
    const float near = 0x1p-19f * far;
    bool again = p.sigmoid && mx > 16.0f;
    uint32_t u[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) u[v] = ordered(p.bias ? key[v] : x[v]);
    if (p.n_group > 1) {
        float* fkey = reinterpret_cast<float*>(skey[warp]);
        __syncwarp();
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v < E) fkey[lane + 32 * v] = key[v];
        __syncwarp();
        float margin;
        const uint32_t kept = kept_groups(fkey, p, lane, &margin);
        again |= margin <= 2.0f * near;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane + 32 * v;
            if (e < E && !(kept >> (e / (E / p.n_group)) & 1u)) u[v] = 0u;
        }
        __syncwarp();
    }
    int ej = -1;   // lane j keeps choice j
    uint32_t prev = 0u;
    for (int j = 0; j <= p.topk && !again; ++j) {   // one further, to see how near it is
        uint32_t best = u[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) best = max(best, u[v]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (j > 0 && best > 0u) {
            const float gap = unordered(prev) - unordered(best);
            again = p.bias ? gap <= near : gap > 0.0f && gap < 0x1p-40f;
        }
        if (best == 0u || j == p.topk) break;
        // the lowest expert of that key
        int i = kMaxExperts;
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v)
            if (u[v] == best) i = lane + 32 * v;
        const uint32_t who = __ballot_sync(0xffffffffu, i < kMaxExperts);
        i = (who & (who - 1u)) ? __reduce_min_sync(0xffffffffu, i) : __shfl_sync(0xffffffffu, i, __ffs(who) - 1);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + 32 * v == i) u[v] = 0u;
        if (lane == j) ej = i;
        prev = best;
    }
    const float xj = ej >= 0 ? load_logit<T>(p.logits, (int64_t)m * E + ej) : -kInf;
    // scores that are small for fp32 (and their sum), or 0 in binary64
    again |= __any_sync(0xffffffffu, ej >= 0 && (p.sigmoid ? xj : xj - mx) < -60.0f);
    if (again) {
        route_exact<T, VPL>(p, mx, false, skey[warp], m, lane);
        return;
    }
    // the weights in binary64, a lane each, rounded once
    double w = 0.0;
    if (ej >= 0) w = p.sigmoid ? 1.0 / (1.0 + exp(-(double)xj)) : exp((double)xj - (double)mx);
    if (p.renorm) {
        double total = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        w = total > 0.0 ? w / total : 0.0;
    } else if (!p.sigmoid && mx > -kInf) {   // by the sum over all experts
        double sum = 0.0;
        for (int e = lane; e < E; e += 32) sum += exp((double)load_logit<T>(p.logits, (int64_t)m * E + e) - (double)mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w /= sum;
    }
    if (lane < p.topk) {
        p.idx[(int64_t)m * p.topk + lane] = ej;
        p.weights[(int64_t)m * p.topk + lane] = (float)(w * (double)p.scale);
    }
}

// ---------------------------------------------------------------------------
// Slot maps: a stable counting sort of the M * topk choices by expert.  Blocks of kSlotBlock
// choices, 128 for each warp in four rounds: in a round the lanes of equal choices find one
// another (match), so a choice's rank is the warp's count so far plus the lanes before it;
// then the warps' counts are summed up, and the blocks' (slot_count_kernel's, unless there is
// but one).  Latency-bound: a launch and a handful of dependent steps each (16 x 8 choices of 64
// experts 4 us, 131072 of 256 experts 14 us; a scan of the block's choices by each thread and a
// serial sum over the experts took 30 us).
// ---------------------------------------------------------------------------
constexpr int kSlotBlock = 4096, kSlotWarps = 32;
// Up to this many blocks each placing block sums up the others' counts; past it slot_sum_kernel does
// that once for all, so that the work stays linear (256 experts, 32 blocks 15.4 us either way; 64 blocks
// 16.4 us with it, 18.4 without; 512 blocks 44 and 114 us; 4096 blocks 0.27 and 4.3 ms).
constexpr int kSlotSum = 32;

struct SlotParams {
    const int32_t* idx;   // [n]
    int32_t* offsets;     // [E + 1]
    int32_t* slot_token;  // [n]
    int32_t* token_slot;  // [n]
    int32_t* hist;        // [blocks][E]: the blocks' choices of each expert; past kSlotSum blocks one row more
    int n, topk, E, blocks;
};

__global__ void __launch_bounds__(32 * kSlotWarps) slot_count_kernel(const SlotParams p)
{
    __shared__ int cnt[kMaxExperts];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int end = min(p.n, ((int)blockIdx.x + 1) * kSlotBlock);
    for (int i = blockIdx.x * kSlotBlock + threadIdx.x; i < end; i += blockDim.x) {
        const int e = p.idx[i];
        if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[blockIdx.x * p.E + e] = cnt[e];
}

// In place of each block's choices of an expert those of the blocks before it, and all of them in the
// last row.  A warp has 32 experts and a 32nd of the blocks.
__global__ void __launch_bounds__(1024) slot_sum_kernel(const SlotParams p)
{
    __shared__ int part[32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = blockIdx.x * 32 + lane;
    const int per = (p.blocks + 31) / 32, k0 = warp * per, k1 = min(p.blocks, k0 + per);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int n = 0;
    if (x < p.E)
#pragma unroll 8
        for (int k = k0; k < k1; ++k) n += p.hist[k * p.E + x];
    part[warp][lane] = n;
    __syncthreads();
    int run = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
        run += w < warp ? part[w][lane] : 0;
        all += part[w][lane];
    }
    if (x >= p.E) return;
    for (int k = k0; k < k1; k += 8) {
        int c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = k + i < k1 ? p.hist[(k + i) * p.E + x] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (k + i < k1) p.hist[(k + i) * p.E + x] = run;
            run += c[i];
        }
    }
    if (warp == 0) p.hist[p.blocks * p.E + x] = all;
}

__global__ void __launch_bounds__(32 * kSlotWarps) slot_place_kernel(const SlotParams p)
{
    __shared__ uint16_t wcnt[kSlotWarps][kMaxExperts];   // the warps' choices, then those of the warps before
    __shared__ int base[kMaxExperts];                    // this block's first slot of each expert
    __shared__ int total[kMaxExperts];
    __shared__ int used_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i0 = blockIdx.x * kSlotBlock + warp * 128 + lane;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = lane; e < p.E; e += 32) wcnt[warp][e] = 0;
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int e[4], rank[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 32 * r;
        e[r] = i < p.n ? p.idx[i] : -1;
        if ((uint32_t)e[r] >= (uint32_t)p.E) {
            if (e[r] != -1) set_status(6u);   // not an expert: left out, like -1
            e[r] = -1;
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t same = __match_any_sync(0xffffffffu, e[r]);
        const int ahead = __popc(same & ((1u << lane) - 1u));
        rank[r] = 0;
        if (e[r] >= 0) rank[r] = wcnt[warp][e[r]] + ahead;
        __syncwarp();
        if (e[r] >= 0 && ahead == 0) wcnt[warp][e[r]] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int x = threadIdx.x; x < p.E; x += blockDim.x) {
        int n = 0;
#pragma unroll 8
        for (int w = 0; w < kSlotWarps; ++w) {
            const int c = wcnt[w][x];
            wcnt[w][x] = n;
            n += c;
        }
        int b = 0, t = n;
        if (p.blocks > kSlotSum) {
            b = p.hist[blockIdx.x * p.E + x];
            t = p.hist[p.blocks * p.E + x];
        } else if (p.blocks > 1) {
            t = 0;
#pragma unroll 8
            for (int k = 0; k < p.blocks; ++k) {
                const int c = __ldcg(p.hist + k * p.E + x);
                b += k < (int)blockIdx.x ? c : 0;
                t += c;
            }
        }
        base[x] = b;
        total[x] = t;
    }
    __syncthreads();
    if (warp == 0) {   // the experts' first slots
        int run = 0;
        for (int x0 = 0; x0 < p.E; x0 += 32) {
            const int x = x0 + lane, t = x < p.E ? total[x] : 0;
            int v = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += a;
            }
            if (x < p.E) {
                base[x] += run + v - t;
                if (blockIdx.x == 0) p.offsets[x] = run + v - t;
            }
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) {
            used_s = run;
            if (blockIdx.x == 0) p.offsets[p.E] = run;
        }
    }
    __syncthreads();
    const int used = used_s;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 32 * r;
        if (i >= p.n) continue;
        const int slot = e[r] >= 0 ? base[e[r]] + wcnt[warp][e[r]] + rank[r] : -1;
        if (slot >= 0) p.slot_token[slot] = i / p.topk;
        p.token_slot[i] = slot;
        if (i >= used) p.slot_token[i] = -1;   // entries without a choice
    }
}

// Y[m] = rn( sum_j weights[m][j] D[token_slot[m][j]] ), j in order, fp32.  One thread per 8
// columns of a token.  HBM-bound: every slot's row is read once (16384 x 8 x 4096: 207 us, 5.8 TB/s).
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
