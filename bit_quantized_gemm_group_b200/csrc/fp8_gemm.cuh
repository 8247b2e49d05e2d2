// fp8_gemm.cuh -- products of e4m3 operands with a scale for each 128 of K, on the tcgen05
// tensor cores:
//
//   Y[m][n] = rn( sum_g (xs[m][g] ws[g][n / 128]) sum_{k in g} Xq[m][k] Wq[k][n] )   (fp32)
//
// and the same per expert over the rows of its slots.  ("AI Infra guide, ch.4
// Quantization" sec. 5, e4m3; "LLM inference cost ..." sec. 2.2, groups of 128.)
//
// The scales change every 128 of K, so the tensor core sums one group at a time (fp32, tensor
// memory) and the epilogue warps fold each group's sums into fp32 registers with one fma,
// acc += P * (xs * ws), while the tensor core works on the next group in another buffer.  The
// weights stay as they are stored, [K][N]: a TMA box of 128 k x 128 columns, 128-byte swizzle, is
// the MMA's MN-major operand.  A dense product is the experts' product with one expert that has
// all the rows.
//
// Every wait is bounded (2 s); one that gives up records QG_ERR_TIMEOUT, and the role
// stops issuing, waits for its own copies and MMAs, and leaves.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "fp8_quant.cuh"

namespace qg {

struct Fp8Params {
    const float* xs;         // [Mx][G]
    const float* ws;         // [E][G][NB]
    const int32_t* rows;     // slot -> row of Xq, or NULL: the slot itself
    const int32_t* offsets;  // [E + 1], or NULL: one expert with all S slots
    uint16_t* Y;             // [S][N]
    int Mx, S, E, K, N, G, NB;
    int join_rows;           // rows of a tile, about
    int box;                 // rows of a TMA box of activations: what a tile can have
    bool bf16;
    // the workspace of split tiles
    unsigned long long* counters;  // [grid]
    float* partials;               // [grid][2][128][BN]
    unsigned long long token;      // this launch's token (its low byte is 0, the rest is not)
};

constexpr int kFp8MaxE = 512;

// D = fp32; A, B = e4m3.  `a_mn`, `b_mn`: the operand is MN-major (else K-major).
__host__ __device__ constexpr uint32_t idesc_e4m3(int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

QG_DEV_INLINE void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accum)
        : "memory");
}

template <int R>
QG_DEV_INLINE void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
QG_DEV_INLINE void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// A bounded wait in a few instructions: kFp8Polls polls, then QG_ERR_TIMEOUT and false.  A poll that
// finds nothing is suspended for 4.0 us (measured, with a hint of 1 us), so that all of them take 2 s.  The waits lie between the steps of loops whose instructions have to stay at hand:
// with mbar_wait's clock and limit inlined in each, a product of 8192 x 8192 x 28672 took 4 % longer.
constexpr uint32_t kFp8Polls = 500000;
QG_DEV_INLINE bool short_wait(uint64_t* bar, uint32_t parity, uint32_t polls = kFp8Polls)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        ".reg .u32 n;\n\t"
        "mov.u32 n, %3;\n\t"
        "POLL:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 p, n, 0;\n\t"
        "@p bra POLL;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(polls)
        : "memory");
    if (!ok) set_status(7u);
    return ok != 0;
}

// One lane of the (converged) warp.  The role loops below run warp-uniform and only the TMA,
// MMA and commit instructions are the elected lane's: the compiler then keeps descriptors in
// uniform registers.  In code that a whole branch gives to one lane an MMA took 110 issue
// cycles (512 cycles of MMA a step became 900 beside the folding warps).
QG_DEV_INLINE bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

QG_DEV_INLINE int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// every lane waits; the result is the warp's
QG_DEV_INLINE bool all_wait(uint64_t* bar, uint32_t parity, uint32_t polls = kFp8Polls)
{
    return __all_sync(0xffffffffu, short_wait(bar, parity, polls));
}

// ---------------------------------------------------------------------------
// Tiles: T rows x (one column slab), numbered expert by expert, slab by slab, rows fastest
// (tiles that share weights are neighbours).
// ---------------------------------------------------------------------------
struct Fp8Sched {
    int off[kFp8MaxE + 1];  // the experts' slots
    int pre[kFp8MaxE + 1];  // tiles before each expert's
};

// All threads of the block.  False: the offsets do not ascend from 0 to at most S.
template <int T>
QG_DEV_INLINE bool fp8_schedule(Fp8Sched& sc, const Fp8Params& p, int slabs)
{
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) sc.off[i] = p.offsets ? p.offsets[i] : i ? p.S : 0;
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x)
        bad |= i == 0 ? sc.off[0] != 0 : sc.off[i] < sc.off[i - 1] || sc.off[i] > p.S;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_status(6u);
        return false;
    }
    if (threadIdx.x < 32) {
        int run = 0;
        if (threadIdx.x == 0) sc.pre[0] = 0;
        for (int b = 0; b < p.E; b += 32) {
            const int e = b + threadIdx.x;
            int v = e < p.E ? (sc.off[e + 1] - sc.off[e] + T - 1) / T * slabs : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if ((int)threadIdx.x >= o) v += u;
            }
            if (e < p.E) sc.pre[e + 1] = run + v;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    return true;
}

template <int T>
struct Fp8Walk {
    const Fp8Sched& sc;
    int E, slabs;
    int e, slab, chunk, chunks;
    QG_DEV_INLINE Fp8Walk(const Fp8Sched& s, int E_, int slabs_) : sc(s), E(E_), slabs(slabs_), e(0), slab(0), chunk(0), chunks(0) {}
    QG_DEV_INLINE void at(int tile)
    {
        int lo = 0, hi = E - 1;   // the last expert whose first tile is at or before this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sc.pre[mid] <= tile) lo = mid;
            else hi = mid - 1;
        }
        e = lo;
        chunks = (sc.off[e + 1] - sc.off[e] + T - 1) / T;
        const int r = tile - sc.pre[e];
        slab = r / chunks;
        chunk = r - slab * chunks;
    }
    QG_DEV_INLINE int first() const { return sc.off[e] + chunk * T; }
    QG_DEV_INLINE int rows() const { return min(T, sc.off[e + 1] - first()); }
};

// The row of Xq that slot s reads; -1 where the map is wrong.  Maps, scales and rows are read with
// plain loads: a kernel that this one started beside may write them until the wait for it, and the
// read-only path (__ldg) is for memory that nothing writes during the whole launch.
QG_DEV_INLINE int fp8_row(const Fp8Params& p, int s)
{
    if (!p.rows) return s;
    const int r = p.rows[s];
    return (uint32_t)r < (uint32_t)p.Mx ? r : -1;
}

template <bool BF16>
QG_DEV_INLINE uint32_t fp8_out2(float a, float b) { return BF16 ? pack_bf16x2_rn(a, b) : pack_f16x2_rn(a, b); }

// acc[0 .. CW) += (CW sums of tensor memory at `addr`) * sc.  Sixteen columns at a time, the next
// ones' load in flight while the ones before are folded; `release` runs once all are read.
template <int CW, typename F>
QG_DEV_INLINE void fp8_fold(float (&acc)[CW], uint32_t addr, float sc, F release)
{
    uint32_t v[2][16];
    tmem_ld_32x32b_x16(addr, v[0]);
#pragma unroll
    for (int c = 0; c < CW; c += 16) {
        uint32_t(&u)[16] = v[(c / 16) & 1];
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 16; ++t) asm volatile("" : "+r"(u[t]));   // read only after the wait
        if (c + 16 < CW) tmem_ld_32x32b_x16(addr + c + 16, v[(c / 16 + 1) & 1]);
        else release();
#pragma unroll
        for (int t = 0; t < 16; ++t) acc[c + t] = fmaf(__uint_as_float(u[t]), sc, acc[c + t]);
    }
}

// ---------------------------------------------------------------------------
// Which tiles, and which groups of K, a CTA takes
//
// Whole waves of tiles go one to a CTA, `grid` apart, so that CTAs running together share
// weights and rows.  Where the tiles left over would leave many CTAs idle, their units (tile,
// group of K) are split evenly over all of them: CTA c takes units
// [c U / eff, (c + 1) U / eff), at most two pieces of tiles.  A split tile is joined by whichever
// of its CTAs arrives last: each leaves its fp32 sums in the workspace and counts itself in; the
// last one adds all of them in CTA order (the result does not depend on who is last) and
// writes Y.  No CTA waits for another.  The counter word holds the launch's token above an
// 8-bit count, so whatever an unused workspace holds reads as 0, and the last arrival clears
// it, so a replayed graph finds it so again.
// ---------------------------------------------------------------------------
// Splitting costs the join: about 11 us for a few rows and 20 us for 128, where a step of 128
// columns takes 0.32 us (256: 0.6), so the longest CTA has to save fp8_min_saved() steps of 128
// columns.  K = 11008, N = 4096, 4 rows (86 steps down to 19): 27.5 us whole, 18.5 split; K = 4096
// (32 down to 7): 11.8 and 13.8 us, left whole; K = 11008 with 128 rows: no difference.
constexpr int kFp8MinUnits = 4;   // of a piece
__host__ __device__ inline int fp8_min_saved(int rows) { return 34 + rows / 4; }

struct Fp8Work {   // in shared memory: the folding threads have no registers to spare
    int G, grid, cta;
    int whole;       // whole tiles of this CTA: cta, cta + grid, ..
    int base;        // the first split tile
    int eff;         // CTAs that take units of split tiles
    int64_t units;   // of all split tiles
    int64_t u0;      // this CTA's: [u0, u0 + n)
    int n;
    // `wide`: columns of a tile over 128; `rows`: of a tile, about
    QG_DEV_INLINE void init(int tiles, int wide, int rows, int G_, int grid_, int cta_)
    {
        G = G_;
        grid = grid_;
        cta = cta_;
        base = tiles;
        eff = n = 0;
        units = u0 = 0;
        const int left = tiles % grid;
        const int parts = left ? (int)min((int64_t)grid, max((int64_t)left, (int64_t)left * G / kFp8MinUnits)) : 1;
        if (left > 0 && (G - (int)((int64_t)left * G / parts)) * wide >= fp8_min_saved(rows)) {
            whole = tiles / grid;
            base = tiles - left;
            units = (int64_t)left * G;
            eff = parts;
            if (cta < eff) {
                u0 = first(cta);
                n = (int)(first(cta + 1) - u0);
            }
        } else {
            whole = cta < tiles ? (tiles - 1 - cta) / grid + 1 : 0;
        }
    }
    QG_DEV_INLINE int64_t first(int c) const { return c * units / eff; }
    QG_DEV_INLINE int cta_of(int64_t u) const
    {
        int c = (int)(u * eff / units);
        while (c > 0 && first(c) > u) --c;
        while (first(c + 1) <= u) ++c;
        return c;
    }
    QG_DEV_INLINE int64_t steps() const { return (int64_t)whole * G + n; }
    // Piece i: groups [k0, k1) of a tile; false: no such piece.
    QG_DEV_INLINE bool piece(int i, int& tile, int& k0, int& k1) const
    {
        if (i < whole) {
            tile = cta + i * grid;
            k0 = 0;
            k1 = G;
            return true;
        }
        if (n == 0) return false;
        const int t = (int)(u0 / G), k = (int)(u0 - (int64_t)t * G), len = min(n, G - k);
        if (i == whole) {
            tile = base + t;
            k0 = k;
            k1 = k + len;
            return true;
        }
        tile = base + t + 1;
        k0 = 0;
        k1 = n - len;
        return i == whole + 1 && k1 > 0;
    }
};

// Counts one arrival of `n` under `token`; true for the last, which clears the word.
QG_DEV_INLINE bool fp8_arrive(unsigned long long* word, unsigned long long token, int n)
{
    unsigned long long old = 0;   // what it holds between launches, mostly
    for (;;) {
        const unsigned long long have = (old & ~0xFFull) == token ? old & 0xFFull : 0ull;
        const bool last = have + 1 == (unsigned long long)n;
        const unsigned long long seen = atomicCAS(word, old, last ? 0ull : token | (have + 1));
        if (seen == old) return last;
        old = seen;
    }
}

// Self-test: each block (a warp) is a piece of one split tile whose wait runs out, on a barrier
// that nothing arrives at, and counts itself in without work.  result: 1 where the wait gave up,
// plus 2 in the piece that arrived last.  No block waits for another.
__global__ void fp8_selftest_wait_kernel(uint32_t polls, unsigned long long* word, unsigned long long token, int32_t* result)
{
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncwarp();
    const bool ok = all_wait(&bar, 0, polls);
    if (threadIdx.x == 0) result[blockIdx.x] = (ok ? 0 : 1) + (fp8_arrive(word, token, gridDim.x) ? 2 : 0);
}

// ---------------------------------------------------------------------------
// The mapped rows in slot order, for the tile kernel (a wrong map entry: row 0, whose sums go
// nowhere).  Four slots and 4 KB of K per CTA, 64 threads a slot.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fp8_rows_kernel(const Fp8Params p, const uint8_t* Xq, uint8_t* xg)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (s >= min(p.offsets[p.E], p.S)) return;
    const uint4* src = reinterpret_cast<const uint4*>(Xq + (int64_t)max(fp8_row(p, s), 0) * p.K);
    uint4* dst = reinterpret_cast<uint4*>(xg + (int64_t)s * p.K);
    const int k0 = blockIdx.y * 256 + (threadIdx.x & 63), end = min(p.K / 16, ((int)blockIdx.y + 1) * 256);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k0 + 64 * i < end) v[i] = src[k0 + 64 * i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k0 + 64 * i < end) dst[k0 + 64 * i] = v[i];
}

// ---------------------------------------------------------------------------
// The product: tiles of 128 rows x BN columns, one group of K a step, persistent.
//
// Roles: warp 0 TMA; warps 1 and 3 issue the MMAs of even and odd steps, into DB buffers; warps
// 4..11 fold: thread = row, BN / 2 columns, whose weight scale is one number, so a step costs a
// thread one scale (which it loads itself, four groups ahead) and BN / 2 fma.
//
// Measured in a graph: 8192 x 8192 x 28672 2.0..2.15 ms (1.8..1.9 PFLOP/s; the fold bounds it, and the
// power cap: 2.2..2.3 ms on normal data); 4096 x 4096 x 4096 74..84 us; 1 x 4096 x 12288 13.6 us
// (3.7 TB/s), 16 x 8192 x 28672 41..44 us (5.3..5.7 TB/s).
// Few rows: the tensor core then multiplies rows that go nowhere, but a step's weights (16 or
// 32 KB) take HBM as long as a step takes the tensor core; with operands swapped and a narrow N
// it was no faster.  Mapped rows are gathered by
// fp8_rows_kernel before it (TMA's gather of four rows an instruction took three times as long
// as a step's MMAs).
// ---------------------------------------------------------------------------
template <int BN>
struct Fp8TileCfg {
    static constexpr int BM = 128, DB = 512 / BN;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int ST = BN == 256 ? 4 : 6;          // even: a stage always serves the same issuer
    static constexpr int THREADS = 384, TMEM_COLS = DB * BN;
    static constexpr int REGS_ISSUE = 72, REGS_FOLD = 216;   // after the split: of warps 0..3 and 4..11
    static constexpr int OUT_OFF = ST * STAGE;            // per fold warp: 32 rows x 32 columns of Y
    static constexpr int SCHED_OFF = OUT_OFF + 8 * 32 * 64;
    static constexpr int BAR_OFF = SCHED_OFF + (int)((sizeof(Fp8Sched) + 15) / 16 * 16);
    static constexpr int NBAR = 2 * ST + 2 * DB + 2;
    static constexpr int TOTAL = BAR_OFF + NBAR * 8 + 16 + 1024;
    static constexpr int PARTIAL = 128 * BN;              // floats of a piece's sums
    static_assert(TOTAL <= 227 * 1024 - 64 && ST % 2 == 0, "tile kernel shared memory");
};

// The 256 folding threads: the sums of pieces cf .. cl of a tile, added in that order, to Y.  PER
// times four columns and PIECES pieces a thread are in flight.
template <int BN, int PER, int PIECES>
QG_DEV_INLINE void fp8_join(const Fp8Params& p, int s0, int rows, int n0, int cf, int cl)
{
    const int count = min(rows, 128) * (BN / 4);
    const float4* base = reinterpret_cast<const float4*>(p.partials);
    for (int e0 = threadIdx.x - 128; e0 < count; e0 += 256 * PER) {
        float4 a[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) a[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c0 = cf; c0 <= cl; c0 += PIECES) {
            float4 v[PIECES][PER];
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int c = c0 + i;
                const float4* o = base + ((int64_t)c * 2 + (c == cf ? 1 : 0)) * (Fp8TileCfg<BN>::PARTIAL / 4) + e0;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    v[i][j] = c <= cl && e0 + 256 * j < count ? __ldcg(o + 256 * j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    a[j].x += v[i][j].x;
                    a[j].y += v[i][j].y;
                    a[j].z += v[i][j].z;
                    a[j].w += v[i][j].w;
                }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = e0 + 256 * j, r = e / (BN / 4), n = n0 + 4 * (e % (BN / 4));
            if (e >= count || n >= p.N) continue;
            uint2 v = p.bf16 ? make_uint2(pack_bf16x2_rn(a[j].x, a[j].y), pack_bf16x2_rn(a[j].z, a[j].w))
                             : make_uint2(pack_f16x2_rn(a[j].x, a[j].y), pack_f16x2_rn(a[j].z, a[j].w));
            if (fp8_row(p, s0 + r) < 0) v = make_uint2(0u, 0u);   // a wrong map entry
            *reinterpret_cast<uint2*>(p.Y + (int64_t)(s0 + r) * p.N + n) = v;
        }
    }
}

template <int BN>
__global__ void __launch_bounds__(Fp8TileCfg<BN>::THREADS, 1)
    fp8_tile_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x)
{
    using C = Fp8TileCfg<BN>;
    constexpr int ST = C::ST, DB = C::DB, HW = BN / 2;   // HW: columns of a fold warp
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Fp8Sched& sched = *reinterpret_cast<Fp8Sched*>(smem + C::SCHED_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + ST;
    uint64_t* dfull = empty + ST;
    uint64_t* dempty = dfull + DB;
    uint64_t* done = dempty + DB;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 2);
    __shared__ int s_last;
    __shared__ Fp8Work work;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int G = p.G, slabs = (p.N + BN - 1) / BN;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < DB; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 8);
        }
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    // Whatever memory this kernel reads, weights and scales too, may have been written by the kernel
    // before it, so every thread waits for that one first (and no bounded wait below counts the
    // time of another kernel).  Only a dense product's schedule comes from the parameters alone.
    if (p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!fp8_schedule<C::BM>(sched, p, slabs)) return;
    if (threadIdx.x == 0) work.init(sched.pre[p.E], BN / 128, p.join_rows, G, gridDim.x, blockIdx.x);
    __syncthreads();
    if (!p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (work.steps() == 0) return;
    if (warp == 1) {
        tmem_alloc(tslot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    if (warp < 4) {
        setmaxnreg_dec<C::REGS_ISSUE>();
        if (warp == 0) {
            // ---------------- producer ----------------
            Fp8Walk<C::BM> walk(sched, p.E, slabs);
            const bool one = elect_one();
            bool ok = true;
            int tile, k0, k1;
            int64_t issued = 0;
            int s = 0;
            uint32_t sp = 1;   // parity
            for (int i = 0; ok && work.piece(i, tile, k0, k1); ++i) {
                walk.at(tile);
                const int s0 = walk.first(), n0 = walk.slab * BN;
                for (int kb = k0; kb < k1; ++kb) {
                    ok = all_wait(&empty[s], sp);
                    if (!ok) break;
                    if (one) {
                        uint8_t* st = smem + s * C::STAGE;
                        mbar_arrive_expect_tx(&full[s], C::B_BYTES + p.box * 128);
                        tma_load_3d(&tm_w, &full[s], st + C::A_BYTES, n0, kb * 128, walk.e);
                        if (BN == 256) tma_load_3d(&tm_w, &full[s], st + C::A_BYTES + 16384, n0 + 128, kb * 128, walk.e);
                        tma_load_2d(&tm_x, &full[s], st, kb * 128, s0);
                    }
                    __syncwarp();
                    if (++s == ST) { s = 0; sp ^= 1; }
                    ++issued;
                }
            }
            if (!ok)   // copies in flight land before the block leaves
                for (int64_t j = issued > ST ? issued - ST : 0; j < issued; ++j) all_wait(&full[j % ST], (int)(j / ST) & 1);
        } else if (warp & 1) {
            // ---------------- MMA issuers (two, so that one's waits lie beside the other's MMAs) ----------------
            constexpr uint32_t idesc = idesc_e4m3(BN, false, true);
            const uint64_t a0 = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t b0 = smem_desc(smem_u32(smem + C::A_BYTES), 16384, 1024, 2);
            const bool one = elect_one();
            const int64_t steps = work.steps();
            const int e = warp >> 1;
            int64_t i = e;
            int s = e, b = e;
            uint32_t sp = 0, bp = 1;   // parities
            for (; i < steps; i += 2) {
                if (!all_wait(&full[s], sp) || !all_wait(&dempty[b], bp)) break;
                tc_fence_after();
                if (one) {
                    const uint64_t ad = a0 + s * (C::STAGE >> 4), bd = b0 + s * (C::STAGE >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_e4m3_ss(tmem + b * BN, ad + kk * (32 >> 4), bd + kk * (4096 >> 4), idesc, kk > 0 ? 1u : 0u);
                    mma_commit(&dfull[b]);
                    mma_commit(&empty[s]);
                }
                __syncwarp();
                if ((s += 2) >= ST) { s = e; sp ^= 1; }
                if ((b += 2) >= DB) { b = e; bp ^= 1; }
            }
            if (i > 1) {   // every MMA has completed before tensor memory is released
                if (one) mma_commit(&done[e]);
                __syncwarp();
                all_wait(&done[e], 0);
            }
        }
    } else {
        setmaxnreg_inc<C::REGS_FOLD>();
        // ---------------- fold: thread = row, HW columns ----------------
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * HW;
        uint8_t* out = smem + C::OUT_OFF + (warp - 4) * 2048;
        const bool vec = G % 4 == 0;   // then every row of xs starts on 16 bytes
        // the scales of this thread's row and columns, four groups at a time, the next four loading
        float x[4], w[4];
        int s0, rows, n0, row, tile, k0, k1;
        const float *xp, *wp;
        auto load = [&](int kb) {
            if (vec) {
                const float4 v = *reinterpret_cast<const float4*>(xp + kb);
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = xp[min(kb + j, G - 1)];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = wp[(int64_t)min(kb + j, G - 1) * p.NB];
        };
        auto open = [&]() {
            Fp8Walk<C::BM> walk(sched, p.E, slabs);
            walk.at(tile);
            s0 = walk.first() + 32 * q;
            rows = walk.rows() - 32 * q;
            n0 = walk.slab * BN + half * HW;
            row = lane < rows ? fp8_row(p, s0 + lane) : -2;
            if (row == -1 && walk.slab == 0 && half == 0) set_status(6u);
            xp = p.xs + (int64_t)max(row, 0) * G;
            wp = p.ws + (int64_t)walk.e * G * p.NB + min(n0 / 128, p.NB - 1);
            load(k0 & ~3);
        };
        bool ok = true, more = work.piece(0, tile, k0, k1);
        int b = 0;
        uint32_t bp = 0;
        open();
        // after a wait that gave up, the pieces of split tiles are still counted in, without work: a
        // replay of this launch starts from cleared counters
        for (int i = 0; more; ++i) {
            float acc[HW];
#pragma unroll
            for (int t = 0; t < HW; ++t) acc[t] = 0.0f;
            for (int k4 = k0 & ~3; k4 < k1 && ok; k4 += 4) {
                float sc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[j] = row >= 0 ? __fmul_rn(x[j], w[j]) : 0.0f;
                if (k4 + 4 < k1) load(k4 + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k4 + j < k0) continue;
                    if (k4 + j >= k1 || !ok) break;
                    ok = all_wait(&dfull[b], bp);
                    if (!ok) break;
                    tc_fence_after();
                    fp8_fold<HW>(acc, lanes + b * BN, sc[j], [&]() {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&dempty[b]);
                    });
                    if (++b == DB) { b = 0; bp ^= 1; }
                }
            }
            const bool zero = row < 0;
            const int os0 = s0, orows = rows, on0 = n0, ok0 = k0, ok1 = k1;
            more = work.piece(i + 1, tile, k0, k1);
            if (more) open();   // its scales load meanwhile
            bool write = ok;
            if (ok0 > 0 || ok1 < G) {   // a piece of a split tile
                const int64_t first = work.u0 + (i > work.whole ? work.n - ok1 : -ok0);   // the tile's first unit
                const int cf = work.cta_of(first), cl = work.cta_of(first + G - 1);
                float4* mine = reinterpret_cast<float4*>(p.partials + ((int64_t)blockIdx.x * 2 + (ok0 == 0 ? 1 : 0)) * C::PARTIAL +
                                                         (32 * q + lane) * BN + half * HW);
                if (lane < orows)
#pragma unroll
                    for (int c = 0; c < HW / 4; ++c)
                        __stcg(mine + c, make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
                named_bar_sync(1, 256);
                if (threadIdx.x == 128) {
                    __threadfence();   // of all 256 threads' stores, by the barrier
                    s_last = fp8_arrive(p.counters + cf, p.token, cl - cf + 1);
                    __threadfence();
                }
                named_bar_sync(1, 256);
                write = false;
                if (ok && s_last) {
                    const int tr = orows + 32 * q;   // the tile's rows
                    if (tr * (BN / 4) <= 256) fp8_join<BN, 1, 8>(p, os0 - 32 * q, tr, on0 - half * HW, cf, cl);
                    else fp8_join<BN, 4, 4>(p, os0 - 32 * q, tr, on0 - half * HW, cf, cl);
                }
                named_bar_sync(1, 256);   // s_last has been read
            }
            // Y: 32 x 32 blocks turned in shared memory, so that four lanes store 64 bytes of a row
            auto store = [&](auto bf) {
#pragma unroll
                for (int c = 0; c < HW; c += 32) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            o[t] = zero ? 0u : fp8_out2<decltype(bf)::value>(acc[c + 8 * j + 2 * t], acc[c + 8 * j + 2 * t + 1]);
                        *reinterpret_cast<uint4*>(out + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    __syncwarp();
                    const int n = on0 + c + 8 * (lane & 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 8 * j + (lane >> 2);
                        const uint4 v = *reinterpret_cast<const uint4*>(out + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                        if (r < orows && n < p.N) *reinterpret_cast<uint4*>(p.Y + (int64_t)(os0 + r) * p.N + n) = v;
                    }
                }
            };
            if (!write) continue;
            if (p.bf16) store(std::true_type{});
            else store(std::false_type{});
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace qg
