// fp8_gemm.cuh -- products of e4m3 operands with a scale for each 128 of K, on the tcgen05
// tensor cores:
//
//   Y[m][n] = rn( sum_g (xs[m][g] ws[g][n / 128]) sum_{k in g} Xq[m][k] Wq[k][n] )   (fp32)
//
// and the same per expert over the rows of its slots.  ("AI Infra guide, ch.4
// Quantization" sec. 5, e4m3; "LLM inference cost ..." sec. 2.2, groups of 128.)
//
// What both kernels share.  The scales change every 128 of K, so the tensor core sums one
// group at a time (fp32, tensor memory) and the epilogue warps fold each group's sums into
// fp32 registers with one fma, acc += P * (xs * ws), while the tensor core works on the next
// group in another buffer.  The weights stay as they are stored, [K][N]: a TMA box of
// 128 k x 128 columns, 128-byte swizzle, is the MMA's MN-major operand.  A dense product is
// the experts' product with one expert that has all the rows; rows are gathered by TMA
// (four rows an instruction) when a map is given.
//
//   fp8_stream_kernel: few rows.  128 columns are the MMA's M, 16..128 rows its N; the
//     weights are streamed once, the (tile, group) units split evenly over the CTAs.
//   fp8_tile_kernel: many rows.  128 rows x 256 columns, persistent.
//
// Every wait is bounded (mbar_wait); one that gives up records QG_ERR_TIMEOUT, and the role
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
    bool bf16;
    // stream kernel: the workspace
    unsigned long long* counters;  // [grid]
    float* partials;               // [grid][2][NT][256]
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

// Four rows y[0..3] of a 2-D map whose box is one row high, to consecutive rows of the tile.
QG_DEV_INLINE void tma_gather4(const CUtensorMap* m, uint64_t* bar, void* smem_dst, int x, const int (&y)[4])
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
        : "memory");
}

template <int R>
QG_DEV_INLINE void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
QG_DEV_INLINE void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// A bounded wait like mbar_wait's that looks at the clock and the limit only after many polls:
// here a wait is mostly a few hundred cycles long and lies on the chain between the tensor core
// and the warps that fold.
QG_DEV_INLINE bool short_wait(uint64_t* bar, uint32_t parity)
{
    for (uint32_t it = 0; it < 256; ++it)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity);
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
QG_DEV_INLINE bool all_wait(uint64_t* bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, short_wait(bar, parity));
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
    QG_DEV_INLINE void next()
    {
        if (++chunk < chunks) return;
        chunk = 0;
        if (++slab < slabs) return;
        slab = 0;
        do ++e;
        while (e < E && sc.off[e + 1] == sc.off[e]);
        if (e < E) chunks = (sc.off[e + 1] - sc.off[e] + T - 1) / T;
    }
    QG_DEV_INLINE int first() const { return sc.off[e] + chunk * T; }
    QG_DEV_INLINE int rows() const { return min(T, sc.off[e + 1] - first()); }
};

// The row of Xq that slot s reads; -1 where the map is wrong.
QG_DEV_INLINE int fp8_row(const Fp8Params& p, int s)
{
    if (!p.rows) return s;
    const int r = __ldg(p.rows + s);
    return (uint32_t)r < (uint32_t)p.Mx ? r : -1;
}

// The four rows that this lane gathers of a tile (lane l: rows 4l .. 4l + 3); rows past the
// tile's and wrong entries read row 0, whose sums go nowhere.
QG_DEV_INLINE void fp8_gather_rows(const Fp8Params& p, int s0, int rows, int lane, int (&y)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * lane + i;
        y[i] = t < rows ? max(fp8_row(p, s0 + t), 0) : 0;
    }
}

template <bool BF16>
QG_DEV_INLINE uint32_t fp8_out2(float a, float b) { return BF16 ? pack_bf16x2_rn(a, b) : pack_f16x2_rn(a, b); }

// The scales of a run of units (tiles of T rows x 256 columns), four groups at a time: a lane holds R rows, the four groups in
// use and, loading, the four after them, so that a load has four units' time to arrive.  (One
// load per unit, four units ahead, was slower: a wait for one of them waited for all.)
template <int T, int R>
struct Fp8Scales {
    const Fp8Params& p;
    Fp8Walk<T> walk;      // of the tile being loaded
    int64_t left;         // units not yet loaded
    int lane, kb;         // first group not yet loaded
    int row[R];
    const float* wsp;     // the tile's first weight scale
    bool wide;            // its second 128 columns exist
    float x[R][4], w[2][4], nx[R][4], nw[2][4];
    int n, nn;            // groups held and loading

    QG_DEV_INLINE Fp8Scales(const Fp8Params& p_, const Fp8Walk<T>& w_, int64_t units, int kb0, int lane_)
        : p(p_), walk(w_), left(units), lane(lane_), kb(kb0), n(0), nn(0)
    {
        tile();
        load();
    }
    QG_DEV_INLINE void tile()
    {
        const int s0 = walk.first(), rows = walk.rows();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = lane + 32 * r;
            row[r] = t < rows ? fp8_row(p, s0 + t) : -2;
            if (row[r] == -1) set_status(6u);
        }
        wsp = p.ws + (int64_t)walk.e * p.G * p.NB + 2 * walk.slab;
        wide = 2 * walk.slab + 1 < p.NB;
    }
    QG_DEV_INLINE void load()
    {
        nn = (int)min((int64_t)min(4 - (kb & 3), p.G - kb), left);
        if (nn == 0) return;
        const bool vec = p.G % 4 == 0;   // then every row starts on 16 bytes
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float* src = p.xs + (int64_t)max(row[r], 0) * p.G + kb;
            if (vec && nn == 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(src));
                nx[r][0] = v.x; nx[r][1] = v.y; nx[r][2] = v.z; nx[r][3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) nx[r][j] = j < nn ? __ldg(src + j) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float* src = wsp + (int64_t)(kb + j) * p.NB;
            nw[0][j] = j < nn ? __ldg(src) : 0.0f;
            nw[1][j] = j < nn && wide ? __ldg(src + 1) : 0.0f;
        }
    }
    // The loaded groups become those in use, the next ones are requested; false: none left.
    QG_DEV_INLINE bool advance()
    {
        n = nn;
        if (n == 0) return false;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[r][j] = row[r] >= 0 ? nx[r][j] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[0][j] = nw[0][j];
            w[1][j] = nw[1][j];
        }
        left -= n;
        kb += n;
        if (kb == p.G) {
            kb = 0;
            if (left > 0) {
                walk.next();
                tile();
            }
        }
        load();
        return true;
    }
};

// acc[0 .. CW) += (CW sums of tensor memory at `addr`) * scale, where the scale of sum t is
// sv[t] (shared memory, 16-byte aligned; PER = true) or the one number sc.  Sixteen columns at a
// time, the next ones' load in flight while the ones before are folded; `release` runs once all
// are read (PER: and their scales too).
template <int CW, bool PER, typename F>
QG_DEV_INLINE void fp8_fold(float (&acc)[CW], uint32_t addr, const float* sv, float sc, F release)
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
        else if (!PER) release();
#pragma unroll
        for (int t = 0; t < 16; t += 4) {
            float4 s4 = make_float4(sc, sc, sc, sc);
            if constexpr (PER) s4 = *reinterpret_cast<const float4*>(sv + c + t);
            acc[c + t] = fmaf(__uint_as_float(u[t]), s4.x, acc[c + t]);
            acc[c + t + 1] = fmaf(__uint_as_float(u[t + 1]), s4.y, acc[c + t + 1]);
            acc[c + t + 2] = fmaf(__uint_as_float(u[t + 2]), s4.z, acc[c + t + 2]);
            acc[c + t + 3] = fmaf(__uint_as_float(u[t + 3]), s4.w, acc[c + t + 3]);
        }
    }
    if (PER) release();
}

// ---------------------------------------------------------------------------
// Few rows: stream-K
//
// Tiles of NT rows x 256 columns (256 so that a weight row is read 256 bytes at a time: with
// 128-byte boxes DRAM read 1.37 times the weights).  Units are (tile, group of K); CTA c takes
// units [c U / grid, (c + 1) U / grid).  A tile whose units lie in several CTAs is joined by
// whichever of them arrives last: each leaves its fp32 sums in the workspace and counts itself
// in; the last one adds all of them in CTA order (the result does not depend on who is last)
// and writes Y.  No CTA waits for another.  The counter word holds the launch's token above an
// 8-bit count, so whatever an unused workspace holds reads as 0, and the last arrival clears
// it, so a replayed graph finds it so again.
//
// Roles: warp 0 TMA; warp 1 issues the MMAs (the 128-column halves are M, the rows N; each
// unit into one of DB buffers); warp 2 writes the units' scales; warps 4..11 fold the units
// (thread = column).
// ---------------------------------------------------------------------------
template <int NT>
struct Fp8StreamCfg {
    static constexpr int W_BYTES = 2 * 128 * 128, X_BYTES = NT * 128;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int ST = NT <= 32 ? 6 : 4;     // even: a stage always serves the same issuer
    static constexpr int DB = NT == 128 ? 2 : 4;    // buffers of sums [2][NT]
    static constexpr int SC = 8;                    // slots of scales [2][NT]
    static constexpr int EPI = 8;
    static constexpr int THREADS = 32 * (4 + EPI);
    static constexpr int TMEM_COLS = DB * 2 * NT;
    static constexpr int SC_OFF = ST * STAGE;
    static constexpr int SCHED_OFF = SC_OFF + SC * 2 * NT * 4;
    static constexpr int BAR_OFF = SCHED_OFF + (int)((sizeof(Fp8Sched) + 15) / 16 * 16);
    static constexpr int NBAR = 2 * ST + 2 * DB + 2 * SC + 2;
    static constexpr int TOTAL = BAR_OFF + NBAR * 8 + 16 + 1024;
    static constexpr int PARTIAL = NT * 256;        // floats of a piece's sums
    static_assert(STAGE % 1024 == 0 && TOTAL <= 227 * 1024 - 64 && ST % 2 == 0, "stream kernel shared memory");
};

QG_DEV_INLINE int64_t fp8_first_unit(int c, int64_t units, int grid) { return c * units / grid; }

QG_DEV_INLINE int fp8_cta_of_unit(int64_t u, int64_t units, int grid)
{
    int c = (int)(u * grid / units);
    while (c > 0 && fp8_first_unit(c, units, grid) > u) --c;
    while (fp8_first_unit(c + 1, units, grid) <= u) ++c;
    return c;
}

// Counts one arrival of `n` under `token`; true for the last, which clears the word.
QG_DEV_INLINE bool fp8_arrive(unsigned long long* word, unsigned long long token, int n)
{
    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
    for (;;) {
        const unsigned long long have = (old & ~0xFFull) == token ? old & 0xFFull : 0ull;
        const bool last = have + 1 == (unsigned long long)n;
        const unsigned long long seen = atomicCAS(word, old, last ? 0ull : token | (have + 1));
        if (seen == old) return last;
        old = seen;
    }
}

template <int NT>
__global__ void __launch_bounds__(Fp8StreamCfg<NT>::THREADS, 1)
    fp8_stream_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_x)
{
    using C = Fp8StreamCfg<NT>;
    constexpr int ST = C::ST, DB = C::DB, SC = C::SC;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);   // [SC][2][NT]
    Fp8Sched& sched = *reinterpret_cast<Fp8Sched*>(smem + C::SCHED_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + ST;
    uint64_t* dfull = empty + ST;
    uint64_t* dempty = dfull + DB;
    uint64_t* sfull = dempty + DB;
    uint64_t* sempty = sfull + SC;
    uint64_t* done = sempty + SC;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 2);
    __shared__ int s_last;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int G = p.G, slabs = (p.N + 255) / 256;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < DB; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], C::EPI);
        }
        for (int i = 0; i < SC; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], C::EPI);
        }
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    // the experts' offsets come from the kernel before; a dense product's schedule does not
    if (p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!fp8_schedule<NT>(sched, p, slabs)) return;
    const int64_t units = (int64_t)sched.pre[p.E] * G;
    const int grid = (int)min((int64_t)gridDim.x, units);
    if ((int)blockIdx.x >= grid) return;
    const int64_t u0 = fp8_first_unit(blockIdx.x, units, grid);
    const int n_it = (int)(fp8_first_unit(blockIdx.x + 1, units, grid) - u0);
    const int tile0 = (int)(u0 / G), kb0 = (int)(u0 - (int64_t)tile0 * G);
    if (warp == 1) {
        tmem_alloc(tslot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    Fp8Walk<NT> walk(sched, p.E, slabs);
    walk.at(tile0);
    if (warp < 4) {
        if constexpr (NT == 128) setmaxnreg_dec<72>();
        if (warp == 0) {
            // ---------------- producer ----------------
            int kb = kb0, i = 0, y[4];
            const bool one = elect_one();
            const int early = p.offsets ? 0 : min(ST, n_it);
            auto weights = [&](int s, const Fp8Walk<NT>& w, int k) {
                uint8_t* st = smem + s * C::STAGE;
                mbar_arrive_expect_tx(&full[s], C::STAGE);
                tma_load_3d(&tm_w, &full[s], st, w.slab * 256, k * 128, w.e);
                tma_load_3d(&tm_w, &full[s], st + 16384, w.slab * 256 + 128, k * 128, w.e);
            };
            if (early) {
                // weights do not depend on the kernel before: the ring's first are requested
                // before waiting for it
                Fp8Walk<NT> w = walk;
                for (int j = 0, k = kb0; j < early; ++j) {
                    if (one) weights(j, w, k);
                    if (++k == G) { k = 0; w.next(); }
                }
                asm volatile("griddepcontrol.wait;" ::: "memory");
            }
            if (p.rows) fp8_gather_rows(p, walk.first(), walk.rows(), lane, y);
            bool ok = true;
            for (; i < n_it; ++i) {
                const int s = i % ST;
                if (i >= early) {
                    ok = all_wait(&empty[s], ((i / ST) & 1) ^ 1);
                    if (!ok) break;
                    if (one) weights(s, walk, kb);
                    __syncwarp();
                }
                uint8_t* xt = smem + s * C::STAGE + C::W_BYTES;
                if (!p.rows) {
                    if (one) tma_load_2d(&tm_x, &full[s], xt, kb * 128, walk.first());
                } else if (lane < NT / 4) {
                    tma_gather4(&tm_x, &full[s], xt + lane * 512, kb * 128, y);
                }
                if (++kb == G) {
                    kb = 0;
                    walk.next();
                    if (p.rows && i + 1 < n_it) fp8_gather_rows(p, walk.first(), walk.rows(), lane, y);
                }
            }
            if (!ok)   // copies in flight land before the block leaves
                for (int j = max(i - ST, 0); j < i; ++j) all_wait(&full[j % ST], (j / ST) & 1);
        } else if (warp & 1) {
            // ------- MMA issuers: warp 1 the even units, warp 3 the odd ones, so that one's waits
            // lie beside the other's MMAs -------
            constexpr uint32_t idesc = idesc_e4m3(NT, true, false);
            const uint64_t w0 = smem_desc(smem_u32(smem), 16384, 1024, 2), x0 = smem_desc(smem_u32(smem + C::W_BYTES), 16, 1024, 2);
            const bool one = elect_one();
            const int e = warp >> 1;
            int i = e, s = e, b = e;
            uint32_t sp = 0, bp = 1;   // parities
            for (; i < n_it; i += 2) {
                if (!all_wait(&full[s], sp) || !all_wait(&dempty[b], bp)) break;
                tc_fence_after();
                if (one) {
                    const uint64_t w = w0 + s * (C::STAGE >> 4), x = x0 + s * (C::STAGE >> 4);
                    const uint32_t d = tmem + 2 * b * NT;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_e4m3_ss(d + h * NT, w + h * (16384 >> 4) + kk * (4096 >> 4), x + kk * (32 >> 4), idesc, kk > 0 ? 1u : 0u);
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
        } else if (warp == 2) {
            // ---------------- scales ----------------
            if (!p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
            constexpr int R = (NT + 31) / 32;
            Fp8Scales<NT, R> sc(p, walk, n_it, kb0, lane);
            bool ok = true;
            int i = 0;
            while (ok && sc.advance()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < sc.n && ok) {
                        const int b = i % SC;
                        ok = all_wait(&sempty[b], ((i / SC) & 1) ^ 1);
                        if (ok) {
                            float* o = scales + b * 2 * NT;
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                if (lane + 32 * r < NT) {
                                    o[lane + 32 * r] = __fmul_rn(sc.x[r][j], sc.w[0][j]);
                                    o[NT + lane + 32 * r] = __fmul_rn(sc.x[r][j], sc.w[1][j]);
                                }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sfull[b]);
                            ++i;
                        }
                    }
                }
            }
        }
    } else {
        if constexpr (NT == 128) setmaxnreg_inc<216>();
        // ---------------- fold: thread = column ----------------
        asm volatile("griddepcontrol.wait;" ::: "memory");   // Y and the workspace follow the kernel before
        const int q = warp & 3, half = (warp - 4) >> 2, col = half * 128 + 32 * q + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * NT;
        float acc[NT];
        bool ok = true;
        int i = 0, kb = kb0;
        while (i < n_it) {
            const int ie = min(n_it, i + G - kb);   // this piece: units [i, ie)
            const bool head = kb == 0, whole = head && ie - i == G;
            const int64_t first = u0 + i - kb;      // the tile's first unit
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = 0.0f;
            for (; i < ie; ++i) {
                const int b = i % DB, sl = i % SC;
                if (ok) ok = all_wait(&sfull[sl], (i / SC) & 1) && all_wait(&dfull[b], (i / DB) & 1);
                if (!ok) continue;
                tc_fence_after();
                fp8_fold<NT, true>(acc, lanes + b * 2 * NT, scales + (2 * sl + half) * NT, 0.0f, [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&dempty[b]);
                        mbar_arrive(&sempty[sl]);
                    }
                });
            }
            const int rows = walk.rows(), s0 = walk.first(), n = walk.slab * 256 + col;
            bool write = whole;
            if (!whole) {
                float* mine = p.partials + ((int64_t)blockIdx.x * 2 + (head ? 1 : 0)) * C::PARTIAL + col;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if ((t & ~15) < rows) __stcg(mine + t * 256, acc[t]);
                // the pieces of this tile are CTAs cf .. cl
                const int cf = head ? (int)blockIdx.x : fp8_cta_of_unit(first, units, grid);
                const int cl = fp8_cta_of_unit(first + G - 1, units, grid);
                __threadfence();
                named_bar_sync(1, 32 * C::EPI);
                if (threadIdx.x == 128) {
                    s_last = fp8_arrive(p.counters + cf, p.token, cl - cf + 1);
                    __threadfence();
                }
                named_bar_sync(1, 32 * C::EPI);
                write = s_last;
                if (write) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t] = 0.0f;
                    for (int c = cf; c <= cl; ++c) {
                        const float* o = p.partials + ((int64_t)c * 2 + (c == cf ? 1 : 0)) * C::PARTIAL + col;
#pragma unroll
                        for (int t0 = 0; t0 < NT; t0 += 16) {   // 16 loads in flight
                            if (t0 < rows) {
                                float v[16];
#pragma unroll
                                for (int t = 0; t < 16; ++t) v[t] = __ldcg(o + (t0 + t) * 256);
#pragma unroll
                                for (int t = 0; t < 16; ++t) acc[t0 + t] += v[t];
                            }
                        }
                    }
                }
                named_bar_sync(1, 32 * C::EPI);   // s_last has been read
            }
            if (write && ok) {
                uint32_t zero[(NT + 31) / 32];   // rows whose map entry is wrong
#pragma unroll
                for (int r = 0; r < (NT + 31) / 32; ++r) {
                    const int t = lane + 32 * r;
                    zero[r] = p.rows ? __ballot_sync(0xffffffffu, t < rows && fp8_row(p, s0 + t) < 0) : 0u;
                }
                auto store = [&](auto bf) {
                    // lane pairs exchange, so that a lane stores two adjacent columns of a row
                    const int odd = lane & 1;
                    uint16_t* y = p.Y + (int64_t)(s0 + odd) * p.N + n - odd;
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        if ((t & ~15) >= rows) break;
                        uint32_t ab = fp8_out2<decltype(bf)::value>(acc[t], acc[t + 1]);   // two rows of a column
                        if (zero[t / 32] >> (t & 31) & 1u) ab &= 0xFFFF0000u;
                        if (zero[t / 32] >> ((t + 1) & 31) & 1u) ab &= 0xFFFFu;
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, ab, 1);
                        if (t + odd < rows && n < p.N)
                            *reinterpret_cast<uint32_t*>(y + (int64_t)t * p.N) = odd ? prmt(got, ab, 0x7632) : prmt(ab, got, 0x5410);
                    }
                };
                if (p.bf16) store(std::true_type{});
                else store(std::false_type{});
            }
            kb = 0;
            walk.next();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// The mapped rows in slot order, for the tile kernel (a wrong map entry: row 0, whose sums go
// nowhere).  Four slots and 4 KB of K per CTA, 64 threads a slot.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fp8_rows_kernel(const Fp8Params p, const uint8_t* __restrict__ Xq,
                                                       uint8_t* __restrict__ xg)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (s >= min(p.offsets[p.E], p.S)) return;
    const uint4* src = reinterpret_cast<const uint4*>(Xq + (int64_t)max(fp8_row(p, s), 0) * p.K);
    uint4* dst = reinterpret_cast<uint4*>(xg + (int64_t)s * p.K);
    const int end = min(p.K / 16, ((int)blockIdx.y + 1) * 256);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = blockIdx.y * 256 + i * 64 + (threadIdx.x & 63);
        if (k < end) dst[k] = __ldg(src + k);
    }
}

// ---------------------------------------------------------------------------
// Many rows: 128 rows x BN columns, one group of K a step, persistent.
//
// Mapped rows are gathered by fp8_rows_kernel before it (TMA's gather of four rows an
// instruction took three times as long as a step's MMAs).
//
// Roles: warp 0 TMA; warps 1 and 3 issue the MMAs, step by step into DB buffers; warps 4..11
// fold: thread = row, BN / 2 columns, whose weight scale is one number, so a step costs a thread
// one scale and BN / 2 fma.
// ---------------------------------------------------------------------------
template <int BN>
struct Fp8TileCfg {
    static constexpr int BM = 128, DB = 512 / BN;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int ST = BN == 256 ? 4 : 6;
    static constexpr int THREADS = 384;
    static constexpr int OUT_OFF = ST * STAGE;            // per fold warp: 32 rows x 32 columns of Y
    static constexpr int SCHED_OFF = OUT_OFF + 8 * 32 * 64;
    static constexpr int BAR_OFF = SCHED_OFF + (int)((sizeof(Fp8Sched) + 15) / 16 * 16);
    static constexpr int NBAR = 2 * ST + 2 * DB + 2;
    static constexpr int TOTAL = BAR_OFF + NBAR * 8 + 16 + 1024;
    static_assert(TOTAL <= 227 * 1024 && ST % 2 == 0, "tile kernel shared memory");
};

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

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int G = p.G, slabs = (p.N + BN - 1) / BN;
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
    if (p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!fp8_schedule<C::BM>(sched, p, slabs)) return;
    const int tiles = sched.pre[p.E];
    if ((int)blockIdx.x >= tiles) return;
    if (warp == 1) {
        tmem_alloc(tslot, C::DB * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    Fp8Walk<C::BM> walk(sched, p.E, slabs);

    if (warp < 4) {
        setmaxnreg_dec<72>();
        if (warp == 0) {
            // ---------------- producer ----------------
            const bool one = elect_one();
            bool ok = true;
            int64_t issued = 0;
            asm volatile("griddepcontrol.wait;" ::: "memory");
            int s = 0;
            uint32_t sp = 1;   // parity
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                walk.at(tile);
                const int s0 = walk.first(), n0 = walk.slab * BN;
                for (int kb = 0; kb < G; ++kb) {
                    ok = all_wait(&empty[s], sp);
                    if (!ok) break;
                    uint8_t* st = smem + s * C::STAGE;
                    if (one) {
                        mbar_arrive_expect_tx(&full[s], C::STAGE);
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
            // ------- MMA issuers: warp 1 the even units, warp 3 the odd ones, so that one's waits
            // lie beside the other's MMAs -------
            constexpr uint32_t idesc = idesc_e4m3(BN, false, true);
            const uint64_t a0 = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t b0 = smem_desc(smem_u32(smem + C::A_BYTES), 16384, 1024, 2);
            const bool one = elect_one();
            const int64_t steps = (int64_t)((tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * G;
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
        setmaxnreg_inc<216>();
        // ---------------- fold: thread = row, HW columns ----------------
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * HW;
        uint8_t* out = smem + C::OUT_OFF + (warp - 4) * 2048;
        const bool vec = G % 4 == 0;   // then every row of xs starts on 16 bytes
        // the scales of this thread's row and columns, four groups at a time, the next four loading
        float x[4], w[4];
        int s0, rows, n0, row;
        const float *xp, *wp;
        auto open = [&](int tile) {
            walk.at(tile);
            s0 = walk.first() + 32 * q;
            rows = walk.rows() - 32 * q;
            n0 = walk.slab * BN + half * HW;
            row = lane < rows ? fp8_row(p, s0 + lane) : -2;
            if (row == -1 && walk.slab == 0 && half == 0) set_status(6u);
            xp = p.xs + (int64_t)max(row, 0) * G;
            wp = p.ws + (int64_t)walk.e * G * p.NB + min(n0 / 128, p.NB - 1);
        };
        auto load = [&](int kb) {
            if (vec) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(xp + kb));
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = __ldg(xp + min(kb + j, G - 1));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __ldg(wp + (int64_t)min(kb + j, G - 1) * p.NB);
        };
        bool ok = true;
        int b = 0;
        uint32_t bp = 0;
        asm volatile("griddepcontrol.wait;" ::: "memory");   // xs and Y follow the kernel before
        open(blockIdx.x);
        load(0);
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            float acc[HW];
#pragma unroll
            for (int t = 0; t < HW; ++t) acc[t] = 0.0f;
            for (int k0 = 0; k0 < G && ok; k0 += 4) {
                float sc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[j] = row >= 0 ? __fmul_rn(x[j], w[j]) : 0.0f;
                if (k0 + 4 < G) load(k0 + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k0 + j >= G || !ok) break;
                    ok = all_wait(&dfull[b], bp);
                    if (!ok) break;
                    tc_fence_after();
                    fp8_fold<HW, false>(acc, lanes + b * BN, nullptr, sc[j], [&]() {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&dempty[b]);
                    });
                    if (++b == DB) { b = 0; bp ^= 1; }
                }
            }
            if (!ok) break;
            // Y: 32 x 32 blocks turned in shared memory, so that four lanes store 64 bytes of a row
            const bool zero = row < 0;
            const int os0 = s0, orows = rows, on0 = n0;
            if (tile + (int)gridDim.x < tiles) {
                open(tile + gridDim.x);
                load(0);
            }
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
            if (p.bf16) store(std::true_type{});
            else store(std::false_type{});
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::DB * BN);
    }
}

}  // namespace qg
