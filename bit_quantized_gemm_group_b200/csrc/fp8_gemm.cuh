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
    float* partials;               // [grid][2][NT][128]
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

// every lane waits; the result is the warp's
QG_DEV_INLINE bool all_wait(uint64_t* bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
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

QG_DEV_INLINE uint16_t fp8_out(const Fp8Params& p, float v) { return p.bf16 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v); }
QG_DEV_INLINE uint32_t fp8_out2(const Fp8Params& p, float a, float b) { return p.bf16 ? pack_bf16x2_rn(a, b) : pack_f16x2_rn(a, b); }

// ---------------------------------------------------------------------------
// Few rows: stream-K
//
// Units are (tile, group of K); CTA c takes units [c U / grid, (c + 1) U / grid).  A tile
// whose units lie in several CTAs is joined by whichever of them arrives last: each leaves
// its fp32 sums in the workspace and counts itself in; the last one adds all of them in CTA
// order (the result does not depend on who is last) and writes Y.  No CTA waits for another.
// The counter word holds the launch's token above an 8-bit count, so whatever an unused
// workspace holds reads as 0, and the last arrival clears it, so a replayed graph finds it
// so again.
//
// Roles: warp 0 TMA; warp 1 issues the MMAs (each unit into one of four buffers); warp 2
// multiplies the scales (four units ahead in registers) into the buffer's slot; warps 4..
// fold the units (thread = column).
// ---------------------------------------------------------------------------
template <int NT>
struct Fp8StreamCfg {
    static constexpr int W_BYTES = 128 * 128, X_BYTES = NT * 128;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int ST = NT == 16 ? 10 : NT == 32 ? 9 : NT == 64 ? 8 : 6;
    static constexpr int DB = 4;                    // buffers of sums and scales
    static constexpr int EPI = NT == 128 ? 8 : 4;   // epilogue warps
    static constexpr int CW = NT * 4 / EPI;         // rows of the tile per epilogue thread
    static constexpr int THREADS = 32 * (4 + EPI);
    static constexpr int TMEM_COLS = DB * NT;
    static constexpr int SC_OFF = ST * STAGE;
    static constexpr int SCHED_OFF = SC_OFF + DB * NT * 4;
    static constexpr int BAR_OFF = SCHED_OFF + (int)((sizeof(Fp8Sched) + 15) / 16 * 16);
    static constexpr int NBAR = 2 * ST + 2 * DB + 1;
    static constexpr int TOTAL = BAR_OFF + NBAR * 8 + 16 + 1024;
    static_assert(STAGE % 1024 == 0 && TOTAL <= 227 * 1024, "stream kernel shared memory");
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
    constexpr int ST = C::ST, DB = C::DB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);   // [DB][NT]
    Fp8Sched& sched = *reinterpret_cast<Fp8Sched*>(smem + C::SCHED_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + ST;
    uint64_t* dfull = empty + ST;     // the buffer's sums (the MMAs' commit) and scales (warp 2)
    uint64_t* dempty = dfull + DB;
    uint64_t* done = dempty + DB;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    __shared__ int s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G, slabs = (p.N + 127) / 128;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < DB; ++i) {
            mbar_init(&dfull[i], 2);
            mbar_init(&dempty[i], C::EPI);
        }
        mbar_init(done, 1);
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
    if (warp == 0) {
        // ---------------- producer ----------------
        int kb = kb0, i = 0, y[4];
        const int early = p.offsets ? 0 : min(ST, n_it);
        if (early) {
            // weights do not depend on the kernel before: the ring's first are requested
            // before waiting for it
            Fp8Walk<NT> w = walk;
            for (int j = 0, k = kb0; j < early; ++j) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[j], C::STAGE);
                    tma_load_3d(&tm_w, &full[j], smem + j * C::STAGE, w.slab * 128, k * 128, w.e);
                }
                if (++k == G) { k = 0; w.next(); }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
        }
        if (p.rows) fp8_gather_rows(p, walk.first(), walk.rows(), lane, y);
        bool ok = true;
        for (; i < n_it; ++i) {
            const int s = i % ST;
            uint8_t* st = smem + s * C::STAGE;
            if (i >= early) {
                ok = all_wait(&empty[s], ((i / ST) & 1) ^ 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], C::STAGE);
                    tma_load_3d(&tm_w, &full[s], st, walk.slab * 128, kb * 128, walk.e);
                }
                __syncwarp();
            }
            if (!p.rows) {
                if (lane == 0) tma_load_2d(&tm_x, &full[s], st + C::W_BYTES, kb * 128, walk.first());
            } else if (lane < NT / 4) {
                tma_gather4(&tm_x, &full[s], st + C::W_BYTES + lane * 512, kb * 128, y);
            }
            if (++kb == G) {
                kb = 0;
                walk.next();
                if (p.rows && i + 1 < n_it) fp8_gather_rows(p, walk.first(), walk.rows(), lane, y);
            }
        }
        if (!ok)   // copies in flight land before the block leaves
            for (int j = max(i - ST, 0); j < i; ++j) all_wait(&full[j % ST], (j / ST) & 1);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(NT, true, false);
            int i = 0;
            for (; i < n_it; ++i) {
                const int s = i % ST, b = i % DB;
                if (!mbar_wait(&dempty[b], ((i / DB) & 1) ^ 1) || !mbar_wait(&full[s], (i / ST) & 1)) break;
                tc_fence_after();
                const uint32_t w = smem_u32(smem + s * C::STAGE), x = w + C::W_BYTES;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_e4m3_ss(tmem + b * NT, smem_desc(w + 4096 * kk, 16384, 1024, 2),
                                smem_desc(x + 32 * kk, 16, 1024, 2), idesc, kk > 0 ? 1u : 0u);
                mma_commit(&empty[s]);
                mma_commit(&dfull[b]);
            }
            if (i > 0) {   // every MMA has completed before tensor memory is released
                mma_commit(done);
                mbar_wait(done, 0);
            }
        }
    } else if (warp == 2) {
        // ---------------- scales ----------------
        if (!p.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int R = (NT + 31) / 32, AHEAD = 4;
        static_assert(AHEAD == DB, "one register set per buffer");
        int row[R], kb = kb0;
        float x[AHEAD][R], w[AHEAD];
        const float* wsp = nullptr;
        auto tile_rows = [&]() {
            const int s0 = walk.first(), rows = walk.rows();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int t = lane + 32 * r;
                row[r] = t < rows ? fp8_row(p, s0 + t) : -2;
                if (row[r] == -1) set_status(6u);
            }
            wsp = p.ws + (int64_t)walk.e * G * p.NB + walk.slab;
        };
        auto load = [&](int slot) {
#pragma unroll
            for (int r = 0; r < R; ++r) x[slot][r] = row[r] >= 0 ? __ldg(p.xs + (int64_t)row[r] * G + kb) : 0.0f;
            w[slot] = __ldg(wsp + (int64_t)kb * p.NB);
        };
        auto step = [&](bool more) {
            if (++kb == G) {
                kb = 0;
                if (more) {
                    walk.next();
                    tile_rows();
                }
            }
        };
        tile_rows();
        int ahead = 0;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (ahead < n_it) {
                load(a);
                ++ahead;
                step(ahead < n_it);
            }
        bool ok = true;
        for (int i0 = 0; i0 < n_it && ok; i0 += AHEAD) {
#pragma unroll
            for (int b = 0; b < AHEAD; ++b) {
                if (i0 + b >= n_it || !ok) break;
                ok = all_wait(&dempty[b], ((i0 / DB) & 1) ^ 1);
                if (!ok) break;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (lane + 32 * r < NT) scales[b * NT + lane + 32 * r] = __fmul_rn(x[b][r], w[b]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&dfull[b]);
                if (ahead < n_it) {
                    load(b);
                    ++ahead;
                    step(ahead < n_it);
                }
            }
        }
    } else if (warp >= 4) {
        // ---------------- epilogue: thread = column ----------------
        asm volatile("griddepcontrol.wait;" ::: "memory");   // Y and the workspace follow the kernel before
        constexpr int CW = C::CW;
        const int q = warp & 3, t0 = (warp - 4) / 4 * CW, col = 32 * q + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + t0;
        float acc[CW];
        bool ok = true;
        int i = 0, kb = kb0;
        while (i < n_it) {
            const int ie = min(n_it, i + G - kb);   // this piece: units [i, ie)
            const bool head = kb == 0, whole = head && ie - i == G;
#pragma unroll
            for (int t = 0; t < CW; ++t) acc[t] = 0.0f;
            const int piece0 = i;
            for (; i < ie; ++i) {
                const int b = i % DB;
                ok = ok && all_wait(&dfull[b], (i / DB) & 1);
                if (!ok) continue;
                tc_fence_after();
                const float* sv = scales + b * NT + t0;
                constexpr int CH = CW < 32 ? 16 : 32;
#pragma unroll
                for (int c = 0; c < CW; c += CH) {
                    uint32_t r[CH];
                    if constexpr (CH == 16) tmem_ld_32x32b_x16(lanes + b * NT + c, r);
                    else tmem_ld_32x32b_x32(lanes + b * NT + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < CH; t += 4) {
                        const float4 s4 = *reinterpret_cast<const float4*>(sv + c + t);
                        acc[c + t] = fmaf(__uint_as_float(r[t]), s4.x, acc[c + t]);
                        acc[c + t + 1] = fmaf(__uint_as_float(r[t + 1]), s4.y, acc[c + t + 1]);
                        acc[c + t + 2] = fmaf(__uint_as_float(r[t + 2]), s4.z, acc[c + t + 2]);
                        acc[c + t + 3] = fmaf(__uint_as_float(r[t + 3]), s4.w, acc[c + t + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[b]);
            }
            const int rows = walk.rows(), s0 = walk.first(), n = walk.slab * 128 + col;
            bool write = whole;
            if (!whole) {
                float* mine = p.partials + ((int64_t)blockIdx.x * 2 + (head ? 1 : 0)) * NT * 128 + col;
#pragma unroll
                for (int t = 0; t < CW; ++t)
                    if (t0 + t < rows) __stcg(mine + (t0 + t) * 128, acc[t]);
                // pieces of this tile: CTAs cf .. cl
                const int64_t first = u0 + piece0 - (head ? 0 : kb);
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
                    for (int t = 0; t < CW; ++t) acc[t] = 0.0f;
                    for (int c = cf; c <= cl; ++c) {
                        const float* o = p.partials + ((int64_t)c * 2 + (c == cf ? 1 : 0)) * NT * 128 + col;
#pragma unroll
                        for (int t = 0; t < CW; ++t)
                            if (t0 + t < rows) acc[t] += __ldcg(o + (t0 + t) * 128);
                    }
                }
                named_bar_sync(1, 32 * C::EPI);   // s_last has been read
            }
            if (write && ok && n < p.N) {
#pragma unroll
                for (int t = 0; t < CW; ++t)
                    if (t0 + t < rows) {
                        const int s = s0 + t0 + t;
                        p.Y[(int64_t)s * p.N + n] = fp8_row(p, s) < 0 ? 0 : fp8_out(p, acc[t]);
                    }
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
// Many rows: 128 rows x 256 columns, one group of K a step, persistent.
//
// Two 256-column buffers alternate from step to step.  Roles: warp 0 TMA, warp 1 MMA, warps
// 2 and 3 the scales (two rows a lane, four groups ahead), warps 4..11 fold: warp e holds
// rows 32 (e % 4) .. + 31 (thread = row) and 128 of the columns, whose weight scale is one
// number, so a step costs a thread one scale and 128 fma.
// ---------------------------------------------------------------------------
struct Fp8TileCfg {
    static constexpr int BM = 128, BN = 256;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 256 * 128, STAGE = A_BYTES + B_BYTES, ST = 4;
    static constexpr int SC = 8;   // slots of scales [2][128]
    static constexpr int THREADS = 384, TMEM_COLS = 512;
    static constexpr int SC_OFF = ST * STAGE;
    static constexpr int SCHED_OFF = SC_OFF + SC * 256 * 4;
    static constexpr int BAR_OFF = SCHED_OFF + (int)((sizeof(Fp8Sched) + 15) / 16 * 16);
    static constexpr int NBAR = 2 * ST + 4 + 2 * SC + 1;
    static constexpr int TOTAL = BAR_OFF + NBAR * 8 + 16 + 1024;
    static_assert(TOTAL <= 227 * 1024, "tile kernel shared memory");
};

__global__ void __launch_bounds__(Fp8TileCfg::THREADS, 1)
    fp8_tile_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x)
{
    using C = Fp8TileCfg;
    constexpr int ST = C::ST, SC = C::SC;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);   // [SC][2][128]
    Fp8Sched& sched = *reinterpret_cast<Fp8Sched*>(smem + C::SCHED_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + ST;
    uint64_t* dfull = empty + ST;
    uint64_t* dempty = dfull + 2;
    uint64_t* sfull = dempty + 2;
    uint64_t* sempty = sfull + SC;
    uint64_t* done = sempty + SC;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G, slabs = (p.N + 255) / 256;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 8);
        }
        for (int i = 0; i < SC; ++i) {
            mbar_init(&sfull[i], 2);
            mbar_init(&sempty[i], 8);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (!fp8_schedule<C::BM>(sched, p, slabs)) return;
    const int tiles = sched.pre[p.E];
    if ((int)blockIdx.x >= tiles) return;
    if (warp == 1) {
        tmem_alloc(tslot, C::TMEM_COLS);
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
            int i = 0, y[4];
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                walk.at(tile);
                const int s0 = walk.first(), n0 = walk.slab * 256;
                if (p.rows) fp8_gather_rows(p, s0, walk.rows(), lane, y);
                for (int kb = 0; kb < G; ++kb, ++i) {
                    const int s = i % ST;
                    ok = all_wait(&empty[s], ((i / ST) & 1) ^ 1);
                    if (!ok) break;
                    uint8_t* st = smem + s * C::STAGE;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&full[s], C::STAGE);
                        tma_load_3d(&tm_w, &full[s], st + C::A_BYTES, n0, kb * 128, walk.e);
                        tma_load_3d(&tm_w, &full[s], st + C::A_BYTES + 16384, n0 + 128, kb * 128, walk.e);
                        if (!p.rows) tma_load_2d(&tm_x, &full[s], st, kb * 128, s0);
                    }
                    __syncwarp();
                    if (p.rows) tma_gather4(&tm_x, &full[s], st + lane * 512, kb * 128, y);
                }
            }
            if (!ok)
                for (int j = max(i - ST, 0); j < i; ++j) all_wait(&full[j % ST], (j / ST) & 1);
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            if (lane == 0) {
                constexpr uint32_t idesc = idesc_e4m3(256, false, true);
                bool ok = true;
                int i = 0;
                for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x)
                    for (int kb = 0; kb < G; ++kb, ++i) {
                        const int s = i % ST, b = i & 1;
                        if (!mbar_wait(&dempty[b], ((i >> 1) & 1) ^ 1) || !mbar_wait(&full[s], (i / ST) & 1)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a0 = smem_u32(smem + s * C::STAGE), b0 = a0 + C::A_BYTES;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_e4m3_ss(tmem + b * 256, smem_desc(a0 + 32 * kk, 16, 1024, 2),
                                        smem_desc(b0 + 4096 * kk, 16384, 1024, 2), idesc, kk > 0 ? 1u : 0u);
                        mma_commit(&empty[s]);
                        mma_commit(&dfull[b]);
                    }
                if (i > 0) {
                    mma_commit(done);
                    mbar_wait(done, 0);
                }
            }
        } else {
            // ---------------- scales: rows 2 r, 2 r + 1 of r = 0 .. 63 ----------------
            const int r = threadIdx.x - 64;
            bool ok = true;
            int i = 0;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                walk.at(tile);
                const int s0 = walk.first(), rows = walk.rows();
                int row[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    row[j] = 2 * r + j < rows ? fp8_row(p, s0 + 2 * r + j) : -2;
                    if (row[j] == -1 && walk.slab == 0) set_status(6u);
                }
                const float* w = p.ws + (int64_t)walk.e * G * p.NB + 2 * walk.slab;
                const bool wide = 2 * walk.slab + 1 < p.NB;
                float x[4][2], w0[4], w1[4];
                auto load = [&](int kb, int a) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[a][j] = row[j] >= 0 ? __ldg(p.xs + (int64_t)row[j] * G + kb) : 0.0f;
                    w0[a] = __ldg(w + (int64_t)kb * p.NB);
                    w1[a] = wide ? __ldg(w + (int64_t)kb * p.NB + 1) : 0.0f;
                };
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    if (a < G) load(a, a);
                for (int k0 = 0; k0 < G && ok; k0 += 4) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        if (k0 + a >= G || !ok) break;
                        const int s = i % SC;
                        ok = all_wait(&sempty[s], ((i / SC) & 1) ^ 1);
                        if (!ok) break;
                        float2* o = reinterpret_cast<float2*>(scales + s * 256);
                        o[r] = make_float2(__fmul_rn(x[a][0], w0[a]), __fmul_rn(x[a][1], w0[a]));
                        o[64 + r] = make_float2(__fmul_rn(x[a][0], w1[a]), __fmul_rn(x[a][1], w1[a]));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sfull[s]);
                        ++i;
                        if (k0 + a + 4 < G) load(k0 + a + 4, a);
                    }
                }
            }
        }
    } else {
        setmaxnreg_inc<216>();
        // ---------------- fold: thread = row, 128 columns ----------------
        const int q = warp & 3, half = (warp - 4) >> 2, r = 32 * q + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * 128;
        bool ok = true;
        int i = 0;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            float acc[128];
#pragma unroll
            for (int t = 0; t < 128; ++t) acc[t] = 0.0f;
            for (int kb = 0; kb < G; ++kb, ++i) {
                const int b = i & 1, s = i % SC;
                ok = all_wait(&sfull[s], (i / SC) & 1);
                if (!ok) break;
                const float sc = scales[s * 256 + half * 128 + r];
                ok = all_wait(&dfull[b], (i >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(lanes + b * 256 + c, v);
                    tmem_ld_wait();
                    if (c == 96) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&dempty[b]);
                            mbar_arrive(&sempty[s]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 32; ++t) acc[c + t] = fmaf(__uint_as_float(v[t]), sc, acc[c + t]);
                }
            }
            if (!ok) break;
            walk.at(tile);
            const int slot = walk.first() + r, n0 = walk.slab * 256 + half * 128;
            if (r < walk.rows()) {
                const bool zero = fp8_row(p, slot) < 0;
                uint16_t* y = p.Y + (int64_t)slot * p.N + n0;
#pragma unroll
                for (int c = 0; c < 128; c += 8) {
                    if (n0 + c < p.N) {
                        uint4 v = make_uint4(fp8_out2(p, acc[c], acc[c + 1]), fp8_out2(p, acc[c + 2], acc[c + 3]),
                                             fp8_out2(p, acc[c + 4], acc[c + 5]), fp8_out2(p, acc[c + 6], acc[c + 7]));
                        if (zero) v = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(y + c) = v;
                    }
                }
            }
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
