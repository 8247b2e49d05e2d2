// fp8_host.cuh -- launch configuration of the FP8 layer, the router and the experts' calls
// (included by qgemm.cu after its launch helpers).

namespace {

// ---------------------------------------------------------------------------
// FP8 quantizers
// ---------------------------------------------------------------------------
template <int T>
qg_status quantize_act_fp8(const void* X, int M, int K, uint8_t* Xq, float* xs, qg_stream_t stream)
{
    const uint32_t G = ((uint32_t)K + 127) / 128;
    const uint64_t groups = (uint64_t)M * G;
    if (groups > 0xFFFFFF00ull) return QG_ERR_SHAPE;
    const uint32_t grid = (uint32_t)((groups + 31) / 32);
    qg::quantize_act_fp8_kernel<T><<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t*>(X), (uint32_t)groups, K, G, Xq, xs);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
}

template <int T>
qg_status quantize_weight_fp8(const void* W, int E, int K, int N, uint8_t* Wq, float* ws, qg_stream_t stream)
{
    const dim3 grid((N + 127) / 128, (K + 127) / 128, E);
    qg::quantize_weight_fp8_kernel<T><<<grid, 512, 0, reinterpret_cast<cudaStream_t>(stream)>>>(W, K, N, Wq, ws);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
}

// ---------------------------------------------------------------------------
// FP8 products
// ---------------------------------------------------------------------------
// Rows, K and N are rounded up to tiles of at most 256 in 32 bits.
bool fp8_bad_shape(int M, int K, int N)
{
    constexpr int most = 0x7FFFFFFF - 255;
    return M < 0 || M > most || K < 16 || K % 16 || K > most || N < 16 || N % 16 || N > most;
}

// Rows of a TMA box of activations: what a tile can have.
int fp8_box(int S) { return S >= 128 ? 128 : (S + 7) / 8 * 8; }

// The workspace: counters and partial sums of split tiles (where K is long enough to be split),
// then, for experts, the rows in slot order.  256 columns a tile are assumed: the number of
// experts, and so the choice, is not known.
struct Fp8Workspace {
    size_t partials, rows, bytes;   // where the second and third part start, and all
};

Fp8Workspace fp8_carve(int S, int K, bool experts)
{
    const size_t grid = num_sms();
    const bool split = (K + 127) / 128 * 2 > qg::fp8_min_saved(experts ? 1 : fp8_box(S));
    Fp8Workspace w;
    w.partials = (grid * 8 + 255) / 256 * 256;
    w.rows = split ? w.partials + grid * 2 * 128 * 256 * sizeof(float) : 0;
    w.bytes = w.rows + (experts ? (size_t)S * K : 0);
    return w;
}

size_t fp8_workspace(int S, int K, bool experts) { return fp8_carve(S, K, experts).bytes; }

// The kernel's register split draws on what the block was launched with: a build that gives it
// fewer would wait for ever.
template <typename C, typename Kern>
qg_status fp8_check_registers(Kern kern)
{
    static std::atomic<int> fine{0};
    if (fine.load(std::memory_order_relaxed)) return QG_OK;
    cudaFuncAttributes a;
    QG_CUDA(cudaFuncGetAttributes(&a, kern));
    if (a.numRegs * C::THREADS < 128 * C::REGS_ISSUE + 256 * C::REGS_FOLD) {
        snprintf(g_last_error, sizeof(g_last_error), "FP8 tile kernel built with %d registers a thread", a.numRegs);
        return QG_ERR_UNSUPPORTED;
    }
    fine.store(1, std::memory_order_relaxed);
    return QG_OK;
}

// A token for the counters of split tiles: its low byte is 0, the rest is not.
unsigned long long fp8_token()
{
    unsigned long long t;
    do t = next_decode_token() << 8;
    while (t == 0);
    return t;
}

// The weights as {N, K, E} (boxes of 128 columns x 128 k), the activations as {K, rows} (boxes of
// 128 k x p.box rows).
qg_status fp8_maps(CUtensorMap* tw, CUtensorMap* tx, const uint8_t* X, int rows, const uint8_t* Wq, const qg::Fp8Params& p)
{
    const uint64_t N = p.N, K = p.K;
    qg_status st = make_tmap_3d(tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, N, K, p.E, N, N * K, 128, 128, 1,
                                CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QG_OK) return st;
    return make_tmap_2d(tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, X, K, rows, 128, p.box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int BN>
qg_status launch_fp8_tile(qg::Fp8Params p, const uint8_t* X, const uint8_t* Wq, void* ws, qg_stream_t stream)
{
    using C = qg::Fp8TileCfg<BN>;
    auto kern = qg::fp8_tile_kernel<BN>;
    static KernelInfo info;
    int occ = 1;
    qg_status st = prepare_kernel(info, kern, C::THREADS, C::TOTAL, &occ);
    if (st != QG_OK || (st = fp8_check_registers<C>(kern)) != QG_OK) return st;
    const Fp8Workspace w = fp8_carve(p.S, p.K, p.offsets != nullptr);
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.counters = reinterpret_cast<unsigned long long*>(base);
    p.partials = reinterpret_cast<float*>(base + w.partials);
    p.token = fp8_token();
    int rows = p.Mx;
    if (p.rows) {
        const dim3 g((p.S + 3) / 4, (p.K + 4095) / 4096);
        if ((st = launch_pdl(qg::fp8_rows_kernel, g, dim3(256), 0, stream, p, X, base + w.rows)) != QG_OK) return st;
        X = base + w.rows;
        rows = p.S;
    }
    CUtensorMap tw, tx;
    if ((st = fp8_maps(&tw, &tx, X, rows, Wq, p)) != QG_OK) return st;
    return launch_pdl(kern, dim3(num_sms()), dim3(C::THREADS), C::TOTAL, stream, p, tw, tx);
}

qg_status fp8_gemm(const uint8_t* Xq, const float* xs, int Mx, int K, const int32_t* rows, const int32_t* offsets, int S,
                   int E, const uint8_t* Wq, const float* ws, int N, void* Y, qg_dtype ydt, void* workspace,
                   size_t ws_bytes, qg_stream_t stream)
{
    const size_t need = fp8_workspace(S, K, offsets != nullptr);
    if (!Xq || !xs || !Wq || !ws || !Y || (need && !workspace)) return QG_ERR_NULL;
    if (misaligned(Xq) || misaligned(xs) || misaligned(rows) || misaligned(offsets) || misaligned(Wq) ||
        misaligned(ws) || misaligned(Y) || misaligned(workspace))
        return QG_ERR_ALIGN;
    if (ws_bytes < need) return QG_ERR_WORKSPACE;
    qg::Fp8Params p{};
    p.xs = xs;
    p.ws = ws;
    p.rows = rows;
    p.offsets = offsets;
    p.Y = static_cast<uint16_t*>(Y);
    p.Mx = Mx;
    p.S = S;
    p.E = E;
    p.K = K;
    p.N = N;
    p.G = (K + 127) / 128;
    p.NB = (N + 127) / 128;
    p.bf16 = ydt == QG_BF16;
    // an expert's tiles have some four times the average of rows at most, mostly
    p.join_rows = offsets ? (int)std::min<int64_t>(fp8_box(S), 4 * (((int64_t)S + E - 1) / E)) : fp8_box(S);
    p.box = fp8_box(S);   // the rest of a tile holds what it held: rows of sums that go nowhere
    // 256 columns a tile where those tiles still fill half of the GPU
    const int64_t m_tiles = (int64_t)(S + 127) / 128 + (offsets ? std::min(S, E) / 2 : 0);
    if (m_tiles * ((N + 255) / 256) * 2 < num_sms()) return launch_fp8_tile<128>(p, Xq, Wq, workspace, stream);
    return launch_fp8_tile<256>(p, Xq, Wq, workspace, stream);
}

// ---------------------------------------------------------------------------
// Router, slot maps, combine
// ---------------------------------------------------------------------------
template <int T>
qg_status route_topk(const qg::RouteParams& p, qg_stream_t stream)
{
    const int grid = (p.M + 3) / 4;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (p.E <= 32) qg::route_topk_kernel<T, 1><<<grid, 128, 0, st>>>(p);
    else if (p.E <= 64) qg::route_topk_kernel<T, 2><<<grid, 128, 0, st>>>(p);
    else if (p.E <= 128) qg::route_topk_kernel<T, 4><<<grid, 128, 0, st>>>(p);
    else if (p.E <= 256) qg::route_topk_kernel<T, 8><<<grid, 128, 0, st>>>(p);
    else qg::route_topk_kernel<T, 16><<<grid, 128, 0, st>>>(p);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
}

bool slots_bad_shape(int M, int topk, int E)
{
    return M < 0 || topk < 1 || E < 1 || E > qg::kMaxExperts || (int64_t)M * topk > 0x7FFFFFFF - qg::kSlotBlock;
}

size_t slots_workspace(int M, int topk, int E)
{
    const size_t blocks = ((size_t)M * topk + qg::kSlotBlock - 1) / qg::kSlotBlock;
    return blocks > 1 ? ((blocks + (blocks > qg::kSlotSum)) * E * sizeof(int32_t) + 255) / 256 * 256 : 0;
}

qg_status expert_slots(const int32_t* idx, int M, int topk, int E, int32_t* offsets, int32_t* slot_token,
                       int32_t* token_slot, void* workspace, size_t ws_bytes, qg_stream_t stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        QG_CUDA(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), st));
        return QG_OK;
    }
    const size_t need = slots_workspace(M, topk, E);
    if (need && !workspace) return QG_ERR_NULL;
    if (ws_bytes < need) return QG_ERR_WORKSPACE;
    const int n = M * topk, blocks = (n + qg::kSlotBlock - 1) / qg::kSlotBlock;
    const qg::SlotParams p{idx, offsets, slot_token, token_slot, static_cast<int32_t*>(workspace), n, topk, E, blocks};
    const dim3 threads(32 * qg::kSlotWarps);
    if (blocks > 1) {
        const qg_status r = launch_pdl(qg::slot_count_kernel, dim3(blocks), threads, 0, stream, p);
        if (r != QG_OK) return r;
    }
    if (blocks > qg::kSlotSum) {
        const qg_status r = launch_pdl(qg::slot_sum_kernel, dim3((E + 31) / 32), dim3(1024), 0, stream, p);
        if (r != QG_OK) return r;
    }
    return launch_pdl(qg::slot_place_kernel, dim3(blocks), threads, 0, stream, p);
}

qg_status combine_experts(const void* D, qg_dtype dt, int S, int N, const int32_t* token_slot, const float* weights,
                          int M, int topk, void* Y, qg_stream_t stream)
{
    const int64_t items = (int64_t)M * (N / 8);
    if ((items + 255) / 256 > 0x7FFFFFFF) return QG_ERR_SHAPE;
    const unsigned grid = (unsigned)((items + 255) / 256);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uint16_t* d = static_cast<const uint16_t*>(D);
    uint16_t* y = static_cast<uint16_t*>(Y);
    if (dt == QG_BF16) qg::combine_experts_kernel<true><<<grid, 256, 0, st>>>(d, S, N, M, topk, token_slot, weights, y);
    else qg::combine_experts_kernel<false><<<grid, 256, 0, st>>>(d, S, N, M, topk, token_slot, weights, y);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
}

}  // namespace
