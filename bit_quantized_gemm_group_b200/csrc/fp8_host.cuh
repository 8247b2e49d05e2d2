// fp8_host.cuh -- launch configuration of the FP8 layer, the router and the experts' calls
// (included by qgemm.cu after its launch helpers).

namespace {

// ---------------------------------------------------------------------------
// FP8 quantizers
// ---------------------------------------------------------------------------
template <int T>
qg_status quantize_act_fp8(const void* X, int M, int K, uint8_t* Xq, float* xs, qg_stream_t stream)
{
    const uint32_t G = (K + 127) / 128;
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
bool fp8_bad_shape(int K, int N) { return K < 16 || K % 16 || N < 16 || N % 16; }

size_t fp8_workspace(int M, int K, int N, bool experts) { return 0; }

qg_status fp8_gemm(const uint8_t* Xq, const float* xs, int Mx, int K, const int32_t* rows, const int32_t* offsets, int S,
                   int E, const uint8_t* Wq, const float* ws, int N, void* Y, qg_dtype ydt, void* workspace,
                   size_t ws_bytes, qg_stream_t stream)
{
    if (!Xq || !xs || !Wq || !ws || !Y) return QG_ERR_NULL;
    if (misaligned(Xq) || misaligned(xs) || misaligned(rows) || misaligned(offsets) || misaligned(Wq) ||
        misaligned(ws) || misaligned(Y) || misaligned(workspace))
        return QG_ERR_ALIGN;
    const size_t need = fp8_workspace(S, K, N, offsets != nullptr);
    if (need && !workspace) return QG_ERR_NULL;
    if (need > ws_bytes) return QG_ERR_WORKSPACE;
    const qg::Fp8Params p{Xq, xs, Wq, ws, rows, offsets, static_cast<uint16_t*>(Y), Mx, S, E, K, N,
                          (K + 127) / 128, (N + 127) / 128, ydt == QG_BF16};
    const int tiles = offsets ? S / 64 + std::min(S, E) : (S + 63) / 64;
    qg::fp8_gemm_simple_kernel<<<dim3((N + 63) / 64, tiles), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
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
    return (blocks * E * sizeof(int32_t) + 255) / 256 * 256;
}

qg_status expert_slots(const int32_t* idx, int M, int topk, int E, int32_t* offsets, int32_t* slot_token,
                       int32_t* token_slot, void* workspace, size_t ws_bytes, qg_stream_t stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        QG_CUDA(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), st));
        return QG_OK;
    }
    if (!workspace) return QG_ERR_NULL;
    if (ws_bytes < slots_workspace(M, topk, E)) return QG_ERR_WORKSPACE;
    const int n = M * topk, blocks = (n + qg::kSlotBlock - 1) / qg::kSlotBlock;
    const qg::SlotParams p{idx, offsets, slot_token, token_slot, static_cast<int32_t*>(workspace), n, topk, E, blocks};
    qg::slot_count_kernel<<<blocks, 256, 0, st>>>(p);
    qg::slot_place_kernel<<<blocks, 256, 0, st>>>(p);
    QG_CUDA(cudaGetLastError());
    return QG_OK;
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
