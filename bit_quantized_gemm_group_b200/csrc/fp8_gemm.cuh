// fp8_gemm.cuh -- products of e4m3 operands with a scale for each 128 of K:
//
//   Y[m][n] = rn( sum_g xs[m][g] ws[g][n / 128] sum_{k in g} Xq[m][k] Wq[k][n] )   (fp32)
//
// and the same per expert over the rows of its slots.
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"

namespace qg {

struct Fp8Params {
    const uint8_t* Xq;       // [Mx][K]
    const float* xs;         // [Mx][G]
    const uint8_t* Wq;       // [E][K][N]
    const float* ws;         // [E][G][NB]
    const int32_t* rows;     // slot -> row of Xq, or NULL: the slot itself
    const int32_t* offsets;  // [E + 1], or NULL: one expert with all S slots
    uint16_t* Y;             // [S][N]
    int Mx, S, E, K, N, G, NB;
    bool bf16;
};

// Simple form: 64 slots x 64 columns per CTA, fp32 FMA.
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(const Fp8Params p)
{
    __shared__ float a[64][33], b[32][65];
    int e = 0, s0 = 0, s1 = p.S, tile = blockIdx.y;
    if (p.offsets) {
        bool bad = false;   // offsets that do not ascend from 0 to at most S: nothing is computed
        for (int i = threadIdx.x; i <= p.E; i += 256) {
            const int o = p.offsets[i];
            bad |= i == 0 ? o != 0 : o < p.offsets[i - 1] || o > p.S;
        }
        if (__syncthreads_or(bad)) {
            set_status(6u);
            return;
        }
        for (e = 0; e < p.E; ++e) {
            s0 = p.offsets[e];
            s1 = p.offsets[e + 1];
            const int t = (s1 - s0 + 63) / 64;
            if (tile < t) break;
            tile -= t;
        }
        if (e == p.E) return;
    }
    s0 += tile * 64;
    const int n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, part[4][4];
    for (int g = 0; g < p.G; ++g) {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) part[i][j] = 0.0f;
        for (int k0 = g * 128; k0 < min(p.K, g * 128 + 128); k0 += 32) {
            __syncthreads();
            for (int i = threadIdx.x; i < 64 * 32; i += 256) {
                const int r = i >> 5, k = k0 + (i & 31), s = s0 + r;
                int row = s < s1 ? (p.rows ? p.rows[s] : s) : -1;
                float v = 0.0f;
                if (row >= 0 && row < p.Mx && k < p.K) {
                    __nv_fp8_e4m3 f;
                    f.__x = p.Xq[(int64_t)row * p.K + k];
                    v = float(f);
                }
                a[r][i & 31] = v;
            }
            for (int i = threadIdx.x; i < 32 * 64; i += 256) {
                const int k = k0 + (i >> 6), n = n0 + (i & 63);
                float v = 0.0f;
                if (k < p.K && n < p.N) {
                    __nv_fp8_e4m3 f;
                    f.__x = p.Wq[((int64_t)e * p.K + k) * p.N + n];
                    v = float(f);
                }
                b[i >> 6][i & 63] = v;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[ty * 4 + i][k], b[k][tx + 16 * j], part[i][j]);
        }
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + ty * 4 + i;
            const int row = s < s1 ? (p.rows ? p.rows[s] : s) : -1;
            const float x = row >= 0 && row < p.Mx ? p.xs[(int64_t)row * p.G + g] : 0.0f;
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                if (n < p.N) acc[i][j] = fmaf(x * p.ws[((int64_t)e * p.G + g) * p.NB + n / 128], part[i][j], acc[i][j]);
            }
        }
    }
    for (int i = 0; i < 4; ++i) {
        const int s = s0 + ty * 4 + i;
        if (s >= s1) continue;
        if (p.rows && threadIdx.x == 0 && (uint32_t)p.rows[s] >= (uint32_t)p.Mx) set_status(6u);
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            if (n < p.N) p.Y[(int64_t)s * p.N + n] = p.bf16 ? f32_to_bf16_bits(acc[i][j]) : f32_to_f16_bits(acc[i][j]);
        }
    }
}

}  // namespace qg
