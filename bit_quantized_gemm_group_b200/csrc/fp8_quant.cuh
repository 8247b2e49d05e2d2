// fp8_quant.cuh -- e4m3 operands of the FP8 layer: activations in groups of 128 along a
// row, weights in blocks of 128 x 128, one fp32 scale each.
//
//   s = max|x| / 448 (fp32),  code = e4m3(fp32(x / s)), both rounded to nearest even
//   s == 0 (a zero group, or one whose scale underflows): codes 0
//   a NaN or an infinity in the group: s = NaN, codes 0, QG_ERR_NONFINITE -- the product
//   of such a group is NaN, as the unquantized one would be
// ("AI Infra guide, ch.4 Quantization" sec. 1.1-1.3 for the scale, sec. 5 for e4m3.)
// 448 is the largest e4m3 number, so the largest element gets the code 448.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace qg {

constexpr float kE4M3Max = 448.0f;

enum Fp8In { IN_F16 = 0, IN_BF16 = 1, IN_F32 = 2 };

// two e4m3 codes, `lo` in the low byte (round to nearest even, saturating)
QG_DEV_INLINE uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scale of a group from its largest magnitude; `q` divides by it.
struct Fp8Scale {
    float s, r;
    bool plain;   // r may stand for the division
    QG_DEV_INLINE explicit Fp8Scale(float amax)
    {
        s = __fdiv_rn(amax, kE4M3Max);
        if (!(amax <= 3.402823466e38f)) {   // Inf or NaN
            set_status(5u);
            s = __int_as_float(0x7fffffff);
        }
        plain = s > 0x1p-60f && s < 0x1p60f;   // no product below underflows or overflows
        r = plain ? __frcp_rn(s) : 0.0f;
    }
    QG_DEV_INLINE float q(float x) const { return s > 0.0f ? __fdiv_rn(x, s) : 0.0f; }
    // For x of at most 11 significant bits (fp16, bf16), where `plain`: a quotient that has the
    // same e4m3 code as fp32(x / s).  Markstein's division: with r = fp32(1 / s) and the exact
    // remainder x - q0 s, q0 + (x - q0 s) r is within 2^-23 of an ulp of x / s before it is rounded,
    // so it can only differ from fp32(x / s) where x / s is that near to a midpoint of two fp32
    // numbers, and the code only where that midpoint is next to a midpoint c (5 significant
    // bits) of two e4m3 numbers.  x - c s is then a multiple of s's last bit times 2^-4, which
    // forces s to within two last bits of a multiple of 1/8 and x = c k / 8, and then x / s is
    // off that fp32 midpoint by more than the bound.  The remainder is taken as q0 s - x, whose zero is
    // +0 for x of either sign, so that -0 stays -0 as in the quotient.  Three instructions for about ten.
    QG_DEV_INLINE float quick(float x) const
    {
        const float q0 = __fmul_rn(x, r);
        return fmaf(-fmaf(q0, s, -x), r, q0);
    }
};

template <int T>
QG_DEV_INLINE float half_word(uint32_t w, int hi)
{
    if (T == IN_BF16) return __uint_as_float(hi ? (w & 0xFFFF0000u) : (w << 16));
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return hi ? __high2float(h) : __low2float(h);
}

// Activations [M][K], K % 16 == 0.  Eight lanes share a group, each with 16 elements (two
// 16-byte loads, one 16-byte store); a warp takes four groups.  Groups are numbered row by
// row over the whole tensor; the last of a row may be short.  HBM-bound once the division is
// three instructions (8192 x 28672 bf16: 178 -> 124 us, 5.7 TB/s; fp32 divisions filled the
// issue slots).
template <int T>
__global__ void __launch_bounds__(256) quantize_act_fp8_kernel(const uint16_t* __restrict__ X, uint32_t groups, int K,
                                                               uint32_t G, uint8_t* __restrict__ Xq,
                                                               float* __restrict__ xs)
{
    const uint32_t id = blockIdx.x * 32u + (threadIdx.x >> 3), l = threadIdx.x & 7;
    if (id >= groups) return;   // all eight lanes of the group
    const uint32_t row = id / G, k = (id - row * G) * 128 + l * 16;
    const bool in = k < (uint32_t)K;
    const int64_t at = (int64_t)row * K + k;
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) {
        const uint4 a = ldg_stream_v4(X + at), b = ldg_stream_v4(X + at + 8);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    // the magnitudes' bits order like the magnitudes, with Inf and NaN above every number
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    const uint32_t lanes = 0xFFu << (threadIdx.x & 24);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(lanes, m, o));
    const Fp8Scale s(half_word<T>(max(m & 0xFFFFu, m >> 16), 0));
    if (l == 0) xs[id] = s.s;
    if (!in) return;
    uint32_t o[4];
    if (s.plain) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = e4m3x2(s.quick(half_word<T>(w[2 * i], 0)), s.quick(half_word<T>(w[2 * i], 1))) |
                   e4m3x2(s.quick(half_word<T>(w[2 * i + 1], 0)), s.quick(half_word<T>(w[2 * i + 1], 1))) << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = e4m3x2(s.q(half_word<T>(w[2 * i], 0)), s.q(half_word<T>(w[2 * i], 1))) |
                   e4m3x2(s.q(half_word<T>(w[2 * i + 1], 0)), s.q(half_word<T>(w[2 * i + 1], 1))) << 16;
    }
    *reinterpret_cast<uint4*>(Xq + at) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Weights [E][K][N] (fp32, bf16 or fp16), N % 16 == 0: one CTA per block of 128 x 128, held
// in registers between the maximum and the codes.  Thread (q, r) has columns 4q .. 4q+3 of
// rows r, r + 16, ..: a warp reads and writes whole row segments.  4096 x 12288: fp32 60 us, 4.2
// TB/s, bf16 54 us, 2.8 TB/s (two CTAs fit an SM, and their load and store phases leave HBM idle in
// between; three, with spills, were no faster; a checked three-instruction quotient for fp32
// slower, 64 us).
template <int T>
__global__ void __launch_bounds__(512) quantize_weight_fp8_kernel(const void* __restrict__ W, int K, int N,
                                                                  uint8_t* __restrict__ Wq, float* __restrict__ ws)
{
    const int nb = blockIdx.x, kb = blockIdx.y;
    const int64_t e = blockIdx.z;
    const int c = nb * 128 + 4 * (threadIdx.x & 31), r0 = kb * 128 + (threadIdx.x >> 5);
    float v[8][4];
    float a = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const int64_t at = (e * K + r) * N + c;
        if (r < K && c < N) {
            if constexpr (T == IN_F32) {
                const uint4 x = ldg_stream_v4(static_cast<const float*>(W) + at);
                v[i][0] = __uint_as_float(x.x);
                v[i][1] = __uint_as_float(x.y);
                v[i][2] = __uint_as_float(x.z);
                v[i][3] = __uint_as_float(x.w);
            } else {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(W) + at));
                v[i][0] = half_word<T>(x.x, 0);
                v[i][1] = half_word<T>(x.x, 1);
                v[i][2] = half_word<T>(x.y, 0);
                v[i][3] = half_word<T>(x.y, 1);
            }
        } else {
            v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bad |= !isfinite(v[i][j]);
            a = fmaxf(a, fabsf(v[i][j]));
        }
    }
    if (bad) a = __int_as_float(0x7f800000);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    __shared__ float red[16];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = red[threadIdx.x & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const Fp8Scale s(a);
    if (threadIdx.x == 0) ws[(e * gridDim.y + kb) * gridDim.x + nb] = s.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = T != IN_F32 && s.plain ? s.quick(v[i][j]) : s.q(v[i][j]);
        if (r < K && c < N)
            *reinterpret_cast<uint32_t*>(Wq + (e * K + r) * N + c) = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
    }
}

}  // namespace qg
