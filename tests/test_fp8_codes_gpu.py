"""The e4m3 codes of the quantizers byte by byte: the sign of zero, and every fp16 quotient."""
import pytest
import torch

import bit_quantized_gemm_group_b200 as q

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def e4m3(v):
    """The nearest e4m3 value (ties to even) of fp32 values, by arithmetic in 64 bits; the sign of zero is kept."""
    v = v.double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((v.abs() / step).round().mul(step).clamp(max=448.0), v)


def bytes_of(x, amax):
    """The codes of x in groups of the largest magnitudes `amax` (of x's shape).  Quotients of fp32 numbers in 64 bits,
    rounded to fp32, are the fp32 quotients (53 >= 2 * 24 + 2)."""
    s = (amax.double() / 448.0).float().double()
    quot = (x.double() / torch.where(s > 0, s, 1.0)).float()
    return torch.where(s > 0, e4m3(quot), 0.0).to(F8).view(torch.uint8)


def zeros_of_both_signs(rows, columns, dtype):
    """Group (row) 0: ordinary; 1: zeros alone; 2: too small a scale to divide by in short; 3: too large a one."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, columns, generator=g, device="cuda")
    x[:, ::3] = 0.0
    x[:, 1::6] = -0.0
    x[:, 2::6] *= 1e-6                               # what rounds to zero keeps its sign
    x[1::4] = torch.copysign(torch.zeros_like(x[1::4]), x[1::4])
    if dtype != torch.float16:
        x[2::4] *= 2.0 ** -80
        x[3::4] *= 2.0 ** 80
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_activations_keep_the_sign_of_zero(dtype):
    X = zeros_of_both_signs(8, 128, dtype)
    Xq, xs = torch.empty(8, 128, dtype=F8, device="cuda"), torch.empty(8, 1, device="cuda")
    q.qg_quantize_act_fp8(X, Xq, xs)
    want = bytes_of(X, X.float().abs().amax(1, keepdim=True).expand(8, 128))
    assert (want == 0x80).any()
    assert torch.equal(Xq.view(torch.uint8), want)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_weights_keep_the_sign_of_zero(dtype):
    for kind in range(4):
        W = zeros_of_both_signs(4, 128 * 128, dtype)[kind].view(128, 128)
        Wq, ws = torch.empty(128, 128, dtype=F8, device="cuda"), torch.empty(1, 1, device="cuda")
        q.qg_quantize_weight_fp8(W, Wq, ws)
        assert torch.equal(Wq.view(torch.uint8), bytes_of(W, W.float().abs().amax().expand(128, 128)))
    assert q.qg_device_status() == q.QG_OK


def test_every_fp16_quotient():
    """Every fp16 significand under the scale of every other one, over 21 binades: from the largest code to zero."""
    sig = torch.arange(1024, 2048, device="cuda") / 1024.0
    amax = sig * 2.0 ** 15                           # a row each; the largest is 65504
    part = torch.cat([sig, sig[:119]]).view(9, 127)  # nine groups of 127 beside the largest
    x = part[None] * torch.exp2(15.0 - torch.arange(21, device="cuda"))[:, None, None]       # [21, 9, 127]
    x = torch.minimum(x.reshape(1, 189, 127), amax[:, None, None])
    x[..., ::2] *= -1.0
    X = torch.cat([amax[:, None, None].expand(1024, 189, 1), x], 2).to(torch.float16).view(1024, 189 * 128)
    assert torch.equal(X.view(1024, 189, 128)[..., 1:].float(), x)      # all of them are fp16 numbers
    Xq, xs = torch.empty(X.shape, dtype=F8, device="cuda"), torch.empty(1024, 189, device="cuda")
    q.qg_quantize_act_fp8(X, Xq, xs)
    for rows in range(0, 1024, 128):
        at = slice(rows, rows + 128)
        want = bytes_of(X[at], amax[at, None].expand(128, 189 * 128))
        assert torch.equal(Xq[at].view(torch.uint8), want)
    assert q.qg_device_status() == q.QG_OK
