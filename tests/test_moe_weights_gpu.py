"""The router's weights are binary64 values rounded once to fp32."""
import pytest
import torch

import bit_quantized_gemm_group_b200 as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("spread", [0.5, 2.0, 8.0])
@pytest.mark.parametrize("E,topk,kw", [
    (64, 8, {}), (256, 8, {"renorm": False}), (40, 1, {"renorm": False, "scale": 2.5}), (512, 32, {}),
    (64, 6, {"score": "sigmoid"}), (128, 8, {"score": "sigmoid", "renorm": False, "scale": 16.0}),
    (256, 8, {"score": "sigmoid", "bias": True, "n_group": 8, "topk_group": 4, "group_top": 2, "scale": 2.5}),
    (256, 8, {"bias": True, "renorm": False}), (160, 6, {"n_group": 8, "topk_group": 3, "renorm": False}),
])
def test_weights_are_rounded_once(E, topk, kw, spread, dtype):
    kw, M = dict(kw), 3000
    g = torch.Generator(device="cuda").manual_seed(E + topk)
    x = (torch.randn(M, E, generator=g, device="cuda") * spread).to(dtype)
    x[5, topk:] = -torch.inf                         # as many experts as choices
    x[6] = -torch.inf                                # none
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if kw.pop("bias", False) else None
    idx = torch.empty(M, topk, dtype=torch.int32, device="cuda")
    w = torch.full((M, topk), torch.nan, device="cuda")
    q.qg_route_topk(x, bias, idx, w, **kw)
    assert q.qg_device_status() == q.QG_OK
    v = x.double()
    score = torch.sigmoid(v) if kw.get("score") == "sigmoid" else torch.softmax(v, 1).nan_to_num(0.0)
    ref = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0).long()), 0.0)
    if kw.get("renorm", True):
        total = ref.sum(1, keepdim=True)
        ref = torch.where(total > 0, ref / total, 0.0)
    ref = ref * kw.get("scale", 1.0)
    # half a step of fp32 (below 2^-126 half of its smallest one), and what both sides' binary64 is off by: 512 sums and
    # a handful of functions and quotients, 2^-52 each
    tol = ref * (2.0 ** -24 + 600 * 2.0 ** -52) + 2.0 ** -150
    off = (w.double() - ref).abs()
    assert (off <= tol).all(), f"off by {float((off / ref.clamp(min=2.0 ** -126)).max() * 2 ** 24):.3f} half steps"
    assert not w[6].any() and (idx[6] == -1).all()
