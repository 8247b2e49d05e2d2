"""The FP8 layer's and the experts' calls refuse what they cannot run, before any launch (CPU: no CUDA call is
reached), at the C ABI and in the Python binding."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = P(0x10000)   # aligned fake device address (never dereferenced: validation fails first)
B = P(0x10008)   # not 16-byte aligned
WS = (A, 1 << 40)
F = ctypes.c_float


def gemm(Xq=A, xs=A, M=4, K=256, Wq=A, ws=A, N=64, Y=A, ydt=1, wsp=WS):
    return "qg_gemm_fp8", (Xq, xs, M, K, Wq, ws, N, Y, ydt, *wsp, None)


def experts(Xq=A, xs=A, Mx=4, K=256, tok=A, off=A, S=8, E=4, Wq=A, ws=A, N=64, Y=A, ydt=1, wsp=WS):
    return "qg_gemm_fp8_experts", (Xq, xs, Mx, K, tok, off, S, E, Wq, ws, N, Y, ydt, *wsp, None)


def route(lg=A, dt=2, M=4, E=64, bias=None, score=0, ng=1, kg=1, gt=1, k=8, idx=A, w=A):
    return "qg_route_topk", (lg, dt, M, E, bias, score, ng, kg, gt, k, 1, F(1.0), idx, w, None)


def slots(idx=A, M=4, k=8, E=64, off=A, st=A, ts=A, wsp=WS):
    return "qg_expert_slots", (idx, M, k, E, off, st, ts, *wsp, None)


def combine(D=A, dt=1, S=32, N=64, ts=A, w=A, M=4, k=8, Y=A):
    return "qg_combine_experts", (D, dt, S, N, ts, w, M, k, Y, None)


def act(X=A, dt=1, M=4, K=256, Xq=A, xs=A):
    return "qg_quantize_act_fp8", (X, dt, M, K, Xq, xs, None)


def weight(W=A, dt=2, E=1, K=256, N=64, Wq=A, ws=A):
    return "qg_quantize_weight_fp8", (W, dt, E, K, N, Wq, ws, None)


OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 10


@pytest.mark.parametrize("call,want", [
    (act(dt=2), DTYPE), (act(dt=9), DTYPE), (act(K=8), SHAPE), (act(K=24), SHAPE), (act(M=-1), SHAPE),
    (act(X=None), NULL), (act(Xq=None), NULL), (act(xs=None), NULL), (act(X=B), ALIGN), (act(xs=B), ALIGN),
    (act(X=None, M=0, Xq=None, xs=None), OK),
    (weight(dt=3), DTYPE), (weight(N=72), SHAPE), (weight(K=136), SHAPE), (weight(E=0), SHAPE),
    (weight(E=65536), SHAPE), (weight(W=None), NULL), (weight(Wq=B), ALIGN),
    (gemm(ydt=2), DTYPE), (gemm(K=200), SHAPE), (gemm(K=0), SHAPE), (gemm(N=60), SHAPE), (gemm(M=-1), SHAPE),
    (gemm(Xq=None), NULL), (gemm(xs=None), NULL), (gemm(Wq=None), NULL), (gemm(ws=None), NULL), (gemm(Y=None), NULL),
    (gemm(Y=B), ALIGN), (gemm(ws=B), ALIGN), (gemm(M=0, Xq=None, Y=None, wsp=(None, 0)), OK),
    (experts(ydt=7), DTYPE), (experts(E=0), SHAPE), (experts(E=513), SHAPE), (experts(K=24), SHAPE),
    (experts(S=-1), SHAPE), (experts(Mx=0), SHAPE), (experts(tok=None), SHAPE),   # without a map: as many rows as slots
    (experts(off=None), NULL), (experts(Wq=None), NULL), (experts(tok=B), ALIGN), (experts(off=B), ALIGN),
    (experts(S=0, Xq=None, Y=None, off=None), OK),
    (route(dt=3), DTYPE), (route(score=2), DTYPE), (route(E=513), SHAPE), (route(E=0), SHAPE), (route(k=0), SHAPE),
    (route(k=33), SHAPE), (route(E=4, k=5), SHAPE), (route(ng=3), SHAPE), (route(ng=64), SHAPE),
    (route(ng=8, kg=9), SHAPE), (route(ng=8, kg=0), SHAPE), (route(gt=3), SHAPE), (route(gt=0), SHAPE),
    (route(E=16, ng=8, kg=2, k=8), SHAPE),   # more choices than the kept groups hold
    (route(lg=None), NULL), (route(idx=None), NULL), (route(w=None), NULL), (route(bias=B), ALIGN), (route(lg=B), ALIGN),
    (route(M=0, lg=None, idx=None, w=None), OK),
    (slots(E=0), SHAPE), (slots(E=513), SHAPE), (slots(k=0), SHAPE), (slots(M=1 << 28, k=8), SHAPE),
    (slots(off=None), NULL), (slots(idx=None), NULL), (slots(st=None), NULL), (slots(ts=B), ALIGN),
    (combine(dt=2), DTYPE), (combine(N=12), SHAPE), (combine(N=0), SHAPE), (combine(k=0), SHAPE), (combine(S=-1), SHAPE),
    (combine(D=None), NULL), (combine(ts=None), NULL), (combine(w=None), NULL), (combine(Y=None), NULL),
    (combine(Y=B), ALIGN), (combine(M=0, D=None, ts=None, w=None, Y=None), OK),
])
def test_refused(call, want):
    import bit_quantized_gemm_group_b200 as q
    assert getattr(q.lib(), call[0])(*call[1]) == want


@pytest.mark.parametrize("op,M,K,N,call", [(5, 4, 4096, 4096, gemm), (6, 8, 4096, 4096, experts), (7, 4096, 8, 64, slots)])
def test_workspace_is_required_where_it_has_a_size(op, M, K, N, call):
    import bit_quantized_gemm_group_b200 as q
    need = q.qg_workspace_size(op, M, K, N)
    kw = {"M": M, "k": K, "E": N} if op == 7 else {"K": K, "N": N, ("M" if op == 5 else "S"): M}
    if need == 0:
        return
    for wsp, want in (((None, 0), NULL), ((A, need - 1), WORKSPACE), ((B, need), ALIGN)):
        name, args = call(**kw, wsp=wsp)
        assert getattr(q.lib(), name)(*args) == want
    assert q.qg_workspace_size(op, 0, K, N) == 0


def test_binding_refuses_wrong_tensors():
    """Types, ranks, shapes and devices are looked at before the library is called."""
    import bit_quantized_gemm_group_b200 as q
    t = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt)   # noqa: E731
    f8, i32 = torch.float8_e4m3fn, torch.int32
    with pytest.raises(ValueError, match="one GPU"):
        q.qg_quantize_act_fp8(t(4, 256, dt=torch.bfloat16), t(4, 256, dt=f8), t(4, 2))
    with pytest.raises(ValueError, match="dtype"):
        q.qg_quantize_act_fp8(t(4, 256), t(4, 256, dt=f8), t(4, 2))
    with pytest.raises(ValueError, match="dimensions"):
        q.qg_quantize_act_fp8(t(256, dt=torch.bfloat16), t(4, 256, dt=f8), t(4, 2))
    with pytest.raises(ValueError, match="dimensions"):
        q.qg_quantize_weight_fp8(t(256), t(256, dt=f8), t(2))
    with pytest.raises(ValueError, match="dimensions"):
        q.qg_gemm_fp8(t(4, 256, dt=f8), t(4, 2), t(1, 256, 64, dt=f8), t(2, 1), t(4, 64, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="score"):
        q.qg_route_topk(t(4, 8), None, t(4, 2, dt=i32), t(4, 2), score="tanh")
    with pytest.raises(ValueError, match="dimensions"):
        q.qg_expert_slots(t(4, 2, dt=i32), t(9, 1, dt=i32), t(8, dt=i32), t(4, 2, dt=i32))
    with pytest.raises(ValueError, match="dimensions"):
        q.qg_gemm_fp8_experts(t(4, 256, dt=f8), t(4, 2), None, t(3, dt=i32), t(256, 64, dt=f8), t(2, 1), t(4, 64))
    with pytest.raises(ValueError, match="one GPU"):
        q.qg_combine_experts(t(8, 64, dt=torch.float16), t(4, 2, dt=i32), t(4, 2), t(4, 64, dt=torch.float16))
