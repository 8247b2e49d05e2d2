"""The router, the slot maps and the weighted sum on the GPU, and a run of all of them around the experts' products."""
import math

import pytest
import torch

import bit_quantized_gemm_group_b200 as q

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def route(logits, bias, topk, **kw):
    idx = torch.full((logits.shape[0], topk), -9, dtype=torch.int32, device="cuda")
    w = torch.full((logits.shape[0], topk), NAN, device="cuda")
    q.qg_route_topk(logits, bias, idx, w, **kw)
    return idx, w


def order(vals):
    """Indices by falling value, the lower first among equals."""
    return sorted(range(len(vals)), key=lambda i: (-vals[i], i))


def route_ref(logits, bias, topk, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """Token by token in Python floats (64 bits), straight from the definition."""
    idx, weights = [], []
    b = [0.0] * logits.shape[1] if bias is None else bias.double().tolist()
    for row in logits.double().tolist():
        E = len(row)
        bad = any(math.isnan(x) or x == INF for x in row)
        top = max(row)
        if bad or top == -INF:
            s = [0.0] * E
        elif score == "softmax":
            s = [math.exp(x - top) for x in row]
            s = [x / math.fsum(s) for x in s]
        else:
            s = [1.0 / (1.0 + math.exp(-x)) if x > -700 else math.exp(x) if x > -INF else 0.0 for x in row]
        key = [-INF if row[e] == -INF else s[e] + b[e] for e in range(E)]
        if bad or any(math.isnan(k) or k == INF for k in key):
            key = [-INF] * E
        if n_group > 1:
            size = E // n_group
            value = [sum(sorted(key[g * size:(g + 1) * size], reverse=True)[:group_top]) for g in range(n_group)]
            kept = order(value)[:topk_group]
            key = [key[e] if e // size in kept else -INF for e in range(E)]
        pick = [e if key[e] > -INF else -1 for e in order(key)[:topk]]
        w = [s[e] if e >= 0 else 0.0 for e in pick]
        if renorm:
            t = math.fsum(w)
            w = [x / t if t > 0 else 0.0 for x in w]
        idx.append(pick)
        weights.append([x * scale for x in w])
    return torch.tensor(idx, dtype=torch.int32, device="cuda"), torch.tensor(weights, dtype=torch.float64, device="cuda")


def assert_weights(w, ref):
    """Computed in at least fp32 from the scores: the exponential and its argument's rounding, sums, the quotients and the
    rounding of the result stay within 16 half steps of fp32 (2 ulp of expf at most, one each for the rest)."""
    assert ((w.double() - ref).abs() <= 16 * 2.0 ** -24 * ref + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,E,topk,kw", [
    (1, 1, 1, {}), (3, 8, 2, {}), (7, 64, 8, {"renorm": False}), (5, 33, 5, {"score": "sigmoid"}),
    (16, 128, 8, {"score": "sigmoid", "scale": 2.5}), (9, 160, 6, {"n_group": 8, "topk_group": 3}),
    (40, 256, 8, {"score": "sigmoid", "n_group": 8, "topk_group": 4, "group_top": 2, "bias": True}),
    (6, 512, 32, {"bias": True}), (4, 96, 4, {"n_group": 32, "topk_group": 2, "group_top": 2}),
    (11, 24, 24, {}), (5, 300, 12, {"score": "sigmoid", "bias": True, "renorm": False}),
    (8, 16, 2, {"n_group": 16, "topk_group": 2, "group_top": 2, "bias": True}),
])
def test_route(M, E, topk, kw, dtype):
    kw = dict(kw)
    x = (torch.randn(M, E, generator=gen(M + E), device="cuda") * 2).to(dtype)   # 16-bit logits: many equal ones
    bias = torch.randn(E, generator=gen(E), device="cuda") * 0.1 if kw.pop("bias", False) else None
    idx, w = route(x, bias, topk, **kw)
    ri, rw = route_ref(x, bias, topk, **kw)
    assert torch.equal(idx, ri)
    assert_weights(w, rw)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_equal_and_nearly_equal_keys(score):
    """Equal keys go to the lower expert; keys that differ by less than fp32 resolves are still told apart."""
    E = 64
    x = torch.zeros(4, E, device="cuda")
    x[1] = torch.tensor([1.0, 2.0] * 32)
    x[2] = 30.0 + torch.arange(E, device="cuda") * 2.0 ** -18         # sigmoid: all 1 in fp32
    x[3] = torch.randn(E, generator=gen(1), device="cuda")
    bias = torch.zeros(E, device="cuda")
    idx, w = route(x, None, 6, score=score)
    ri, rw = route_ref(x, None, 6, score=score)
    assert torch.equal(idx, ri)
    assert_weights(w, rw)
    # zeros of both signs are equal
    z = torch.zeros(1, E, device="cuda")
    z[0, ::2] = -0.0
    z[0, 10:] = -1.0
    idx, _ = route(z, None, 6, score=score)
    assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]
    # a bias far above the scores swallows their low bits in fp32, not in the definition
    bias[:] = 1000.0
    y = x[3:].repeat(1, 1)
    y[0, 1::2] = y[0, ::2]
    y[0, 1::2] = torch.nextafter(y[0, 1::2], torch.full((32,), 9.0, device="cuda"))
    idx, w = route(y, bias, 8, score=score)
    ri, rw = route_ref(y, bias, 8, score=score)
    assert torch.equal(idx, ri)
    assert_weights(w, rw)


@pytest.mark.parametrize("kw", [{}, {"score": "sigmoid"}, {"n_group": 4, "topk_group": 2, "group_top": 2}])
def test_route_masks(kw):
    """-inf logits and biases, rows that leave nothing, fewer experts left than choices, the types' lowest values."""
    E = 32
    x = torch.randn(7, E, generator=gen(5), device="cuda")
    x[0] = -INF
    x[1, 1:] = -INF
    x[2, :30] = -INF
    x[3] = torch.finfo(torch.float32).min
    x[4, ::2] = torch.finfo(torch.float32).min
    x[5] = -200.0                                    # sigmoid: scores of 1e-87, whose quotients are weights all the same
    bias = torch.zeros(E, device="cuda")
    bias[3] = bias[9] = -INF
    for b in (None, bias):
        idx, w = route(x, b, 4, **kw)
        ri, rw = route_ref(x, b, 4, **kw)
        assert torch.equal(idx, ri)
        assert torch.equal(idx[0], torch.full((4,), -1, dtype=torch.int32, device="cuda")) and not w[0].any()
        assert_weights(w, rw)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.parametrize("value", [NAN, INF])
def test_route_nonfinite(value):
    x = torch.randn(5, 40, generator=gen(6), device="cuda")
    good = route(x, None, 4)
    y = x.clone()
    y[2, 33] = value
    idx, w = route(y, None, 4)
    assert q.qg_device_status() == q.QG_ERR_NONFINITE
    assert (idx[2] == -1).all() and not w[2].any()
    keep = [0, 1, 3, 4]
    assert torch.equal(idx[keep], good[0][keep]) and torch.equal(w[keep], good[1][keep])
    bias = torch.zeros(40, device="cuda")
    bias[7] = value
    idx, _ = route(x, bias, 4)
    assert q.qg_device_status() == q.QG_ERR_NONFINITE and (idx == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_large_batch_matches_64_bits(dtype):
    """20000 tokens in the grouped form against a 64-bit sort: every choice equal."""
    M, E, k = 20000, 256, 8
    x = (torch.randn(M, E, generator=gen(8), device="cuda") * 2).to(dtype)
    bias = torch.randn(E, generator=gen(9), device="cuda") * 0.1
    idx, w = route(x, bias, k, score="sigmoid", n_group=8, topk_group=4, group_top=2)
    s = torch.sigmoid(x.double())
    key = s + bias.double()
    val = key.view(M, 8, 32).topk(2, dim=2).values.sum(2)
    kept = torch.zeros(M, 8, dtype=torch.bool, device="cuda").scatter(
        1, val.sort(dim=1, descending=True, stable=True).indices[:, :4], True)
    key = key.masked_fill(~kept.repeat_interleave(32, 1), -INF)
    ri = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx.long(), ri)
    rw = s.gather(1, ri)
    assert_weights(w, rw / rw.sum(1, keepdim=True))


# ----------------------------------------------------------------------------- slot maps
def slots(idx, E):
    M, k = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    off, st, ts = torch.full((E + 1,), -9, **i32), torch.full((M * k,), -9, **i32), torch.full((M, k), -9, **i32)
    q.qg_expert_slots(idx, off, st, ts)
    return off, st, ts


def slots_ref(idx, E):
    flat = [(e, i) for i, e in enumerate(idx.flatten().tolist()) if 0 <= e < E]
    flat.sort()
    k = idx.shape[1]
    off = [sum(e < b for e, _ in flat) for b in range(E + 1)] if len(flat) < 5000 else None
    if off is None:
        cnt = [0] * (E + 1)
        for e, _ in flat:
            cnt[e + 1] += 1
        off = torch.tensor(cnt).cumsum(0).tolist()
    st = [i // k for _, i in flat] + [-1] * (idx.numel() - len(flat))
    ts = [-1] * idx.numel()
    for s, (_, i) in enumerate(flat):
        ts[i] = s
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    return t(off), t(st), t(ts).view(idx.shape)


@pytest.mark.parametrize("M,k,E", [(1, 1, 1), (1, 8, 64), (16, 8, 64), (127, 8, 8), (128, 8, 512), (129, 8, 256),
                                   (1000, 3, 17), (5000, 4, 512), (16384, 8, 256), (3000, 1, 2)])
def test_slots(M, k, E):
    idx = torch.randint(-1, E, (M, k), generator=gen(M + k), device="cuda", dtype=torch.int32)   # some -1, some repeats
    got = slots(idx, E)
    assert q.qg_device_status() == q.QG_OK
    for a, b in zip(got, slots_ref(idx, E)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [5, 3000])
def test_slots_all_on_one_none_and_bad_entries(M):
    for v in (0, 6, -1):
        idx = torch.full((M, 2), v, dtype=torch.int32, device="cuda")
        for a, b in zip(slots(idx, 7), slots_ref(idx, 7)):
            assert torch.equal(a, b)
    assert q.qg_device_status() == q.QG_OK
    idx = torch.randint(0, 7, (M, 2), generator=gen(2), device="cuda", dtype=torch.int32)
    idx[1, 0], idx[M - 1, 1], idx[2, 1] = 7, -2, -(1 << 31)
    for a, b in zip(slots(idx, 7), slots_ref(idx, 7)):
        assert torch.equal(a, b)
    assert q.qg_device_status() == q.QG_ERR_RANGE


def test_slots_of_no_tokens():
    off, st, ts = slots(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert not off.any() and st.numel() == 0 and ts.numel() == 0


# ------------------------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,k,N", [(1, 1, 8), (1, 8, 4096), (16, 8, 4096), (33, 3, 1032), (300, 2, 8192), (7, 32, 264)])
def test_combine(M, k, N, dtype):
    g = gen(M + N)
    S = M * k + 5
    D = torch.randn(S, N, generator=g, device="cuda").to(dtype)
    ts = torch.randint(-1, S, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(M, k, generator=g, device="cuda")
    ts[0] = -1                                       # a token of no expert
    D[ts.max() if M == 1 else 0] = NAN               # and a row that no choice names
    if M > 1:
        ts[ts == 0] = 1
    w[ts < 0] = NAN                                  # weights that are not read into the sum
    Y = torch.full((M, N), NAN, dtype=dtype, device="cuda")
    q.qg_combine_experts(D, ts, w, Y)
    assert q.qg_device_status() == q.QG_OK
    there = (ts >= 0)[..., None]
    terms = torch.where(there, D[ts.clamp(min=0).long()].double() * w[..., None].double(), 0.0)
    y, a = terms.sum(1), terms.abs().sum(1)
    # k fused multiply-adds in fp32 (one rounding each), then one rounding to the type
    tol = torch.finfo(dtype).eps / 2 * y.abs() + a * k * 2.0 ** -24 * 1.01 + 2.0 ** -25
    assert ((Y.double() - y).abs() <= tol).all()
    assert not Y[0].any()


def test_combine_bad_slots():
    D = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    ts = torch.tensor([[0, 4], [-2, 3], [1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    Y = torch.empty(3, 16, dtype=torch.bfloat16, device="cuda")
    q.qg_combine_experts(D, ts, torch.full((3, 2), 0.5, device="cuda"), Y)
    assert q.qg_device_status() == q.QG_ERR_RANGE
    assert torch.equal(Y[:, 0].float(), torch.tensor([0.5, 0.5, 0.0], device="cuda"))


def test_combine_past_32_bits():
    """More than 2^31 elements of slots: the last rows lie behind them."""
    S, N = 270000, 8192
    D = torch.zeros(S, N, dtype=torch.bfloat16, device="cuda")
    D[-2:] = torch.randn(2, N, generator=gen(1), device="cuda").to(torch.bfloat16)
    ts = torch.tensor([[S - 1, S - 2], [S - 2, -1]], dtype=torch.int32, device="cuda")
    Y = torch.empty(2, N, dtype=torch.bfloat16, device="cuda")
    q.qg_combine_experts(D, ts, torch.ones(2, 2, device="cuda"), Y)
    assert torch.equal(Y[0], (D[-1].float() + D[-2].float()).to(torch.bfloat16)) and torch.equal(Y[1], D[-2])


# ------------------------------------------------------------------------- a run of them
def test_padded_tokens_go_nowhere():
    """Tokens whose logits are -inf, and one that leaves two experts of four choices, through the whole layer."""
    M, E, k, K, N = 20, 6, 4, 256, 128
    g = gen(4)
    X = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    X[15:] = NAN                                     # padding holds anything
    logits = torch.randn(M, E, generator=g, device="cuda")
    logits[15:] = -INF
    logits[3, 2:] = -INF
    Wq = torch.randint(-3, 4, (E, K, N), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    ws = torch.ones(E, 2, 1, device="cuda")
    Xq, xs = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, 2, device="cuda")
    idx, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    off, st = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(M * k, dtype=torch.int32, device="cuda")
    ts, D = torch.empty_like(idx), torch.full((M * k, N), NAN, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    q.qg_quantize_act_fp8(X, Xq, xs)
    assert q.qg_device_status() == q.QG_ERR_NONFINITE   # the padding
    q.qg_route_topk(logits, None, idx, w)
    q.qg_expert_slots(idx, off, st, ts)
    q.qg_gemm_fp8_experts(Xq, xs, st, off, Wq, ws, D)
    q.qg_combine_experts(D, ts, w, Y)
    assert q.qg_device_status() == q.QG_OK
    used = 15 * k - 2
    assert int(off[-1]) == used and (st[used:] == -1).all() and (st[:used] >= 0).all()
    assert torch.isnan(D[used:]).all() and not torch.isnan(D[:used]).any()
    assert (ts[15:] == -1).all() and (ts[3, 2:] == -1).all()
    assert not Y[15:].any() and not torch.isnan(Y).any()
    y = torch.zeros(15, N, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for m in range(15):
        x = Xq[m].double() * xs[m].double().repeat_interleave(128)
        for e, v in zip(idx[m].tolist(), w[m].double().tolist()):
            if e >= 0:
                y[m] += v * (x @ Wq[e].double())
                size[m] += v * (x.abs() @ Wq[e].double().abs())
    # two roundings to bf16, 2^-8 each, and fp32 sums of 256 products: 2^-24 each
    assert ((Y[:15].double() - y).abs() <= (2.0 ** -7 + 2.0 ** -15) * size).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,E,k,K,N", [(1, 16, 4, 512, 272), (50, 8, 2, 400, 528), (700, 16, 4, 512, 512)])
def test_mixture_of_experts_layer(M, E, k, K, N, captured):
    """Quantize, route, map, multiply, combine, as a served layer does, eagerly and replayed from a graph with new inputs."""
    g = gen(M)
    W = torch.randn(E, K, N, generator=g, device="cuda") * 0.05
    Wq, ws = torch.empty(E, K, N, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(E, -(-K // 128), -(-N // 128), device="cuda")
    q.qg_quantize_weight_fp8(W, Wq, ws)
    Wr = torch.randn(K, E, generator=g, device="cuda") * 0.05
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(M, E, device="cuda")
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    kept = {}

    def layer():
        Xq, xs = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, -(-K // 128), device="cuda")
        idx, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
        off, st = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(M * k, dtype=torch.int32, device="cuda")
        ts, D = torch.empty_like(idx), torch.empty(M * k, N, dtype=torch.bfloat16, device="cuda")
        q.qg_quantize_act_fp8(X, Xq, xs)
        q.qg_route_topk(logits, None, idx, w)
        q.qg_expert_slots(idx, off, st, ts)
        q.qg_gemm_fp8_experts(Xq, xs, st, off, Wq, ws, D)
        q.qg_combine_experts(D, ts, w, out)
        kept.update(Xq=Xq, xs=xs, idx=idx, w=w)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()
    Wv = Wq.double() * ws.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 2)[..., :N]
    for turn in range(3):
        X.copy_(torch.randn(M, K, generator=g, device="cuda"))
        logits.copy_(X.float() @ Wr)
        out.fill_(NAN)
        if captured:
            graph.replay()
        else:
            layer()
        assert q.qg_device_status() == q.QG_OK
        x = kept["Xq"].double() * kept["xs"].double().repeat_interleave(128, 1)[:, :K]
        y, a = torch.zeros(M, N, dtype=torch.float64, device="cuda"), torch.zeros(M, N, dtype=torch.float64, device="cuda")
        ri, rw = route_ref(logits, None, k)
        assert torch.equal(kept["idx"], ri)
        for j in range(k):
            for e in range(E):
                m = ri[:, j] == e
                d = x[m] @ Wv[e]
                y[m] += rw[m, j:j + 1] * d
                a[m] += rw[m, j:j + 1] * (x[m].abs() @ Wv[e].abs())
        # each product: its own fp32 sums and one rounding to bf16; the weights 16 half steps; k more fp32 roundings; one to bf16
        tol = 2.0 ** -8 * (1 + 2.0 ** -8) * y.abs() + a * (2.0 ** -8 + 128 * 2.0 ** -23 + (K // 128 + 20 + k) * 2.0 ** -24) * 1.01
        assert ((out.double() - y).abs() <= tol).all(), turn
