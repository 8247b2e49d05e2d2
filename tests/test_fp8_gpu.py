"""The FP8 layer on the GPU: quantizers bit for bit, the product and the experts' product against 64 bits."""
import math

import pytest
import torch

import bit_quantized_gemm_group_b200 as q

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
NAN = float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ quantizers: bit for bit
def e4m3(v):
    """fp32 -> the nearest e4m3 value (ties to even), by arithmetic in 64 bits."""
    v = v.double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def scale_of(amax):
    """fp32(amax / 448): a quotient of fp32 numbers in 64 bits, rounded, is the fp32 quotient (53 >= 2 * 24 + 2)."""
    return (amax.double() / 448.0).float()


def codes_of(x, s):
    """Values of the codes of x under scales s (same shape)."""
    quot = (x.double() / torch.where(s > 0, s, 1.0).double()).float()
    return torch.where(s > 0, e4m3(quot), 0.0)


def quantize_act_ref(X):
    M, K = X.shape
    s = torch.stack([scale_of(X[:, k:k + 128].float().abs().amax(1)) for k in range(0, K, 128)], 1)
    return codes_of(X.float(), s.repeat_interleave(128, 1)[:, :K]), s


def quantize_weight_ref(W):
    K, N = W.shape
    s = torch.stack([torch.stack([scale_of(W[k:k + 128, n:n + 128].float().abs().amax()) for n in range(0, N, 128)])
                     for k in range(0, K, 128)])
    return codes_of(W.float(), s.repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]), s


def quantize_act(X):
    M, K = X.shape
    Xq = torch.full((M, K), 0x7F, dtype=torch.uint8, device="cuda").view(F8)
    xs = torch.full((M, cdiv(K, 128)), NAN, device="cuda")
    q.qg_quantize_act_fp8(X, Xq, xs)
    return Xq, xs


def quantize_weight(W):
    Wq = torch.full(W.shape, 0x7F, dtype=torch.uint8, device="cuda").view(F8)
    ws = torch.full((*W.shape[:-2], cdiv(W.shape[-2], 128), cdiv(W.shape[-1], 128)), NAN, device="cuda")
    q.qg_quantize_weight_fp8(W, Wq, ws)
    return Wq, ws


def activations(M, K, dtype, seed):
    x = torch.randn(M, K, generator=gen(seed), device="cuda")
    x[:, :: max(1, K // 8)] *= 50.0
    x[0, :min(K, 128)] = 0.0                       # a zero group
    if M > 1:
        x[1] *= 2.0 ** -13                         # small (fp16: subnormal) values
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (2, 4096), (37, 1040), (128, 11008), (5, 28672)])
def test_quantize_act(M, K, dtype):
    X = activations(M, K, dtype, M + K)
    Xq, xs = quantize_act(X)
    assert q.qg_device_status() == q.QG_OK
    c, s = quantize_act_ref(X)
    assert torch.equal(xs, s)
    assert torch.equal(Xq.double(), c)


def test_quantize_act_extremes():
    """The largest and smallest magnitudes of bf16: a scale that is subnormal or 0, one that is near fp32's largest."""
    X = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    X[0, 3], X[0, 200] = 3.0e38, -1.0
    X[1, :128] = torch.linspace(-1, 1, 128, device="cuda") * 2.0 ** -120
    X[1, 130] = 2.0 ** -133                        # bf16's smallest subnormal: the scale rounds to 2^-142 or so
    X[2, :] = 2.0 ** -133
    X[3, 5], X[3, 6] = -0.0, 448.0
    Xq, xs = quantize_act(X)
    c, s = quantize_act_ref(X)
    assert torch.equal(xs, s) and torch.equal(Xq.double(), c)
    assert q.qg_device_status() == q.QG_OK


def test_quantize_act_every_quotient():
    """Every positive bf16 significand against scales of many significands: the codes' ties and their neighbours."""
    top = (torch.arange(128, 256, device="cuda") / 128.0)          # all bf16 significands
    X = torch.zeros(128, 8, 128, device="cuda")
    for i, shift in enumerate((0, -1, -2, -3, -5, -8, -9, -11)):
        X[:, i, :] = top[None, :] * 2.0 ** shift
    X[:, :, 0] = top[:, None] * 2.0                                # the group's largest
    X = X.view(128, 1024).to(torch.bfloat16)
    Xq, xs = quantize_act(X)
    c, s = quantize_act_ref(X)
    assert torch.equal(xs, s) and torch.equal(Xq.double(), c)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_act_nonfinite(value, dtype):
    X = activations(3, 400, dtype, 1)
    X[1, 130] = value
    Xq, xs = quantize_act(X)
    assert q.qg_device_status() == q.QG_ERR_NONFINITE and q.qg_device_status() == q.QG_OK
    X[1, 130] = 0
    c, s = quantize_act_ref(X)
    good = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    good[1, 1] = False
    assert torch.equal(xs[good], s[good]) and torch.isnan(xs[1, 1])
    c[1, 128:256] = 0.0
    assert torch.equal(Xq.double(), c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (144, 272), (1024, 1024), (400, 4112)])
def test_quantize_weight(K, N, dtype):
    W = (torch.randn(K, N, generator=gen(K + N), device="cuda") * 0.02)
    if K > 128:
        W[128:256, :128] = 0.0
    W = W.to(dtype)
    Wq, ws = quantize_weight(W)
    assert q.qg_device_status() == q.QG_OK
    c, s = quantize_weight_ref(W)
    assert torch.equal(ws, s) and torch.equal(Wq.double(), c)


def test_quantize_weight_experts_and_nonfinite():
    W = torch.randn(3, 272, 160, generator=gen(3), device="cuda")
    W[1, 200, 150] = NAN
    W[2, 0, 0] = -float("inf")
    Wq, ws = quantize_weight(W)
    assert q.qg_device_status() == q.QG_ERR_NONFINITE
    for e in range(3):
        c, s = quantize_weight_ref(W[e].nan_to_num(0.0, 0.0, 0.0))
        if e == 1:
            c[128:256, 128:], s[1, 1] = 0.0, NAN
        if e == 2:
            c[:128, :128], s[0, 0] = 0.0, NAN
        assert torch.equal(ws[e].nan_to_num(-1.0), s.nan_to_num(-1.0)) and torch.equal(Wq[e].double(), c)


def test_quantize_act_past_32_bits():
    """More than 2^31 elements: the last rows' offsets do not fit 32 bits."""
    M, K = 75000, 28672
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[-3:] = activations(3, K, torch.bfloat16, 9)
    Xq, xs = quantize_act(X)
    c, s = quantize_act_ref(X[-3:])
    assert torch.equal(xs[-3:], s) and torch.equal(Xq[-3:].double(), c)
    assert not xs[:-3].any() and not Xq[:70000:1111].view(torch.uint8).any()


# --------------------------------------------------------------------------------- product
def values(Xq, xs, Wq, ws):
    K, N = Wq.shape
    x = Xq.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    w = Wq.double() * ws.double().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    return x, w


def assert_product(Y, x, w):
    """Y against x w in 64 bits.

    e4m3 products are exact in fp32 (two 4-bit significands).  Adding 128 of them one by one, each sum cut
    rather than rounded, is off by at most 128 * 2^-23 of the group's sum of magnitudes; the scales' product, its
    product with the group and the G sums over the groups by 2^-24 each, so (G + 2) * 2^-24 of the whole; the
    result is rounded once to its type, half a step."""
    K = x.shape[1]
    y = x @ w
    a = x.abs() @ w.abs()
    tol = torch.finfo(Y.dtype).eps / 2 * y.abs() + a * (128 * 2.0 ** -23 + (cdiv(K, 128) + 2) * 2.0 ** -24) * 1.01
    tol = tol + 2.0 ** -25                          # fp16: half its smallest step
    off = (Y.double() - y).abs()
    assert not torch.isnan(Y).any()
    worst = (off - tol).argmax()
    assert (off <= tol).all(), f"off by {off.flatten()[worst]:.3e}, allowed {tol.flatten()[worst]:.3e} at {int(worst)}"


def product(Xq, xs, Wq, ws, dtype=torch.bfloat16, **kw):
    Y = torch.full((Xq.shape[0], Wq.shape[1]), NAN, dtype=dtype, device="cuda")
    q.qg_gemm_fp8(Xq, xs, Wq, ws, Y, **kw)
    return Y


def operands(M, K, N, seed):
    Xq, xs = quantize_act(activations(M, K, torch.bfloat16, seed))
    Wq, ws = quantize_weight(torch.randn(K, N, generator=gen(seed + 1), device="cuda") * 0.02)
    return Xq, xs, Wq, ws


def exact_operands(M, K, N, seed):
    """Small whole codes and scales that are powers of two: every sum is exact in fp32."""
    g = gen(seed)
    Xq = torch.randint(-3, 4, (M, K), generator=g, device="cuda").float().to(F8)
    Wq = torch.randint(-3, 4, (K, N), generator=g, device="cuda").float().to(F8)
    xs = torch.exp2(torch.randint(-2, 3, (M, cdiv(K, 128)), generator=g, device="cuda").float())
    ws = torch.exp2(torch.randint(-2, 3, (cdiv(K, 128), cdiv(N, 128)), generator=g, device="cuda").float())
    return Xq, xs, Wq, ws


MS = [1, 2, 8, 9, 15, 16, 17, 31, 33, 64, 65, 96, 127, 128, 129, 200, 257, 333, 513]


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (400, 272), (1024, 1040)])
def test_gemm_exact(M, K, N):
    o = exact_operands(M, K, N, M + K + N)
    Y = product(*o)
    assert q.qg_device_status() == q.QG_OK
    x, w = values(*o)
    assert torch.equal(Y, (x @ w).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 12288), (4, 11008, 4096), (16, 4096, 4096), (33, 4096, 4112),
                                   (64, 8192, 8192), (100, 4112, 4096), (130, 4096, 22016), (333, 11008, 4144),
                                   (700, 1040, 1024), (2048, 4096, 11008)])
def test_gemm(M, K, N, dtype):
    o = operands(M, K, N, M)
    Y = product(*o, dtype=dtype)
    assert q.qg_device_status() == q.QG_OK
    assert_product(Y, *values(*o))
    again = product(*o, dtype=dtype)
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))   # the same bits every time


@pytest.mark.parametrize("M", [1, 20, 300])
def test_gemm_nan_stays_in_its_row_and_column(M):
    Xq, xs, Wq, ws = operands(M, 400, 272, 5)
    Xq.view(torch.uint8)[M // 2, 130] = 0x7F       # a NaN code
    ws[2, 1] = NAN                                 # columns 128..255
    Y = product(Xq, xs, Wq, ws)
    bad = torch.zeros_like(Y, dtype=torch.bool)
    bad[M // 2], bad[:, 128:256] = True, True
    assert torch.equal(torch.isnan(Y), bad)


def test_gemm_any_scales():
    """Scales that no quantizer gives: negative, zero, large."""
    Xq, xs, Wq, ws = operands(40, 384, 256, 6)
    xs[:, 1] = 0.0
    xs[3] *= -1.0
    ws[0] *= 1e10
    assert_product(product(Xq, xs, Wq, ws), *values(Xq, xs, Wq, ws))


# long K, where tiles are split and joined: one piece's worth to all of a tile's rows, both tile
# widths (the last two), and whole waves of tiles before the split ones (the last)
SPLIT = [(1, 11008, 4096), (5, 8320, 16), (17, 11008, 400), (64, 12304, 1040), (128, 28672, 128), (130, 12800, 272),
         (3, 16384, 20480), (2, 6144, 38416)]


@pytest.mark.parametrize("M,K,N", SPLIT)
def test_gemm_split_exact(M, K, N):
    o = exact_operands(M, K, N, M + N)
    x, w = values(*o)
    want = (x @ w).to(torch.bfloat16)
    for _ in range(3):
        assert torch.equal(product(*o), want)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.parametrize("M,K,N", [(1, 11008, 4096), (64, 12304, 1040)])
def test_gemm_split_rounds_once_and_the_same_every_time(M, K, N):
    o = operands(M, K, N, 3)
    Y = product(*o, dtype=torch.float16)
    assert_product(Y, *values(*o))
    for _ in range(20):
        assert torch.equal(product(*o, dtype=torch.float16).view(torch.int16), Y.view(torch.int16))


def test_gemm_workspace_contents_do_not_matter():
    for M, K, N in ((1, 11008, 4096), (33, 8192, 272), (100, 28672, 128)):
        o = operands(M, K, N, 7)
        want = product(*o)
        need = q.qg_workspace_size(q.QG_OP_GEMM_FP8, M, K, N)
        assert need > 0
        for fill in (0, 0xFF, 0x5A):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            for _ in range(2):
                assert torch.equal(product(*o, workspace=ws).view(torch.int16), want.view(torch.int16))


def test_gemm_on_another_stream_and_two_graphs():
    """Two captured graphs replayed in turn and at once, and an eager call on a stream of its own."""
    sets = [operands(M, 11008, 528, 20 + M) for M in (3, 40)]   # tiles of both are split
    want = [product(*o) for o in sets]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in sets:
        Y = torch.full((o[0].shape[0], 528), NAN, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.qg_gemm_fp8(*o, Y)
            q.qg_gemm_fp8(*o, Y)
        graphs.append(g)
        outs.append(Y)
    for turn in range(6):
        for Y in outs:
            Y.fill_(NAN)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        Y3 = torch.full_like(outs[0], NAN)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        q.qg_gemm_fp8(*sets[0], Y3, stream=side)
        torch.cuda.synchronize()
        for Y, w in zip((*outs, Y3), (*want, want[0])):
            assert torch.equal(Y.view(torch.int16), w.view(torch.int16)), turn


# -------------------------------------------------------------------------------- experts
def experts(Xq, xs, tok, off, Wq, ws, S, dtype=torch.bfloat16, **kw):
    Y = torch.full((S, Wq.shape[2]), NAN, dtype=dtype, device="cuda")
    q.qg_gemm_fp8_experts(Xq, xs, tok, off, Wq, ws, Y, **kw)
    return Y


def expert_operands(M, E, K, N, counts, seed, exact=False):
    g = gen(seed)
    if exact:
        Xq, xs = exact_operands(M, K, 16, seed)[:2]
        w = [exact_operands(1, K, N, seed + e)[2:] for e in range(E)]
        Wq, ws = torch.stack([t[0].view(torch.uint8) for t in w]).view(F8), torch.stack([t[1] for t in w])
    else:
        Xq, xs = quantize_act(activations(M, K, torch.bfloat16, seed))
        Wq, ws = quantize_weight(torch.randn(E, K, N, generator=g, device="cuda") * 0.02)
    off = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    tok = torch.randint(0, M, (sum(counts),), generator=g, device="cuda", dtype=torch.int32)   # some tokens twice
    return Xq, xs, tok, off, Wq, ws


COUNTS = {
    "one slot": [0, 1, 0],
    "all on one": [0, 0, 300, 0],
    "none": [0, 0, 0],
    "few": [1, 2, 0, 3, 1, 1, 0, 2],
    "ragged": [5, 0, 17, 16, 33, 1, 64, 65],
    "tiles": [128, 0, 129, 127, 1, 256, 300],
    "even": [40] * 12,
    "many": [3] * 100,
    "large": [700, 0, 513, 300],
    "512 experts": [0] * 200 + [2, 0, 130] + [0] * 308 + [1],
}


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("K,N", [(16, 16), (400, 272), (1024, 528)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_experts_exact(name, K, N, gather):
    counts = COUNTS[name]
    E, S = len(counts), sum(counts)
    Xq, xs, tok, off, Wq, ws = expert_operands(S + 3 if not gather else 70, E, K, N, counts, 3, exact=True)
    spare = 5                                       # slots behind the last one in use
    tokens = torch.cat([tok, torch.full((spare,), -1, dtype=torch.int32, device="cuda")]) if gather else None
    if not gather:
        Xq, xs = torch.cat([Xq.view(torch.uint8)] * 2)[:S + spare].contiguous().view(F8), torch.cat([xs] * 2)[:S + spare]
    Y = experts(Xq, xs.contiguous(), tokens, off, Wq, ws, S + spare)
    assert q.qg_device_status() == q.QG_OK
    assert torch.isnan(Y[S:]).all()                 # left as they were
    at = off.tolist()
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        src = tok[rows].long() if gather else torch.arange(at[e], at[e + 1], device="cuda")
        x, w = values(Xq.view(torch.uint8)[src].view(F8), xs[src], Wq[e], ws[e])
        assert torch.equal(Y[rows], (x @ w).to(torch.bfloat16)), e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,E,K,N,counts", [(8, 32, 2048, 2064, [1] * 30 + [0, 2]), (100, 8, 4096, 1024, [7, 90, 0, 33, 1, 64, 5, 0]),
                                            (600, 6, 1040, 1552, [600, 0, 411, 129, 128, 60])])
def test_experts(M, E, K, N, counts, dtype):
    Xq, xs, tok, off, Wq, ws = expert_operands(M, E, K, N, counts, M)
    Y = experts(Xq, xs, tok, off, Wq, ws, sum(counts), dtype)
    again = experts(Xq, xs, tok, off, Wq, ws, sum(counts), dtype)
    assert q.qg_device_status() == q.QG_OK
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))
    at = off.tolist()
    for e in range(E):
        if counts[e]:
            src = tok[at[e]:at[e + 1]].long()
            assert_product(Y[at[e]:at[e + 1]], *values(Xq.view(torch.uint8)[src].view(F8), xs[src], Wq[e], ws[e]))


@pytest.mark.parametrize("counts", [[3, 2, 1], [200, 100, 150]])
def test_experts_bad_maps(counts):
    """A token outside X counts as zeros; offsets that do not ascend within the slots compute nothing."""
    Xq, xs, tok, off, Wq, ws = expert_operands(50, 3, 400, 272, counts, 8, exact=True)
    S = sum(counts)
    good = experts(Xq, xs, tok, off, Wq, ws, S)
    bad = tok.clone()
    bad[1], bad[S - 1] = 50, -7
    Y = experts(Xq, xs, bad, off, Wq, ws, S)
    assert q.qg_device_status() == q.QG_ERR_RANGE
    keep = torch.ones(S, dtype=torch.bool, device="cuda")
    keep[1] = keep[S - 1] = False
    assert torch.equal(Y[keep], good[keep]) and not Y[~keep].any()
    for wrong in ([0, 5, 4, S], [1, 2, 3, S], [0, 1, 2, S + 1], [-4, 1, 2, S], [0, 1 << 30, -(1 << 30), S]):
        Y = experts(Xq, xs, tok, torch.tensor(wrong, dtype=torch.int32, device="cuda"), Wq, ws, S)
        assert q.qg_device_status() == q.QG_ERR_RANGE and torch.isnan(Y).all()


@pytest.mark.parametrize("counts", [[1, 0, 2], [0, 70, 0, 3], [1] * 20, [9, 0, 0, 160]])
def test_experts_split_exact(counts):
    """Long K: the last experts' tiles are split along it."""
    Xq, xs, tok, off, Wq, ws = expert_operands(40, len(counts), 11008, 528, counts, 4, exact=True)
    want = torch.cat([(lambda x, w: (x @ w).to(torch.bfloat16))(*values(
        Xq.view(torch.uint8)[t].view(F8), xs[t], Wq[e], ws[e])) for e in range(len(counts))
        if (t := tok[off[e]:off[e + 1]].long()).numel()])
    need = q.qg_workspace_size(q.QG_OP_GEMM_FP8_EXPERTS, tok.numel(), 11008, 528)
    for fill in (0, 0xFF, 0x5A):
        ws8 = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(experts(Xq, xs, tok, off, Wq, ws, tok.numel(), workspace=ws8), want)
    assert q.qg_device_status() == q.QG_OK


def test_experts_two_graphs():
    sets = [expert_operands(16, 12, 8192, 1040, c, 30) for c in ([1, 0, 4] * 4, [40, 3, 0, 21] * 3)]
    want = [experts(*o, o[2].numel()) for o in sets]
    graphs, outs = [], []
    for o in sets:
        Y = torch.full((o[2].numel(), 1040), NAN, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.qg_gemm_fp8_experts(*o, Y)
        graphs.append(g)
        outs.append(Y)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for Y in outs:
            Y.fill_(NAN)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for Y, w in zip(outs, want):
            assert torch.equal(Y.view(torch.int16), w.view(torch.int16))


def test_gemm_outputs_past_32_bits():
    """More than 2^31 outputs."""
    M, K, N = 75008, 16, 28688
    o = exact_operands(M, K, N, 1)
    Y = product(*o)
    for rows in (slice(0, 3), slice(M - 3, M), slice(M // 2, M // 2 + 3)):
        x, w = values(o[0][rows], o[1][rows], *o[2:])
        assert torch.equal(Y[rows], (x @ w).to(torch.bfloat16))


def test_experts_weights_past_32_bits():
    """More than 2^31 weights: the last expert's lie behind them."""
    E, K, N = 9, 16384, 16400
    Xq, xs, Wl, wsl = exact_operands(5, K, N, 2)
    Wq = torch.zeros(E, K, N, dtype=torch.uint8, device="cuda")
    Wq[-1] = Wl.view(torch.uint8)
    ws = torch.ones(E, cdiv(K, 128), cdiv(N, 128), device="cuda")
    ws[-1] = wsl
    off = torch.tensor([0] + [2] * (E - 1) + [5], dtype=torch.int32, device="cuda")
    Y = experts(Xq, xs, None, off, Wq.view(F8), ws, 5)
    x, w = values(Xq, xs, Wl, wsl)
    assert not Y[:2].any() and torch.equal(Y[2:], (x @ w)[2:].to(torch.bfloat16))


def test_empty():
    o = operands(3, 256, 128, 4)
    assert product(o[0][:0], o[1][:0], *o[2:]).shape == (0, 128)
    Xq, xs = quantize_act(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert Xq.shape == (0, 256) and math.prod(xs.shape) == 0
