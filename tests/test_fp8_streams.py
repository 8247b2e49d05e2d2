"""Scratch and order of the FP8 layer's and the experts' calls on several streams."""
import contextlib

import pytest
import torch

import bit_quantized_gemm_group_b200 as q

F8 = torch.float8_e4m3fn


# --------------------------------------------------- which pool scratch comes from (CPU, with a fake library)
class FakeStream:
    def __init__(self, name):
        self.cuda_stream = name


class FakeLib:
    """Notes each launch; every operator wants 512 bytes."""
    def __init__(self):
        self.launches = []

    def qg_workspace_size(self, *op):
        return 512

    def __getattr__(self, name):
        if not name.startswith("qg_"):
            raise AttributeError(name)
        return lambda *args: self.launches.append((name, args)) or q.QG_OK


@pytest.fixture
def fake(monkeypatch):
    """A library and streams without a GPU; `fake.allocated`: the stream that was current at each allocation."""
    lib, now = FakeLib(), [FakeStream("current")]
    lib.allocated = []

    @contextlib.contextmanager
    def enter(stream):
        now.append(stream)
        yield
        now.pop()

    class Scratch:
        def __init__(self, n):
            lib.allocated.append((now[-1].cuda_stream, n))
            self.n, self.dtype, self.shape = n, torch.uint8, (n,)

        def numel(self):
            return self.n

        def data_ptr(self):
            return 0x10000

        def get_device(self):
            return 0

        def is_contiguous(self):
            return True

        def record_stream(self, stream):
            pass

    monkeypatch.setattr(q, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: Scratch(n))
    return lib


@pytest.mark.parametrize("op", ["qg_gemm_fp8", "qg_gemm_fp8_experts", "qg_expert_slots"])
@pytest.mark.parametrize("stream", [None, FakeStream("side")])
def test_scratch_comes_from_the_pool_of_the_calls_stream(fake, op, stream):
    q._run(op, 0, stream, (1, 2, 3), (5, 4, 4096, 4096), "auto")
    on = "current" if stream is None else "side"
    assert fake.allocated == [(on, 512)]
    assert fake.launches == [(op, (1, 2, 3, 0x10000, 512, on))]


# ------------------------------------------------------------------------------------------- on the GPU
NAN = float("nan")


def operands(M, K, N, E, seed):
    """Small whole codes, scales that are powers of two: the same product in whatever order it is summed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float().to(F8)                # noqa: E731
    scale = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g, device="cuda").float())          # noqa: E731
    return code(M, K), scale(M, -(-K // 128)), code(E, K, N), scale(E, -(-K // 128), -(-N // 128))


def value(q8, s, wide):
    v = s.double().repeat_interleave(128, -1)
    if wide:
        v = v[..., :q8.shape[-1]].repeat_interleave(128, -2)
    return q8.double() * v[..., :q8.shape[-2], :q8.shape[-1]]


class Gemm:
    """Products whose tiles are split along K, so that their scratch holds counters and partial sums."""
    def __init__(self, M):
        self.Xq, self.xs, Wq, ws = operands(M, 11008, 528, 1, M)
        self.Wq, self.ws = Wq[0], ws[0]
        self.want = (value(self.Xq, self.xs, False) @ value(self.Wq, self.ws, True)).to(torch.bfloat16),
        self.got = torch.empty(M, 528, dtype=torch.bfloat16, device="cuda"),

    def call(self, **kw):
        q.qg_gemm_fp8(self.Xq, self.xs, self.Wq, self.ws, *self.got, **kw)


class Experts:
    """Experts' products: gathered rows and, at this K, split tiles."""
    def __init__(self, S):
        E, g = 3, torch.Generator(device="cuda").manual_seed(S)
        self.ops = operands(50, 11008, 272, E, S)
        self.token = torch.randint(0, 50, (S,), generator=g, device="cuda", dtype=torch.int32)
        cut = [0, S // 3, S // 3, S]
        self.off = torch.tensor(cut, dtype=torch.int32, device="cuda")
        x, w = value(*self.ops[:2], False)[self.token.long()], value(*self.ops[2:], True)
        self.want = torch.cat([x[a:b] @ w[e] for e, (a, b) in enumerate(zip(cut, cut[1:]))]).to(torch.bfloat16),
        self.got = torch.empty(S, 272, dtype=torch.bfloat16, device="cuda"),

    def call(self, **kw):
        Xq, xs, Wq, ws = self.ops
        q.qg_gemm_fp8_experts(Xq, xs, self.token, self.off, Wq, ws, *self.got, **kw)


class Slots:
    """Slot maps of several blocks, whose counts are in the scratch."""
    def __init__(self, M, E=64):
        g = torch.Generator(device="cuda").manual_seed(M)
        self.idx = torch.randint(0, E, (M, 8), generator=g, device="cuda", dtype=torch.int32)
        flat = self.idx.flatten().long()
        order = flat.sort(stable=True)
        slot = torch.empty_like(flat).scatter_(0, order.indices, torch.arange(8 * M, device="cuda"))
        off = torch.searchsorted(order.values, torch.arange(E + 1, device="cuda"))
        self.want = tuple(t.int() for t in (off, order.indices // 8, slot.view(M, 8)))
        self.got = tuple(torch.empty_like(t) for t in self.want)

    def call(self, **kw):
        q.qg_expert_slots(self.idx, *self.got, **kw)


def clear(*jobs):
    for j in jobs:
        for t in j.got:
            t.fill_(-9)
    torch.cuda.synchronize()


def check(turn, *jobs):
    torch.cuda.synchronize()
    for j in jobs:
        for got, want in zip(j.got, j.want):
            assert torch.equal(got, want), turn


PAIRS = [(Gemm, 128, 40), (Gemm, 3, 100), (Experts, 300, 90), (Slots, 30000, 28000)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,a,b", PAIRS)
def test_two_calls_at_once_share_no_scratch(kind, a, b):
    """One on the current stream, one at once on another, whose inputs are ready: neither waits for the other."""
    here, there, side = kind(a), kind(b), torch.cuda.Stream()
    for turn in range(30):
        clear(here, there)
        here.call()
        there.call(stream=side)
        check(turn, here, there)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind,a,b", PAIRS)
def test_call_beside_a_temporary_that_is_still_in_use(kind, a, b):
    """A block that the current stream freed while its kernels still write it is not the other stream's scratch."""
    job, side = kind(b), torch.cuda.Stream()
    ones = torch.ones(40 << 20, dtype=torch.uint8, device="cuda")
    for turn in range(10):
        clear(job)
        for _ in range(20):
            temporary = ones.clone()      # freed below with its copies still to come
            temporary.add_(1)
        del temporary
        job.call(stream=side)
        check(turn, job)
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind,a,b", PAIRS)
def test_captured_on_two_streams(kind, a, b):
    """A capture that forks to a second stream: replays beside an eager call of the same kind."""
    here, there, eager, side, third = kind(a), kind(b), kind(a), torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        here.call()
        there.call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for turn in range(10):
        clear(here, there, eager)
        graph.replay()
        eager.call(stream=third)
        check(turn, here, there, eager)
    assert q.qg_device_status() == q.QG_OK


# ------------------------------------------------- operands that the kernel right before has written (GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_weights_quantized_right_before(M, captured):
    """A served layer whose weight is updated: the weight quantizer is the last kernel before the product."""
    K, N = 2048, 1040
    Xq, xs = operands(M, K, N, 1, 5)[:2]
    W = torch.zeros(K, N, device="cuda")
    Wq, ws = torch.empty(K, N, dtype=F8, device="cuda"), torch.empty(K // 128, -(-N // 128), device="cuda")
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def update():
        q.qg_quantize_weight_fp8(W, Wq, ws)
        q.qg_gemm_fp8(Xq, xs, Wq, ws, Y)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            update()
    g = torch.Generator(device="cuda").manual_seed(M)
    for turn in range(20):
        # codes -448 and 448 under the scale 1 (and the powers of two beside it): every sum is exact
        W.copy_((torch.randint(0, 2, (K, N), generator=g, device="cuda").float() * 2 - 1) * 448 * 2.0 ** (turn % 3))
        Y.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay() if captured else update()
        want = value(Xq, xs, False) @ W.double()
        assert torch.equal(Y, want.to(torch.bfloat16)), turn
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_weights_written_by_a_kernel_that_lets_the_product_start_early(captured):
    """The bytes of one product's outputs are the next one's weights.  The first occupies some 32 SMs, so the second
    starts beside it."""
    K1, K2, N1 = 4096, 256, 2048
    one = torch.ones(1, device="cuda")
    eye = torch.eye(K2, K1, device="cuda").to(F8)             # Y1 = the first rows of the first weight
    s1, t1 = one.expand(K2, K1 // 128).contiguous(), one.expand(K1 // 128, N1 // 128).contiguous()
    X2, s2 = operands(7, K2, 16, 1, 6)[:2]
    t2 = one.expand(K2 // 128, 2 * N1 // 128).contiguous()
    W1 = torch.empty(K1, N1, dtype=F8, device="cuda")
    Y1 = torch.empty(K2, N1, dtype=torch.bfloat16, device="cuda")
    W2 = Y1.view(torch.uint8).view(F8)                        # of 1.0 and 2.0: the codes -0, 1.875, 0 and 2
    Y2 = torch.empty(7, 2 * N1, dtype=torch.bfloat16, device="cuda")

    def both():
        q.qg_gemm_fp8(eye, s1, W1, t1, Y1)
        q.qg_gemm_fp8(X2, s2, W2, t2, Y2)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
    g = torch.Generator(device="cuda").manual_seed(8)
    for turn in range(20):
        W1.copy_(torch.randint(1, 3, (K1, N1), generator=g, device="cuda").float())
        Y1.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else both()
        torch.cuda.synchronize()
        assert torch.equal(Y1.float(), W1[:K2].float())
        assert torch.equal(Y2, (value(X2, s2, False) @ W2.double()).to(torch.bfloat16)), turn
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,K,N", [(5, 1024, 528), (200, 1024, 528), (12, 11008, 272)])
def test_maps_written_right_before_in_buffers_that_are_still_being_read(M, K, N, captured):
    """Layer after layer with the same map buffers: each product starts beside the one before, which reads the old maps."""
    E, k, layers = 16, 4, 6
    Xq, xs, Wq, ws = operands(M, K, N, E, M)
    g = torch.Generator(device="cuda").manual_seed(M + 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx = [torch.zeros(M, k, **i32) for _ in range(layers)]
    off, token, slot = torch.empty(E + 1, **i32), torch.empty(M * k, **i32), torch.empty(M, k, **i32)
    Y = [torch.empty(M * k, N, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]

    def run():
        for i, y in zip(idx, Y):
            q.qg_expert_slots(i, off, token, slot)
            q.qg_gemm_fp8_experts(Xq, xs, token, off, Wq, ws, y)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    every = torch.einsum("mk,ekn->emn", value(Xq, xs, False), value(Wq, ws, True)).to(torch.bfloat16)
    for turn in range(8):
        for i, y in zip(idx, Y):
            i.copy_(torch.rand(M, E, generator=g, device="cuda").topk(k, 1).indices)
            y.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        for i, y in zip(idx, Y):
            order = i.flatten().long().sort(stable=True)
            assert torch.equal(y, every[order.values, order.indices // k]), turn
    assert q.qg_device_status() == q.QG_OK
