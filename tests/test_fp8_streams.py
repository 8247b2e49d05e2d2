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
