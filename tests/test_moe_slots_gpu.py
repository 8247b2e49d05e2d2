"""Slot maps of many blocks of choices, around and past the number where their counts are summed up once for all."""
import pytest
import torch

import bit_quantized_gemm_group_b200 as q

pytestmark = pytest.mark.gpu
BLOCK = 4096


def maps(idx, E, **kw):
    M, k = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full((E + 1,), -9, **i32), torch.full((M * k,), -9, **i32), torch.full((M, k), -9, **i32)
    q.qg_expert_slots(idx, *out, **kw)
    return out


def maps_ref(idx, E):
    """A stable sort of the choices; what is no expert comes last and has no slot."""
    M, k = idx.shape
    flat = idx.flatten()
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order = flat.sort(stable=True)
    off = torch.searchsorted(order.values, torch.arange(E + 1, dtype=torch.int32, device="cuda"))
    token = torch.where(order.values < E, order.indices // k, -1)
    slot = torch.empty(M * k, dtype=torch.int32, device="cuda")
    slot[order.indices] = torch.arange(M * k, dtype=torch.int32, device="cuda")
    return off.int(), token.int(), torch.where(flat < E, slot, -1).view(M, k)


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def choices(n, k, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, E, (n // k, k), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("E", [1, 31, 33, 256, 512])
@pytest.mark.parametrize("n", [31 * BLOCK, 32 * BLOCK, 32 * BLOCK + 1, 33 * BLOCK, 39 * BLOCK + 77, 64 * BLOCK, 65 * BLOCK + 1,
                               300 * BLOCK - 1])
def test_around_the_rule(n, E):
    idx = choices(n, 1, E, n + E)
    same(maps(idx, E), maps_ref(idx, E))
    assert q.qg_device_status() == q.QG_OK


@pytest.mark.parametrize("fill", ["one", "none", "rising", "falling"])
def test_uneven(fill):
    n, E = 100 * BLOCK, 64
    at = torch.arange(n, device="cuda") * E // n     # whole blocks of one expert
    idx = {"one": torch.full_like(at, 7), "none": torch.full_like(at, -1), "rising": at, "falling": E - 1 - at}[fill]
    idx = idx.int().view(-1, 4)
    same(maps(idx, E), maps_ref(idx, E))
    assert q.qg_device_status() == q.QG_OK


def test_entries_that_are_no_expert():
    idx = choices(50 * BLOCK, 8, 40, 3)
    idx[0, 0], idx[-1, -1], idx[3000, 2] = 40, -2, -(1 << 31)
    same(maps(idx, 40), maps_ref(idx, 40))
    assert q.qg_device_status() == q.QG_ERR_RANGE


def test_workspace_of_the_stated_size_and_replays():
    M, k, E = 40000, 8, 300
    idx = choices(M * k, k, E, 4)
    need = q.qg_workspace_size(q.QG_OP_EXPERT_SLOTS, M, k, E)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    same(maps(idx, E, workspace=ws[:need]), maps_ref(idx, E))
    assert (ws[need:] == 0x5A).all()                 # and not a byte more
    out = tuple(torch.empty_like(t) for t in maps_ref(idx, E))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qg_expert_slots(idx, *out)
    for seed in range(5, 8):
        idx.copy_(choices(M * k, k, E, seed))
        graph.replay()
        same(out, maps_ref(idx, E))


def test_sixteen_million_tokens():
    """2^27 choices: 32768 blocks."""
    idx = choices(1 << 27, 8, 512, 9)
    got = maps(idx, 512)
    assert q.qg_device_status() == q.QG_OK
    same(got, maps_ref(idx, 512))


def test_time_grows_with_the_choices_and_not_with_their_square():
    """Eight times the choices (512 blocks, 4096): eight times the work, and at most sixteen times as long."""
    took = []
    for blocks in (512, 4096):
        idx = choices(blocks * BLOCK, 8, 256, 10)
        out = maps(idx, 256)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            q.qg_expert_slots(idx, *out)
        end.record()
        torch.cuda.synchronize()
        took.append(start.elapsed_time(end))
    assert took[1] < 16 * took[0], took
