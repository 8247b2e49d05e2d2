"""The FP8 product's bounded waits run out: they give up, and a split tile's pieces are counted in all the same."""
import ctypes

import pytest
import torch

import bit_quantized_gemm_group_b200 as q

P = ctypes.c_void_p
A, B = P(0x10000), P(0x10008)   # never dereferenced: validation fails first


@pytest.mark.parametrize("args,want", [
    ((0, 4, A, A, None), 2), ((500001, 4, A, A, None), 2), ((10, 0, A, A, None), 2), ((10, 256, A, A, None), 2),
    ((10, 4, None, A, None), 1), ((10, 4, A, None, None), 1), ((10, 4, B, A, None), 3), ((10, 4, A, B, None), 3),
])
def test_refused(args, want):
    assert q.lib().qg_selftest_split_wait(*args) == want


def test_binding_refuses():
    c, r = torch.zeros(1, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)
    for polls, counter, result in ((10, c, r), (10, c, c), (10, c, r[:, None])):
        with pytest.raises(ValueError):
            q.qg_selftest_split_wait(polls, counter, result)


def outcome(result):
    """All waits gave up and one piece, whichever, was the last."""
    assert ((result & 1) == 1).all() and int((result & 2).sum()) == 2 and (result < 4).all()


@pytest.mark.gpu
@pytest.mark.parametrize("pieces", [1, 2, 5, 148, 255])
@pytest.mark.parametrize("fill", [0, -1, 0x5A5A5A5A5A5A5A5A, 3])
def test_wait_gives_up_and_its_piece_is_counted_in(pieces, fill):
    counter = torch.full((1,), fill, dtype=torch.int64, device="cuda")
    for _ in range(3):                               # the word that a launch leaves serves the next one
        result = torch.full((pieces,), -9, dtype=torch.int32, device="cuda")
        q.qg_selftest_split_wait(50, counter, result)
        assert q.qg_device_status() == q.QG_ERR_TIMEOUT and q.qg_device_status() == q.QG_OK
        outcome(result)
        assert int(counter) == 0


@pytest.mark.gpu
def test_replay_after_a_wait_that_gave_up_starts_from_a_cleared_counter():
    """A replayed launch has the token of the one before it."""
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    result = torch.full((19,), -9, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qg_selftest_split_wait(50, counter, result)
    for _ in range(4):
        result.fill_(-9)
        graph.replay()
        assert q.qg_device_status() == q.QG_ERR_TIMEOUT
        outcome(result)
        assert int(counter) == 0


@pytest.mark.gpu
def test_wait_ends_in_time_and_the_products_work_after_it():
    """The product's own limit is 500000 polls and is meant to be 2 s: a twentieth of it ends within a factor of two of
    100 ms."""
    counter, result = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qg_selftest_split_wait(1, counter, result)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    q.qg_selftest_split_wait(25000, counter, result)
    end.record()
    assert q.qg_device_status() == q.QG_ERR_TIMEOUT
    outcome(result)
    assert 50.0 < start.elapsed_time(end) < 200.0
    F8 = torch.float8_e4m3fn
    one = lambda *s: torch.ones(*s, device="cuda")   # noqa: E731
    Y = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    q.qg_gemm_fp8(one(3, 8192).to(F8), one(3, 64), one(8192, 256).to(F8), one(64, 2), Y)
    assert (Y == 8192).all() and q.qg_device_status() == q.QG_OK
