"""Attention with windows, sinks and accumulated weights against its definition in float64."""
import numpy as np
import pytest
import torch

from budget_cases import ALL, BCase, Budget
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu

CASES = [
    BCase("bf16", 128, 2, 4, (0, 1), kv=((700, 130), (40, 9)), T=(1, 1), sinks=(4, 0), window=(100, ALL)),
    BCase("bf16", 128, 2, 4, (0, 1), kv=((700, 130), (40, 9)), T=(1, 1)),
    BCase("bf16", 128, 1, 3, (0,), kv=((200,), (0,), (64,)), T=(1, 1, 0), sinks=(2,), window=(64,), P=8),
    BCase("bf16", 64, 2, 8, (0, 0), kv=((900, 900),), T=(1,), sinks=(70, 1), window=(65, 63), token_major=True),
    BCase("bf16", 128, 2, 5, (0, 0), kv=((500, 77), (3, 0), (64, 65)), T=(8, 5, 1), sinks=(5, 64), window=(100, 7),
          P=32, fused=True),
    BCase("bf16", 128, 1, 2, (0,), kv=((1000,),), T=(70,), sinks=(3,), window=(50,), P=64),
    BCase("bf16", 64, 1, 7, (0,), kv=((333,), (5,)), T=(20, 3), sinks=(0,), window=(40,), P=128, token_major=True),
    BCase("bf16", 128, 1, 1, (0,), kv=((300,),), T=(128,), sinks=(1,), window=(128,)),
    BCase("bf16", 128, 4, 1, (1, 0, 1, 0), kv=((5000, 4000, 10, 2000),), T=(1,), sinks=(4, 0, 4, 0),
          window=(ALL, 1000, 5, 1)),
    BCase("bf16", 128, 2, 4, (0, 0), kv=((150, 150),), T=(6,), sinks=(0, 0), window=(0, 1)),  # rows that see nothing
    BCase("bf16", 128, 2, 4, (0, 0), kv=((150, 150),), T=(3,), sinks=(-5, 3), window=(-1, 0)),
    BCase("bf16", 128, 1, 4, (0,), kv=((400,),), T=(4,), window=(90,), spread=6.0),
    BCase("f32", 128, 2, 2, (0, 1), kv=((300, 64), (0, 1)), T=(1, 9), sinks=(4, 1), window=(33, 64)),
    BCase("f32", 64, 1, 8, (0,), kv=((1500,),), T=(6,), sinks=(0,), window=(0,), token_major=True, P=8),
    BCase("bf16", 128, 2, 4, (0, 1), kv=((700, 130), (40, 9)), T=(1, 1), sinks=(4, 0), window=(100, ALL), q4=True),
    BCase("bf16", 64, 2, 3, (0, 0), kv=((333, 1), (0, 64)), T=(2, 5), sinks=(1, 65), window=(64, 10), q4=True, P=8),
    BCase("bf16", 128, 1, 8, (0,), kv=((900,),), T=(7,), q4=True, P=64),
    BCase("bf16", 128, 1, 1, (0,), kv=((4000,), (130,)), T=(1, 4), sinks=(3,), window=(500,), q4=True, P=128),
    BCase("bf16", 64, 4, 2, (0, 1, 1, 0), kv=((100, 200, 300, 400),), T=(1,), q4=True, P=32, spread=5.0),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
@pytest.mark.parametrize("weigh", [False, True])
def test_against_the_definition(c, weigh):
    s = Budget(c).upload()
    got = s.run(weigh=weigh)
    s.check(got, s.dw if weigh else None)
    if not weigh:
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(s.dw, s.w))
    assert s.status() == 0


@pytest.mark.parametrize("c", [CASES[4], CASES[5], CASES[8], CASES[15], CASES[12]], ids=lambda c: c.name)
def test_equal_inputs_give_equal_bits(c):
    a, b = Budget(c).upload(), Budget(c).upload()
    assert np.array_equal(a.run(True), b.run(True))
    assert all(torch.equal(x, y) for x, y in zip(a.dw, b.dw))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [1, 9])
def test_what_a_row_does_not_see_has_no_influence(bad, T, q4):
    """Poisoned tokens in the gap, and, for several rows, in those that only some of them see."""
    c = BCase("bf16", 128, 1, 4, (0,), kv=((400,),), T=(T,), sinks=(3,), window=(100,), q4=q4, seed=3)
    clean, dirty = Budget(c).upload(), Budget(c).upload()
    gap = np.arange(3, 400 - 100)       # nobody sees these
    if q4:
        rows = dirty.rows_of(0, 0, gap)
        for d in (dirty.dk[0], dirty.dv[0]):
            b = d.cpu().numpy()
            mask = np.zeros(dirty.k[0].shape[0], bool)
            mask[rows] = True
            dirty.spoil(b, mask)
            d.copy_(torch.from_numpy(b))
    else:
        for d in (dirty.dk[0], dirty.dv[0]):
            d[torch.from_numpy(dirty.rows_of(0, 0, gap)).cuda()] = bad
    a, b = clean.run(True), dirty.run(True)
    assert np.array_equal(a, b)
    seen = torch.from_numpy(clean.rows_of(0, 0, np.setdiff1d(np.arange(400 + T), gap))).cuda()
    assert torch.equal(clean.dw[0][seen], dirty.dw[0][seen])
    if T == 1 or q4:
        return
    # token 301 is seen by new row 0 only (window 100: t > 400 + i - 100), the last new token by the last row
    for t, row in ((301, 0), (400 + T - 1, T - 1)):
        one = Budget(c).upload()
        one.dv[0][torch.from_numpy(one.rows_of(0, 0, np.array([t]))).cuda(), 5:9] = bad
        got = one.run()
        others = [i for i in range(T) if i != row]
        assert np.array_equal(got[others], a[others])
        assert not np.isfinite(got[row][:, 5:9]).any() and np.array_equal(got[row][:, 9:], a[row][:, 9:])


def test_nan_group_of_a_4_bit_row_that_some_rows_see():
    c = BCase("bf16", 128, 1, 4, (0,), kv=((400,),), T=(9,), sinks=(3,), window=(100,), q4=True, seed=3)
    clean, one = Budget(c).upload(), Budget(c).upload()
    b = one.dv[0].cpu().numpy()
    mask = np.zeros(one.k[0].shape[0], bool)
    mask[one.rows_of(0, 0, np.array([301]))] = True
    one.spoil(b, mask)
    one.dv[0].copy_(torch.from_numpy(b))
    a, got = clean.run(), one.run()
    assert np.array_equal(got[1:9], a[1:9]) and np.isnan(got[0]).all()


def test_bad_pages_and_lengths():
    c = BCase("bf16", 128, 2, 4, (0, 0), kv=((100, 100), (90, 90)), T=(2, 2), window=(50, 50))
    s = Budget(c).upload()
    s.dt[0][0, 5] = s.pages[0]
    s.attend()
    assert s.status() == kvx.KVX_DEV_BAD_PAGE
    good = Budget(c).upload().run()
    out = s.out.cpu().numpy()
    assert np.array_equal(out[2:4], good[2:4]) and np.isfinite(out[:4]).all()
    for q4 in (False, True):
        s = Budget(BCase("bf16", 128, 2, 4, (0, 0), kv=((100, 100), (90, 90)), T=(2, 2), q4=q4)).upload()
        s.dt[0][0, 5] = -3
        s.attend(weigh=True)
        assert s.status() == kvx.KVX_DEV_BAD_PAGE and torch.isfinite(s.out[:4]).all()
    s = Budget(c).upload()
    s.dkv[1, 1] = 1 << 20
    before = [w.clone() for w in s.dw]
    s.attend(weigh=True)
    assert s.status() == kvx.KVX_DEV_BAD_LENGTH
    out = s.out.cpu().numpy()
    assert (out[2:4, 4:] == -7).all() and np.array_equal(out[2:4, :4], good[2:4, :4])
    at = torch.from_numpy(s.rows_of(1, 1, np.arange(90))).cuda()
    assert torch.equal(s.dw[0][at], before[0][at])


@pytest.mark.parametrize("q4", [False, True])
def test_captured_step_follows_the_lengths(q4):
    """One graph, replayed after the device lengths, windows and rows changed; on a stream of its own."""
    big = BCase("bf16", 128, 2, 4, (0, 1), kv=((600, 300), (64, 10)), T=(3, 1), sinks=(4, 2), window=(70, ALL), q4=q4)
    s = Budget(big).upload()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        s.attend(weigh=True)
        with torch.cuda.graph(graph, stream=st):
            s.attend(weigh=True)
    st.synchronize()
    for kv, T, window in ((((600, 300), (64, 10)), (3, 1), (70, ALL)), (((599, 20), (0, 11)), (1, 0), (5, 17))):
        s.kv, s.T = np.array(kv, np.int64), np.array(T, np.int64)
        s.q_start = np.concatenate([[0], np.cumsum(s.T)]).astype(np.int32)
        s.N, s.window = int(s.q_start[-1]), np.array(window, np.int64)
        s.dkv.copy_(torch.from_numpy(s.kv.astype(np.int32)))
        s.dqs.copy_(torch.from_numpy(s.q_start))
        s.dwindow.copy_(torch.from_numpy(s.window.astype(np.int32)))
        for d, w in zip(s.dw, s.w):
            d.copy_(torch.from_numpy(w))
        s.out.fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check(s.out.cpu().numpy(), s.dw)
    assert s.status() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_a_wait_that_runs_out_is_reported(q4):
    s = Budget(BCase("bf16", 128, 1, 4, (0,), kv=((500,),), T=(1,), q4=q4)).upload()
    # (one head: the charge of its item is block 0's part, the first tile is block 1's)
    s.cache.inject_stall(1, 5_000_000)
    s.attend()
    torch.cuda.synchronize()
    assert s.status() & kvx.KVX_DEV_TIMEOUT
    s.cache.inject_stall(-1, 2_000_000_000)
    s.ws.zero_()
    s.check(s.run())
    assert s.status() == 0


def test_workspaces_of_two_streams():
    """Two calls at once, each with its own workspace and outputs."""
    c = BCase("bf16", 128, 2, 4, (0, 1), kv=((3000, 1300),), T=(1,), window=(1000, ALL))
    a, b = Budget(c).upload(), Budget(c).upload()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, st in zip((a, b), streams):
            s.attend(stream=st)
    torch.cuda.synchronize()
    for s in (a, b):
        s.check(s.out.cpu().numpy())
