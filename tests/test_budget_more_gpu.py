"""Evictions and windowed attention on paths that the listed sizes do not take: pages outside their pool,
copied weights of heads longer than a block's keys, a long head among many with little room, 4-bit rows
that nobody sees and that hold anything."""
import numpy as np
import pytest
import torch

import synth
from budget_cases import BCase, Budget, ref_evict
from paged_non_uniform_gb300 import kvx
from test_evict_gpu import Evict, case

pytestmark = pytest.mark.gpu


def row_bytes(s, pools):
    return [x.view(torch.uint8).cpu().numpy().reshape(w.size, -1) for x, w in zip(pools, s.w)]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("page,value", [(0, -1), (3, "past"), (11, -5), (17, "past")])
def test_moves_of_a_bad_page_are_skipped_and_no_others(page, value, in_place):
    """Its tokens count as NaN: they stay only as sinks, recent ones or for want of others."""
    n, m, sinks, recent, P = 300, 100, 9, 20, 16
    s = Evict(case(((n, 200),)), ((m, 50),), "skewed")
    s.upload()
    s.dt[0][0, page] = s.pages[0] if value == "past" else value
    k0, v0 = row_bytes(s, s.dk), row_bytes(s, s.dv)
    s.evict(sinks, recent, in_place)
    torch.cuda.synchronize()
    ek, ev = [x.copy() for x in k0], [x.copy() for x in v0]
    ew = [w.copy() if in_place else np.full_like(w, -5.0) for w in s.w]
    bad = False
    for h, (length, most) in enumerate(((n, m), (200, 50))):
        at = s.rows_of(0, h, np.arange(length))
        lost = (np.arange(length) // P == page) if h == 0 else np.zeros(length, bool)
        w = np.where(lost, np.float32(np.nan), s.w[h][at])
        for to, of in enumerate(ref_evict(w, length, most, sinks, recent)):
            if lost[to] or lost[of]:
                bad |= of != to or not in_place
                continue
            for e, x0 in ((ek, k0), (ev, v0)):
                e[h][at[to]] = x0[h][at[of]]
            ew[h][at[to]] = s.w[h][at[of]]
    assert kvx.kvx_workspace_status(s.ews) & ~kvx.KVX_DEV_BAD_PAGE == 0
    assert kvx.kvx_workspace_status(s.ews) or not bad
    assert s.kv_out.cpu().numpy().tolist() == [[m, 50]]
    for got, want in ((row_bytes(s, s.dk), ek), (row_bytes(s, s.dv), ev)):
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    for got, want in zip(s.dw if in_place else s.dout, ew):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["ties", "odd"])
def test_copied_weights_of_a_head_longer_than_the_blocks_keys(kind):
    s = Evict(case(((140000,),), dtype="f32", D=64, groups=(0,), P=128), ((70001,),), kind)
    s.upload()
    before = s.snapshot()
    s.evict(5, 100, False)
    s.check_evicted(5, 100, False, before)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["skewed", "ties"])
def test_a_long_head_among_many_with_little_room(kind, in_place):
    """160 heads, the tables of one group wide, the others' not: their mean room is that of short heads, 4032."""
    kv = ((30000,) + (100, 90, 80, 320, 1, 0, 64),) + ((5, 200, 300, 64, 7, 128, 65, 33),) * 19
    budget = ((11111,) + (40, 90, 0, 64, 1, 5, 63),) + ((3, 100, 64, 1, 9, 128, 64, 32),) * 19
    s = Evict(BCase("bf16", 64, 8, 1, (0,) + (1,) * 7, kv=kv, T=(0,) * 20, P=32), budget, kind)
    assert sum(s.stride[g] * 32 for g in s.hg) // 8 <= 4096
    s.upload()
    before = s.snapshot()
    s.evict(5, 30, in_place)
    s.check_evicted(5, 30, in_place, before)


@pytest.mark.parametrize("in_place", [True, False])
def test_short_heads_in_wide_tables(in_place):
    """Heads of a few tokens whose tables have room for 140,000: most blocks of their clusters have no token."""
    kv, budget = ((140000,), (3,), (130,), (64,), (0,), (700,)), ((9000,), (2,), (70,), (64,), (4,), (0,))
    s = Evict(case(kv, dtype="f32", D=64, groups=(0,), P=128), budget, "odd")
    s.upload()
    before = s.snapshot()
    s.evict(1, 1, in_place)
    s.check_evicted(1, 1, in_place, before)


def spoil(s, buf, rows, step, lo):
    """Other parameters in rows of a 4-bit pool; None: as they were."""
    c = s.c
    b = buf.reshape(-1, c.P * (c.D // 2 + c.D // 16))
    for r in rows:
        at = c.P * c.D // 2 + r % c.P * (c.D // 16)
        par = b[r // c.P, at:at + c.D // 16].view("<u2").reshape(-1, 2)
        for i, x in enumerate((step, lo)):
            if x is not None:
                par[:, i] = synth.f32_to_bf16_bits(np.array([x], np.float32))[0]


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -3e38, -1.0])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 128)])
def test_4_bit_rows_that_nobody_sees_hold_anything(D, P, bad, T):
    c = BCase("bf16", D, 1, 4, (0,), kv=((400,),), T=(T,), sinks=(3,), window=(100,), q4=True, P=P, seed=3)
    clean = Budget(c).upload()
    a = clean.run(True)
    gap = np.arange(3, 400 - 100 + 1)
    for step, lo in ((bad, None), (None, bad), (bad, bad), (bad, 1.0)):
        dirty = Budget(c)
        for bufs in (dirty.bk, dirty.bv):
            spoil(dirty, bufs[0], dirty.rows_of(0, 0, gap), step, lo)
        dirty.upload()
        assert np.array_equal(a, dirty.run(True))
        seen = torch.from_numpy(clean.rows_of(0, 0, np.setdiff1d(np.arange(400 + T), gap))).cuda()
        assert torch.equal(clean.dw[0][seen], dirty.dw[0][seen])
    # token 301 is seen by new row 0 only, the last new token by the last row
    for t, row in ((301, 0), (400 + T - 1, T - 1)):
        if T > 1 and not np.isfinite(bad):
            one = Budget(c)
            spoil(one, one.bv[0], one.rows_of(0, 0, np.array([t])), None, bad)
            got = one.upload().run()
            others = [i for i in range(T) if i != row]
            assert np.array_equal(got[others], a[others]) and not np.isfinite(got[row]).any()


def test_evictions_and_attention_on_two_streams_at_once():
    """Two caches, each evicted again and again on a stream of its own, beside attention over a third."""
    budget = ((3000, 2500, 900),) * 4
    a, b = (Evict(BCase("bf16", 128, 3, 1, (0, 1, 1), kv=((9000, 5000, 4000),) * 4, T=(0,) * 4, seed=i), budget, "skewed")
            for i in (1, 2))
    c = Budget(BCase("bf16", 128, 2, 4, (0, 1), kv=((3000, 1300),), T=(1,), window=(1000, 2 ** 31 - 1))).upload()
    for s in (a, b):
        s.upload()
        s.before = s.snapshot()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(20):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.evict(4, 64, True)
                # all of it again: heads already at their budgets stay as they are
                kvx.kvx_evict(s.cache, s.kv_out, s.dbudget, 4, 64, s.dw, s.dw, s.kv_out, s.ews)
                if i < 19:  # the rows as they were
                    for d, x in zip(s.dk + s.dv, s.before[0] + s.before[1]):
                        d.view(torch.uint8).view(-1).copy_(torch.from_numpy(x.reshape(-1)), non_blocking=True)
                    for d, w in zip(s.dw, s.w):
                        d.copy_(torch.from_numpy(w), non_blocking=True)
        c.attend(stream=streams[2])
    for s in (a, b):
        s.check_evicted(4, 64, True, s.before)
    c.check(c.out.cpu().numpy())
