"""Eviction against a plain reading of its contract (whole numbers and copies: exact)."""
import numpy as np
import pytest
import torch

from budget_cases import BCase, Budget, ref_evict
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu


class Evict(Budget):
    """A cache without new rows, its weights and budgets."""

    def __init__(self, c, budget, kind="random"):
        super().__init__(c)
        r = np.random.default_rng(c.seed + 9)
        self.budget = np.array(budget, np.int32)
        for w in self.w:
            if kind == "equal":
                w[:] = 0.25
            elif kind == "ties":
                w[:] = r.integers(-2, 3, w.size)
            elif kind == "odd":
                w[:] = np.where(r.random(w.size) < 0.3, 0, r.standard_normal(w.size))
                for i, v in enumerate((np.nan, -np.inf, np.inf, -0.0, 1e-42, -1e-42)):
                    w[r.random(w.size) < 0.1] = v
            elif kind == "skewed":
                w[:] = np.exp(6 * r.standard_normal(w.size))

    def upload(self):
        super().upload()
        self.dbudget = torch.from_numpy(self.budget).cuda()
        self.dout = [torch.full_like(w, -5.0) for w in self.dw]
        self.kv_out = torch.full_like(self.dkv, -1)
        n = kvx.kvx_evict_workspace_bytes(self.cache)
        self.ews = torch.zeros(-(-n // 4), dtype=torch.int32, device="cuda")
        return self

    def evict(self, sinks, recent, in_place, kv_out=None):
        kvx.kvx_evict(self.cache, self.dkv, self.dbudget, sinks, recent, self.dw,
                      self.dw if in_place else self.dout, self.kv_out if kv_out is None else kv_out, self.ews)

    def check_evicted(self, sinks, recent, in_place, before):
        torch.cuda.synchronize()
        assert kvx.kvx_workspace_status(self.ews) == 0
        k0, v0, w0 = before
        k = [x.view(torch.uint8).cpu().numpy().reshape(w.size, -1) if not self.c.q4 else x.cpu().numpy()
             for x, w in zip(self.dk, self.w)]
        v = [x.view(torch.uint8).cpu().numpy().reshape(w.size, -1) if not self.c.q4 else x.cpu().numpy()
             for x, w in zip(self.dv, self.w)]
        ek, ev = [x.copy() for x in k0], [x.copy() for x in v0]
        ew = [x.copy() if in_place else np.full_like(x, -5.0) for x in w0]
        n_out = np.zeros_like(self.kv)
        for b in range(self.B):
            for h in range(self.Hkv):
                g, n = self.hg[h], int(self.kv[b, h])
                at = self.rows_of(b, h, np.arange(n))
                keep = ref_evict(w0[g][at], n, int(self.budget[b, h]), sinks, recent)
                n_out[b, h] = keep.size
                to = at[:keep.size]
                ew[g][to] = w0[g][at[keep]]
                for e, x0 in ((ek, k0), (ev, v0)):
                    if self.c.q4:
                        self.move(e[g], x0[g], to, at[keep])
                    else:
                        e[g][to] = x0[g][at[keep]]
        got_w = self.dw if in_place else self.dout
        for g in range(self.G):
            assert np.array_equal(k[g], ek[g]) and np.array_equal(v[g], ev[g])
            assert np.array_equal(got_w[g].cpu().numpy(), ew[g], equal_nan=True)
        assert np.array_equal(self.kv_out.cpu().numpy(), n_out)
        return n_out

    def move(self, to_buf, of_buf, to, of):
        c = self.c
        t, o = (x.reshape(-1, c.P * (c.D // 2 + c.D // 16)) for x in (to_buf, of_buf))
        for a, b in zip(to, of):
            for size, base in ((c.D // 2, 0), (c.D // 16, c.P * c.D // 2)):
                t[a // c.P, base + a % c.P * size:base + (a % c.P + 1) * size] = \
                    o[b // c.P, base + b % c.P * size:base + (b % c.P + 1) * size]

    def snapshot(self):
        q4 = self.c.q4
        f = lambda xs: [x.cpu().numpy().copy() if q4 else  # noqa: E731
                        x.view(torch.uint8).cpu().numpy().reshape(w.size, -1).copy() for x, w in zip(xs, self.w)]
        return f(self.dk), f(self.dv), [w.copy() for w in self.w]


def case(kv, dtype="bf16", D=128, groups=(0, 1), **k):
    return BCase(dtype, D, len(kv[0]), 2, groups, kv=kv, T=(0,) * len(kv), **k)


CASES = [
    (case(((700, 130), (40, 0))), ((300, 100), (40, 5)), 4, 16, "random"),
    (case(((700, 130), (40, 9)), token_major=True, groups=(0, 0)), ((1, 0), (39, 8)), 2, 3, "skewed"),
    (case(((65, 64), (63, 1)), P=8), ((64, 63), (1, 1)), 0, 0, "ties"),
    (case(((1000, 900),), P=128), ((500, 899),), 10, 600, "equal"),       # recent larger than the budget
    (case(((1000, 900),), P=64, D=64), ((500, 400),), 600, 10, "equal"),  # sinks larger than the budget
    (case(((2000, 999), (1500, 77)), dtype="f32"), ((700, 998), (64, 70)), 1, 1, "odd"),
    (case(((400, 333),), dtype="f32", D=64, token_major=True), ((200, 100),), 3, 5, "odd"),
    (case(((777, 300), (5, 130)), q4=True), ((200, 299), (4, 64)), 4, 8, "skewed"),
    (case(((333, 100),), q4=True, D=64, P=8), ((100, 50),), 0, 7, "ties"),
    (case(((20000, 5000),)), ((6000, 4999),), 4, 64, "skewed"),
    (case(((100, 50), (3, 0))), ((200, 50), (1 << 30, 0)), 4, 8, "random"),  # nothing to drop
]


@pytest.mark.parametrize("c,budget,sinks,recent,kind", CASES, ids=lambda x: getattr(x, "name", None))
@pytest.mark.parametrize("in_place", [True, False])
def test_against_the_contract(c, budget, sinks, recent, kind, in_place):
    s = Evict(c, budget, kind)
    s.upload()
    before = s.snapshot()
    s.evict(sinks, recent, in_place)
    s.check_evicted(sinks, recent, in_place, before)


def test_many_short_heads():
    """More heads than SMs: a small block each; and a repeated call on what the first one left."""
    r = np.random.default_rng(1)
    kv = tuple(tuple(int(x) for x in r.integers(0, 400, 2)) for _ in range(90))
    budget = [[int(x) for x in r.integers(0, 300, 2)] for _ in range(90)]
    s = Evict(case(kv, dtype="f32", D=64, P=8), budget, "ties")
    s.upload()
    before = s.snapshot()
    s.evict(2, 9, True)
    s.kv = s.check_evicted(2, 9, True, before)
    s.w = [w.cpu().numpy() for w in s.dw]
    s.dkv.copy_(s.kv_out)
    s.budget //= 2
    s.dbudget.copy_(torch.from_numpy(s.budget))
    before = s.snapshot()
    s.evict(2, 9, True)
    s.check_evicted(2, 9, True, before)


def test_head_longer_than_the_blocks_keys():
    """One head of 140,000 tokens: its eight blocks read part of their keys from memory in every pass."""
    s = Evict(case(((140000,),), dtype="f32", D=64, groups=(0,), P=128), ((70001,),), "ties")
    s.upload()
    before = s.snapshot()
    s.evict(5, 100, True)
    s.check_evicted(5, 100, True, before)


def test_lengths_in_place_and_bad_ones():
    s = Evict(case(((300, 200), (100, 90))), ((100, -1), (50, 40)))
    s.upload()
    s.dkv[1, 0] = -4
    s.kv_out = s.dkv
    k = [x.clone() for x in s.dk]
    s.evict(1, 2, True)
    torch.cuda.synchronize()
    assert kvx.kvx_workspace_status(s.ews) == kvx.KVX_DEV_BAD_LENGTH
    assert s.dkv.cpu().numpy().tolist() == [[100, 200], [-4, 40]]
    at = torch.from_numpy(s.rows_of(0, 1, np.arange(200))).cuda()
    assert torch.equal(s.dk[1][at].view(torch.int16), k[1][at].view(torch.int16))


def test_bad_page_is_skipped():
    s = Evict(case(((300, 200),)), ((100, 50),))
    s.upload()
    s.dt[0][0, 3] = s.pages[0] + 7
    s.evict(1, 2, True)
    torch.cuda.synchronize()
    assert kvx.kvx_workspace_status(s.ews) == kvx.KVX_DEV_BAD_PAGE
    assert s.kv_out.cpu().numpy().tolist() == [[100, 50]]


def test_captured_eviction():
    """A graph replayed on other lengths, budgets and weights; its workspace needs no clearing between."""
    s = Evict(case(((900, 500), (64, 70))), ((300, 100), (10, 70)), "skewed")
    s.upload()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.evict(4, 8, False)
    for kv, budget in ((((900, 500), (64, 70)), ((300, 100), (10, 70))), (((10, 444), (64, 1)), ((9, 443), (0, 1)))):
        s.kv, s.budget = np.array(kv, np.int64), np.array(budget, np.int32)
        s.dkv.copy_(torch.from_numpy(s.kv.astype(np.int32)))
        s.dbudget.copy_(torch.from_numpy(s.budget))
        for d in s.dout:
            d.fill_(-5.0)
        before = s.snapshot()
        graph.replay()
        s.check_evicted(4, 8, False, before)
