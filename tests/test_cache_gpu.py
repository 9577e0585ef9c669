"""Page tables from request lengths, K/V append and branch commit on the GPU
against plain loops (every output is exact), and whole speculative-decoding
steps against a dense model of the cache."""
import math

import numpy as np
import pytest
import torch

import synth
from paged_non_uniform_gb300 import kvx
from tree_cases import Case, Setup, ref_tables, slot_of, to_dev, visible

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Tables:
    """Device state of the table call: tables, free lists, counts."""

    def __init__(self, B, Hkv, hg, P, stride, pages, token_major=False, seed=0, D=64, g=1, dtype="bf16",
                 pools=None):
        self.B, self.Hkv, self.hg, self.P = B, Hkv, list(hg), P
        self.G = max(hg) + 1
        r = self.r = synth.rng(seed)
        self.tm = token_major
        self.pages, self.stride = [pages] * self.G, stride
        self.tables = [np.full((B, stride), -9, np.int32) for _ in range(self.G)]
        self.free = [r.permutation(pages).astype(np.int32) for _ in range(self.G)]
        self.count = np.full(self.G, pages, np.int64)
        self.held = np.zeros((self.G, B), np.int64)
        self.dt = [dev(t) for t in self.tables]
        self.df = [dev(f) for f in self.free]
        dummy = torch.zeros(64, dtype=torch.int32, device="cuda")
        kp, vp = pools or ([dummy] * self.G, [dummy] * self.G)
        self.cache = kvx.Cache(B, Hkv * g, Hkv, D, P, self.G,
                               kvx.KVX_BF16 if dtype == "bf16" else kvx.KVX_F32, self.hg, kp, vp, self.pages,
                               self.dt, [stride] * self.G,
                               layout=kvx.KVX_LAYOUT_TOKEN_MAJOR if token_major else kvx.KVX_LAYOUT_HEAD_MAJOR)
        self.d_in, self.d_out = dev(self.held.astype(np.int32)), torch.zeros_like(dev(self.held.astype(np.int32)))
        self.c_in, self.c_out = dev(self.count.astype(np.int32)), dev(np.zeros(self.G, np.int32))
        self.ws = torch.zeros(64, dtype=torch.int32, device="cuda")
        self.q_start = torch.full((B + 1,), -3, dtype=torch.int32, device="cuda")

    def call(self, kv, new, max_rows=None, stream=None):
        self.max_rows = int(np.maximum(new, 0).sum()) + 2 if max_rows is None else max_rows
        self.slots = torch.full((self.max_rows, self.Hkv), -7, dtype=torch.int64, device="cuda")
        kvx.kvx_build_tables(self.cache, dev(np.asarray(kv, np.int32)), dev(np.asarray(new, np.int32)),
                             self.d_in, self.d_out, self.df, self.c_in, self.c_out, self.max_rows,
                             self.q_start, self.slots, self.ws, stream=stream)

    def check(self, kv, new):
        t, pages, free, left, qs, slots = ref_tables(kv, new, self.hg, self.G, self.P, self.tables, self.held,
                                                     self.free, self.count, self.tm)
        torch.cuda.synchronize()
        for g in range(self.G):
            assert np.array_equal(self.dt[g].cpu().numpy(), t[g]), g
            assert np.array_equal(self.df[g].cpu().numpy(), free[g]), g
        assert np.array_equal(self.d_out.cpu().numpy(), pages)
        assert np.array_equal(self.c_out.cpu().numpy(), left)
        assert np.array_equal(self.q_start.cpu().numpy(), qs)
        got = self.slots.cpu().numpy()
        assert np.array_equal(got[:len(slots)], slots) and np.all(got[len(slots):] == -7)
        assert kvx.kvx_workspace_status(self.ws) == 0
        return t, pages, free, left

    def step(self, kv, new):
        self.call(kv, new)
        self.tables, self.held, self.free, self.count = self.check(kv, new)
        self.d_in, self.d_out = self.d_out, self.d_in
        self.c_in, self.c_out = self.c_out, self.c_in


@pytest.mark.parametrize("seed", range(8))
def test_tables_over_many_steps(seed):
    """Sequences start with prompts, grow by drafts, lose rejected ones, end and start again."""
    r = np.random.default_rng(seed + 50)
    Hkv = int(r.integers(1, 9))
    G = int(r.integers(1, min(Hkv, 4) + 1))
    hg = np.concatenate([np.arange(G), r.integers(0, G, Hkv - G)])
    r.shuffle(hg)
    B, P = int(r.choice([1, 3, 17, 70])), int(r.choice([8, 16, 32, 64, 128]))
    longest = 40 * P
    t = Tables(B, Hkv, hg.tolist(), P, 45, 45 * B + 3, bool(seed % 2), seed)
    kv = np.zeros((B, Hkv), np.int64)
    for _ in range(8):
        new = np.where(r.random(B) < 0.3, 0, r.integers(1, 24, B))
        start = r.random(B) < 0.2
        kv[start] = 0
        new[start] = r.integers(0, 3 * P, int(start.sum()))
        t.step(kv, new)
        kv = np.minimum(kv + r.integers(0, 1 + np.maximum(new, 0))[:, None], longest)
        kv = np.maximum(0, kv - r.integers(0, 2, kv.shape) * r.integers(0, 5))  # heads drift apart
    t.step(np.zeros((B, Hkv)), np.zeros(B, np.int64))  # everything ends: every page is free again
    assert t.count.tolist() == t.pages
    for g in range(G):
        assert sorted(t.free[g].tolist()) == list(range(t.pages[g]))


@pytest.mark.parametrize("B", [1, 255, 256, 257, 4096])
def test_tables_batch_sizes(B):
    r = np.random.default_rng(B)
    t = Tables(B, 2, [0, 1], 16, 12, 12 * B + 1, seed=B)
    t.step(r.integers(0, 60, (B, 2)) * 0, r.integers(0, 60, B))
    t.step(r.integers(0, 60, (B, 2)), r.integers(0, 60, B))


def test_tables_long_prompt_and_no_rows():
    t = Tables(2, 3, [0, 1, 1], 16, 5000, 10000, True)
    t.step(np.zeros((2, 3), np.int64), np.array([70001, 1]))
    t.step(np.array([[70001, 5, 70001], [0, 0, 0]]), np.array([0, 0]))
    t.call(np.zeros((2, 3)), np.zeros(2, np.int64), max_rows=0)
    t.check(np.zeros((2, 3)), np.zeros(2, np.int64))


def test_tables_call_repeats():
    """The same inputs again give the same outputs (counts are not updated in place)."""
    t = Tables(5, 2, [0, 1], 8, 20, 60, seed=3)
    t.step(np.zeros((5, 2), np.int64), np.array([30, 9, 0, 60, 8]))
    kv, new = np.array([[20, 30], [0, 0], [0, 0], [17, 3], [8, 8]]), np.array([4, 0, 33, 1, 9])
    for _ in range(3):
        t.call(kv, new)
        t.check(kv, new)


def unchanged(t, before, status):
    torch.cuda.synchronize()
    assert kvx.kvx_workspace_status(t.ws) == status
    for g in range(t.G):
        assert np.array_equal(t.dt[g].cpu().numpy(), before[0][g])
        assert np.array_equal(t.df[g].cpu().numpy(), before[1][g])
    assert np.array_equal(t.d_out.cpu().numpy(), t.d_in.cpu().numpy())
    assert np.array_equal(t.c_out.cpu().numpy(), t.c_in.cpu().numpy())
    assert np.all(t.q_start.cpu().numpy() == 0) and np.all(t.slots.cpu().numpy() == -7)


@pytest.mark.parametrize("what", ["kv", "new", "length", "rows", "held", "free", "pages", "overfull"])
def test_tables_refuse_bad_lengths_whole(what):
    t = Tables(3, 2, [0, 1], 8, 6, 14, seed=4)
    t.step(np.zeros((3, 2), np.int64), np.array([30, 9, 12]))
    kv, new = np.array([[20, 30], [3, 9], [0, 0]]), np.array([4, 2, 5])
    status, max_rows = kvx.KVX_DEV_BAD_LENGTH, 16
    if what == "kv":
        kv[1, 1] = -1
    elif what == "new":
        new[2] = -2
    elif what == "length":
        kv[0, 0] = 6 * 8 - 3  # 4 new rows pass the table
    elif what == "rows":
        max_rows = 10
    elif what == "held":
        t.d_in[1, 2] = 7
    elif what == "free":
        t.c_in[0] = -1
    elif what == "overfull":
        t.c_in[1] = 14  # more free pages than the pool has besides those released
        kv[:] = 0
        new[:] = 0
    else:
        new[:] = (18, 30, 40)
        kv[:] = ((30, 30), (18, 18), (8, 8))
        status, max_rows = kvx.KVX_DEV_NO_PAGES, 100
    before = [x.cpu().numpy() for x in t.dt], [x.cpu().numpy() for x in t.df]
    t.call(kv, new, max_rows)
    unchanged(t, before, status)


def test_tables_bad_page_ids_give_no_slot():
    t = Tables(2, 1, [0], 8, 4, 8, seed=5)
    t.df[0][-1] = 8
    t.free[0][-1] = 8
    t.call(np.zeros((2, 1)), np.array([8, 9]))
    torch.cuda.synchronize()
    got = t.slots.cpu().numpy()[:17, 0]
    assert np.all(got[:8] == -1) and np.all(got[8:] >= 0)
    assert kvx.kvx_workspace_status(t.ws) == kvx.KVX_DEV_BAD_PAGE


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("case", [
    Case("bf16", 128, 2, 4, (0, 1), kv=((40, 7), (0, 300)), T=(5, 1)),
    Case("bf16", 64, 3, 1, (0, 1, 0), P=8, token_major=True, kv=((40, 7, 1), (9, 8, 7)), T=(0, 33)),
    Case("f32", 128, 1, 2, (0,), P=128, kv=((126,),), T=(400,)),
    Case("f32", 64, 4, 2, (1, 0, 1, 1), P=32, token_major=True, kv=((1, 2, 3, 4),) * 4, T=(3, 0, 1, 65)),
], ids=lambda c: c.name)
@pytest.mark.parametrize("strided", [False, True])
def test_append(case, strided):
    s = Setup(case)
    new = [synth.normal(s.r, (s.max_rows, s.Hkv * case.D), case.dtype) for _ in range(2)]
    want = [[a.copy() for a in pool] for pool in (s.k, s.v)]
    slots = s.slots()
    slots[s.N:] = 0  # rows behind the last sequence are not written
    for r in range(s.N):
        for h in range(s.Hkv):
            for x in range(2):
                want[x][s.hg[h]][slots[r, h]] = new[x][r].reshape(s.Hkv, -1)[h]
    s.cache_ws = None
    c = case
    s.dk = [to_dev(a, c.dtype) for a in s.k]
    s.dv = [to_dev(a, c.dtype) for a in s.v]
    s.dt = [dev(t) for t in s.tables]
    cache = kvx.Cache(s.B, s.Hq, s.Hkv, c.D, c.P, s.G, kvx.KVX_BF16 if c.dtype == "bf16" else kvx.KVX_F32,
                      s.hg, s.dk, s.dv, s.pages, s.dt, s.stride,
                      layout=kvx.KVX_LAYOUT_TOKEN_MAJOR if c.token_major else kvx.KVX_LAYOUT_HEAD_MAJOR)
    k, v = to_dev(new[0], c.dtype), to_dev(new[1], c.dtype).view(s.max_rows, s.Hkv, c.D)
    if strided:
        w = s.Hkv * c.D
        both = torch.cat([torch.zeros_like(k[:, :8]), k, v.reshape(s.max_rows, -1), k[:, :16]], 1)
        k, v = both[:, 8:8 + w], both[:, 8 + w:8 + 2 * w]
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    kvx.kvx_append_kv(cache, k, v, dev(s.q_start), dev(slots), s.max_rows, ws)
    torch.cuda.synchronize()
    for got, ref in zip((s.dk, s.dv), want):
        for g in range(s.G):
            assert np.array_equal(got[g].float().cpu().numpy(), ref[g], equal_nan=True)
    assert kvx.kvx_workspace_status(ws) == 0


def test_append_bad_slots_are_skipped_and_flagged():
    s = Setup(Case(kv=((40, 7),), T=(4,))).upload()
    slots = s.slots()
    limit = s.pages[0] * 2 * 16
    before = s.dk[0].clone()
    new = torch.ones(s.max_rows, 2 * 128, dtype=torch.bfloat16, device="cuda")
    bad = np.full_like(slots, -1)
    kvx.kvx_append_kv(s.cache, new, new, s.dqs, dev(bad), s.max_rows, s.ws)
    torch.cuda.synchronize()
    assert s.status() == 0  # -1: no slot
    bad[:4] = np.array([[limit, -2], [1 << 40, -(1 << 40)], [limit + 7, limit], [-1, -1]])
    kvx.kvx_append_kv(s.cache, new, new, s.dqs, dev(bad), s.max_rows, s.ws)
    torch.cuda.synchronize()
    assert s.status() == kvx.KVX_DEV_BAD_BLOCK
    assert torch.equal(s.dk[0].view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("rows", [0, -5, 10 ** 9])
def test_append_row_count_stays_inside_the_arrays(rows):
    """q_start[B] below 0 writes nothing; above max_rows, max_rows rows are all there is."""
    s = Setup(Case(kv=((40, 7),), T=(4,)), extra_rows=0).upload()
    new = torch.ones(4, 2 * 128, dtype=torch.bfloat16, device="cuda")
    before = s.dk[0].clone()
    kvx.kvx_append_kv(s.cache, new, new, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                      dev(s.slots()), 4, s.ws)
    torch.cuda.synchronize()
    changed = int((s.dk[0].view(torch.int16) != before.view(torch.int16)).any(1).sum())
    assert changed == (8 if rows > 0 else 0)


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("case", [
    Case("bf16", 128, 2, 4, (0, 1), kv=((40, 7), (0, 300), (15, 16)), T=(5, 1, 64)),
    Case("bf16", 64, 3, 1, (0, 1, 0), P=8, token_major=True, kv=((40, 7, 1), (9, 8, 7)), T=(0, 33)),
    Case("f32", 128, 1, 2, (0,), P=128, kv=((126,),), T=(400,)),
    Case("f32", 64, 4, 2, (1, 0, 1, 1), P=32, token_major=True, kv=((1, 2, 3, 4),) * 4, T=(3, 0, 1, 65)),
], ids=lambda c: c.name)
@pytest.mark.parametrize("keep", ["some", "all", "none", "last"])
def test_commit(case, keep):
    s = Setup(case).upload()
    width = max(1, int(max(case.T)))
    path, acc = np.full((s.B, width), 10 ** 6, np.int32), np.zeros(s.B, np.int32)
    want = [[a.copy() for a in pool] for pool in (s.k, s.v)]
    for b in range(s.B):
        T = int(s.T[b])
        p = np.arange(T)
        if keep == "some":
            p = np.flatnonzero(s.r.random(T) < 0.5)
        elif keep == "none":
            p = p[:0]
        elif keep == "last":
            p = p[-1:]
        acc[b] = p.size
        path[b, :p.size] = p
        for h in range(s.Hkv):
            to, of = s.rows_of(b, h, s.kv[b, h] + np.arange(p.size)), s.rows_of(b, h, s.kv[b, h] + p)
            for pool, ref in zip((s.k, s.v), want):
                ref[s.hg[h]][to] = pool[s.hg[h]][of]
    out = torch.full((s.B, s.Hkv), -1, dtype=torch.int32, device="cuda")
    kvx.kvx_tree_commit(s.cache, s.dqs, dev(s.slots()), s.max_rows, dev(path), dev(acc), s.dkv, out, s.ws)
    torch.cuda.synchronize()
    assert s.status() == 0
    assert np.array_equal(out.cpu().numpy(), s.kv + acc[:, None])
    for got, ref in zip((s.dk, s.dv), want):
        for g in range(s.G):
            assert np.array_equal(got[g].float().cpu().numpy(), ref[g], equal_nan=True)


@pytest.mark.parametrize("path,acc", [([2, 1], 2), ([0, 0], 2), ([0, 5], 2), ([-1, 2], 2), ([0, 1], -1),
                                      ([0, 1], 3), ([0, 1], 6)])
def test_commit_refuses_bad_paths_by_sequence(path, acc):
    """A path out of order or range keeps its sequence's rows and lengths; the other sequence moves
    on, in place."""
    s = Setup(Case(kv=((40, 7), (3, 9)), T=(5, 5))).upload()
    before = s.dk[0].clone()
    kvx.kvx_tree_commit(s.cache, s.dqs, dev(s.slots()), s.max_rows,
                        dev(np.array([path, [0, 3]], np.int32)), dev(np.array([acc, 2], np.int32)), s.dkv,
                        s.dkv, s.ws)
    torch.cuda.synchronize()
    assert s.dkv.cpu().numpy().tolist() == [[40, 7], [5, 11]]
    assert s.status() == kvx.KVX_DEV_BAD_LENGTH
    for h in range(2):
        of, to = s.rows_of(1, h, s.kv[1, h] + np.array([3])), s.rows_of(1, h, s.kv[1, h] + np.array([1]))
        before[torch.from_numpy(to).cuda()] = before[torch.from_numpy(of).cuda()]
    assert torch.equal(s.dk[0].view(torch.int16), before.view(torch.int16))


def test_commit_skips_slots_outside_the_pool():
    s = Setup(Case(kv=((40, 7),), T=(5,))).upload()
    slots = s.slots()
    slots[3] = [-1, 1 << 40]
    before = s.dv[0].clone()
    kvx.kvx_tree_commit(s.cache, s.dqs, dev(slots), s.max_rows, dev(np.array([[3]], np.int32)),
                        dev(np.array([1], np.int32)), s.dkv, s.dkv, s.ws)
    torch.cuda.synchronize()
    assert s.status() == kvx.KVX_DEV_BAD_BLOCK
    assert torch.equal(s.dv[0].view(torch.int16), before.view(torch.int16))


# ---------------------------------------------------------------- the step as a whole
@pytest.mark.parametrize("dtype,token_major,graph", [("bf16", False, False), ("bf16", True, True),
                                                     ("f32", False, True)])
def test_speculative_steps_end_to_end(dtype, token_major, graph):
    """Prompts, then verify steps with random trees, ends and restarts: tables -> append -> attention
    -> commit on one stream (or one captured graph replayed with the lengths of each step), against
    dense per-head lists of rows and softmax attention in 64 bits."""
    r = np.random.default_rng(77)
    B, Hkv, g, D, P = 3, 2, 2, 64, 8
    hg, Hq = [0, 1], 4
    pages, stride, max_rows, max_q, depth = 90, 40, 48, 16, 8
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kp = [torch.full((pages * P, D), float("nan"), dtype=tt, device="cuda") for _ in range(2)]
    vp = [torch.full((pages * P, D), float("nan"), dtype=tt, device="cuda") for _ in range(2)]
    t = Tables(B, Hkv, hg, P, stride, pages, token_major, 1, D, g, dtype, (kp, vp))
    i32 = dict(dtype=torch.int32, device="cuda")
    kv, new = torch.zeros(B, Hkv, **i32), torch.zeros(B, **i32)
    slots = torch.zeros(max_rows, Hkv, dtype=torch.int64, device="cuda")
    fused = torch.zeros(max_rows, (Hq + 2 * Hkv) * D, dtype=tt, device="cuda")
    q, k, v = fused[:, :Hq * D], fused[:, Hq * D:(Hq + Hkv) * D], fused[:, (Hq + Hkv) * D:]
    mask, out = torch.zeros(max_rows, 1, **i32), torch.zeros(max_rows, Hq, D, device="cuda")
    path, acc = torch.zeros(B, depth, **i32), torch.zeros(B, **i32)
    ws = torch.zeros(-(-kvx.kvx_tree_attn_workspace_bytes(t.cache, max_q) // 4), **i32)

    def step():
        kvx.kvx_build_tables(t.cache, kv, new, t.d_in, t.d_out, t.df, t.c_in, t.c_out, max_rows, t.q_start,
                             slots, ws)
        kvx.kvx_append_kv(t.cache, k, v, t.q_start, slots, max_rows, ws)
        kvx.kvx_tree_attn(t.cache, q, t.q_start, max_rows, max_q, kv, mask, 0.0, out, ws)
        kvx.kvx_tree_commit(t.cache, t.q_start, slots, max_rows, path, acc, kv, kv, ws)
        t.d_in.copy_(t.d_out)
        t.c_in.copy_(t.c_out)

    captured = None
    cache = [[([], []) for _ in range(Hkv)] for _ in range(B)]  # rows of K and V by head
    for n in range(12):
        T = r.integers(0, max_q + 1, B)
        restart = r.random(B) < 0.15
        words, data = np.zeros((max_rows, 1), np.uint32), synth.normal(r, (max_rows, (Hq + 2 * Hkv) * D), dtype)
        paths, accs, see = np.zeros((B, depth), np.int32), np.zeros(B, np.int32), []
        start = np.concatenate([[0], np.cumsum(T)])
        for b in range(B):
            if restart[b]:
                cache[b] = [([], []) for _ in range(Hkv)]
                kv[b] = 0
            vis = visible(r, "tree", int(T[b]))
            see.append(vis)
            if T[b]:
                leaf = int(r.integers(0, T[b]))
                p = np.flatnonzero(vis[leaf])[:depth]
                accs[b], paths[b, :p.size] = p.size, p
            for i in range(int(T[b])):
                words[start[b] + i, 0] = sum(int(vis[i, j]) << j for j in range(int(T[b])))
        new.copy_(torch.from_numpy(T.astype(np.int32)))
        fused.copy_(to_dev(data, dtype))
        mask.copy_(torch.from_numpy(words.view(np.int32)))
        path.copy_(torch.from_numpy(paths))
        acc.copy_(torch.from_numpy(accs))
        if not graph:
            step()
        else:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    step()
            captured.replay()
        torch.cuda.synchronize()
        assert kvx.kvx_workspace_status(ws) == 0
        got = out.cpu().numpy().astype(np.float64)
        for b in range(B):
            rows = data[start[b]:start[b + 1]].astype(np.float64)
            for h in range(Hkv):
                ck, cv = cache[b][h]
                nk = rows[:, (Hq + h) * D:(Hq + h + 1) * D]
                nv = rows[:, (Hq + Hkv + h) * D:(Hq + Hkv + h + 1) * D]
                K = np.concatenate([np.array(ck).reshape(-1, D), nk])
                V = np.concatenate([np.array(cv).reshape(-1, D), nv])
                for i in range(int(T[b])):
                    ok = np.concatenate([np.ones(len(ck), bool), see[b][i]])
                    for j in range(g):
                        s = K[ok] @ rows[i, (h * g + j) * D:(h * g + j + 1) * D] / math.sqrt(D)
                        w = np.exp(s - s.max())
                        # error bound of tree_cases with |s| < 8, at most 300 keys: below 2e-4 of
                        # the largest value
                        err = np.abs(got[start[b] + i, h * g + j] - (w / w.sum()) @ V[ok]).max()
                        assert err <= 2e-4 * np.abs(V).max(), (n, b, h, i, j, err)
                for x in paths[b, :accs[b]]:
                    ck.append(nk[x])
                    cv.append(nv[x])
        assert kv.cpu().numpy().tolist() == [[len(cache[b][h][0]) for h in range(Hkv)] for b in range(B)]


def test_step_with_too_few_pages_does_nothing():
    """A table call that cannot be served leaves q_start 0, so that the calls after it write nothing."""
    s = Setup(Case(kv=((40, 7), (3, 9)), T=(5, 5))).upload()
    held = dev(s.need.astype(np.int32))
    free_in, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros_like(held)
    free = torch.zeros(s.pages[0], dtype=torch.int32, device="cuda")
    slots = torch.full((40, 2), -7, dtype=torch.int64, device="cuda")
    qs = torch.zeros(3, dtype=torch.int32, device="cuda")
    before = s.dk[0].clone()
    kvx.kvx_build_tables(s.cache, s.dkv, dev(np.array([8, 20], np.int32)), held, out, [free], free_in,
                         torch.zeros_like(free_in), 40, qs, slots, s.ws)
    new = torch.ones(40, 256, dtype=torch.bfloat16, device="cuda")
    kvx.kvx_append_kv(s.cache, new, new, qs, slots, 40, s.ws)
    o = torch.full((40, 8, 128), -7.0, device="cuda")
    s.ws2 = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(s.cache, 20) // 4, dtype=torch.int32, device="cuda")
    kvx.kvx_tree_attn(s.cache, torch.ones(40, 8, 128, dtype=torch.bfloat16, device="cuda"), qs, 40, 20, s.dkv,
                      None, 0.0, o, s.ws2)
    torch.cuda.synchronize()
    assert s.status() == kvx.KVX_DEV_NO_PAGES and kvx.kvx_workspace_status(s.ws2) == 0
    assert torch.all(o == -7.0) and torch.equal(s.dk[0].view(torch.int16), before.view(torch.int16))
