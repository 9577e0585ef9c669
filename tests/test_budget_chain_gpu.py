"""Table, append, weighing attention and eviction as a serving loop runs them: rows appended step by step, heads
held to unequal budgets, pages given back; then a decode over what is left."""
import numpy as np
import pytest
import torch

import synth
from budget_cases import BCase, Budget, ref_evict, values, quantise
from paged_non_uniform_gb300 import kvx
from tree_cases import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(q4, graph):
    B, Hkv, g, D, P, hg = 3, 3, 2, 128, 16, [0, 1, 0]
    G, Hq, T = 2, Hkv * g, 4
    r = synth.rng(5)
    budget = np.array([[40, 100, 33], [64, 17, 20], [1000, 30, 5]], np.int32)
    stride, pages = 16, 60
    size = [hg.count(i) for i in range(G)]
    rank = [hg[:h].count(x) for h, x in enumerate(hg)]
    dt = torch.bfloat16
    pool = lambda i: (torch.full((pages * size[i] * P * 72,), 255, dtype=torch.uint8, device="cuda") if q4 else  # noqa: E731
                      torch.full((pages * size[i] * P, D), float("nan"), dtype=dt, device="cuda"))
    dk, dv = [pool(i) for i in range(G)], [pool(i) for i in range(G)]
    dw = [torch.full((pages * size[i] * P,), float("nan"), device="cuda") for i in range(G)]
    tables = [torch.full((B, stride), -1, dtype=torch.int32, device="cuda") for _ in range(G)]
    cache = kvx.Cache(B, Hq, Hkv, D, P, G, kvx.KVX_Q4 if q4 else kvx.KVX_BF16, hg, dk, dv, [pages] * G, tables,
                      [stride] * G)
    free = [torch.from_numpy(r.permutation(pages).astype(np.int32)).cuda() for _ in range(G)]
    held = [torch.zeros((G, B), dtype=torch.int32, device="cuda") for _ in range(2)]
    left = [torch.full((G,), pages, dtype=torch.int32, device="cuda") for _ in range(2)]
    kv_len = torch.zeros((B, Hkv), dtype=torch.int32, device="cuda")
    none = torch.zeros(B, dtype=torch.int32, device="cuda")
    max_rows = 90
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros((max_rows, Hkv), dtype=torch.int64, device="cuda")
    new_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = [torch.zeros((max_rows, h, D), dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv)]
    out = torch.zeros((max_rows, Hq, D), device="cuda")
    dbudget = torch.from_numpy(budget).cuda()
    max_q = 30
    size_of = lambda n: torch.zeros(-(-n // 4), dtype=torch.int32, device="cuda")  # noqa: E731
    ws, ews = size_of(kvx.kvx_window_attn_workspace_bytes(cache, max_q, True)), size_of(kvx.kvx_evict_workspace_bytes(cache))

    def step():
        kvx.kvx_build_tables(cache, kv_len, new_len, held[0], held[1], free, left[0], left[1], max_rows, q_start,
                             slots, ws)
        kvx.kvx_append_kv(cache, rows[1], rows[2], q_start, slots, max_rows, ws)
        kvx.kvx_window_attn(cache, rows[0], q_start, max_rows, max_q, kv_len, None, None, 0.0, out, dw, ws)

    def drop():
        kv_len.add_(new_len[:, None])  # the new rows stay
        kvx.kvx_evict(cache, kv_len, dbudget, 2, 6, dw, dw, kv_len, ews)
        kvx.kvx_build_tables(cache, kv_len, none, held[1], held[0], free, left[1], left[0], 0, q_start, None, ws)

    graphs = None
    toks = [[[] for _ in range(Hkv)] for _ in range(B)]  # (k, v) float64 of every head's tokens
    wts = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]
    for it, lens in enumerate(([30, 1, 17], [4, 4, 4], [1, 0, 1], [25, 30, 30], [1, 1, 1], [1, 1, 0])):
        host = [synth.normal(r, t.shape, "bf16") for t in rows]
        for t, x in zip(rows, host):
            t.copy_(to_dev(x, "bf16"))
        new_len.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        if graph and it == 1:
            before = [x.clone() for x in dk + dv + dw + tables + free + held + left + [kv_len]]
            graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            for gr, f in zip(graphs, (step, drop)):
                with torch.cuda.graph(gr):
                    f()
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(before, dk + dv + dw + tables + free + held + left + [kv_len]))
        graphs[0].replay() if graphs else step()
        torch.cuda.synchronize()
        assert kvx.kvx_workspace_status(ws) == 0
        cu = np.concatenate([[0], np.cumsum(lens)])
        got = out.cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                k, v = host[1][cu[b]:cu[b + 1], h], host[2][cu[b]:cu[b + 1], h]
                if q4:
                    k, v = (values(*quantise(x)) for x in (k, v))
                n = len(toks[b][h])
                toks[b][h] += [(np.float64(a), np.float64(c)) for a, c in zip(k, v)]
                w = np.concatenate([wts[b][h], np.zeros(lens[b])])
                for i in range(lens[b]):
                    K = np.array([t[0] for t in toks[b][h][:n + i + 1]])
                    V = np.array([t[1] for t in toks[b][h][:n + i + 1]])
                    for j in range(g):
                        s = K @ host[0][cu[b] + i, h * g + j].astype(np.float64) / np.sqrt(D)
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        # bounds far above the roundings that test_window_gpu holds the call to
                        assert np.abs(got[cu[b] + i, h * g + j] - p @ V).max() < 1e-4
                        w[:n + i + 1] += p
                wts[b][h] = w
        at = lambda b, h, t: (tables[hg[h]].cpu().numpy()[b, t // P].astype(np.int64) * size[hg[h]] + rank[h]) * P + t % P  # noqa: E731
        wd = [x.cpu().numpy() for x in dw]
        for b in range(B):
            for h in range(Hkv):
                mine = wd[hg[h]][at(b, h, np.arange(len(toks[b][h])))]
                assert np.abs(mine - wts[b][h]).max(initial=0) < 1e-4
                # what the library weighed decides what it drops
                keep = ref_evict(mine, mine.size, int(budget[b, h]), 2, 6)
                toks[b][h] = [toks[b][h][t] for t in keep]
                wts[b][h] = wts[b][h][keep]
        graphs[1].replay() if graphs else drop()
        torch.cuda.synchronize()
        assert kvx.kvx_workspace_status(ews) == 0 and kvx.kvx_workspace_status(ws) == 0
        n = kv_len.cpu().numpy()
        assert n.tolist() == [[len(toks[b][h]) for h in range(Hkv)] for b in range(B)]
        need = [[-(-max(int(n[b, h]) for h in range(Hkv) if hg[h] == i) // P) for b in range(B)] for i in range(G)]
        assert held[0].cpu().numpy().tolist() == need
        assert left[0].cpu().numpy().tolist() == [pages - sum(x) for x in need]
