"""Inputs and plain 64-bit references for the cache calls (page tables from
request lengths, K/V append, tree attention, branch commit).

Test infrastructure only. The references are plain loops over sequences, heads
and rows in NumPy float64 / int64 and share no code with the library. A
`Setup` holds one random paged cache: head-group pools with permuted pages whose
unused slots are NaN, page tables, lengths, masks and query rows.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

import synth
from paged_non_uniform_gb300 import kvx


def ranks(head_group):
    hg = list(head_group)
    return [hg[:h].count(g) for h, g in enumerate(hg)]


def slot_of(page, r, t, size, P, token_major):
    return (page * P + t % P) * size + r if token_major else (page * size + r) * P + t % P


def ref_tables(kv_len, new_len, head_group, G, P, tables, pages_in, free, free_in, token_major):
    """Sequential reading of kvx_build_tables' contract. Returns (tables, pages, free, free_count,
    q_start, slots); tables and free are copies with the call's writes."""
    kv, new = np.asarray(kv_len, np.int64), np.asarray(new_len, np.int64)
    B, Hkv = kv.shape
    tables = [t.copy() for t in tables]
    free = [f.copy() for f in free]
    pages, left = np.array(pages_in, np.int64), np.array(free_in, np.int64)
    rk = ranks(head_group)
    for g in range(G):
        hs = [h for h in range(Hkv) if head_group[h] == g]
        need = [-(-(int(kv[b, hs].max()) + int(new[b])) // P) for b in range(B)]
        for b in range(B):
            for j in range(need[b], int(pages[g, b])):
                free[g][left[g]] = tables[g][b, j]
                left[g] += 1
        for b in range(B):
            for j in range(int(pages[g, b]), need[b]):
                left[g] -= 1
                tables[g][b, j] = free[g][left[g]]
            pages[g, b] = need[b]
    q_start = np.concatenate([[0], np.cumsum(new)])
    slots = np.zeros((int(q_start[-1]), Hkv), np.int64)
    for b in range(B):
        for i in range(int(new[b])):
            for h in range(Hkv):
                g, t = head_group[h], int(kv[b, h]) + i
                slots[q_start[b] + i, h] = slot_of(int(tables[g][b, t // P]), rk[h], t,
                                                   list(head_group).count(g), P, token_major)
    return tables, pages, free, left, q_start, slots


@dataclass
class Case:
    dtype: str = "bf16"
    D: int = 128
    Hkv: int = 2
    g: int = 4
    groups: tuple = (0, 0)     # head group of each KV head
    P: int = 16
    token_major: bool = False
    kv: tuple = ((40, 7),)     # cached tokens [B][Hkv]
    T: tuple = (5,)            # new rows [B]
    mask: str = "tree"         # tree, chain (NULL), full, empty (some rows see nothing), self
    seed: int = 0
    fused: bool = False        # q as a slice of a wider row
    spread: float = 1.0        # standard deviation of q (large: peaked softmax)

    @property
    def name(self):
        return (f"{self.dtype}-D{self.D}-g{self.g}-P{self.P}-"
                f"{'tok' if self.token_major else 'head'}-kv{self.kv[0][0]}x{len(self.kv)}-"
                f"T{max(self.T)}-{self.mask}")


def to_dev(a, dtype):
    if dtype == "bf16":
        return torch.from_numpy(synth.f32_to_bf16_bits(a).view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def tree_parents(r, T):
    return [int(r.integers(-1, i)) if i else -1 for i in range(T)]


def visible(r, kind, T):
    """bool [T][T]: row i sees draft j."""
    v = np.zeros((T, T), bool)
    if kind == "full":
        v[:] = True
    elif kind == "chain":
        v = np.tril(np.ones((T, T), bool))
    elif kind == "self":
        v = np.eye(T, dtype=bool)
    else:
        par = tree_parents(r, T)
        for i in range(T):
            if par[i] >= 0:
                v[i] = v[par[i]]
            v[i, i] = True
        if kind == "empty":
            v[::3] = False
    return v


class Setup:
    def __init__(self, c: Case, spare=3, extra_rows=2, fill=float("nan")):
        self.c = c
        r = self.r = synth.rng(c.seed)
        kv = self.kv = np.array(c.kv, np.int64)
        self.B, self.Hkv, self.Hq = kv.shape[0], c.Hkv, c.Hkv * c.g
        T = self.T = np.array(c.T, np.int64)
        hg = self.hg = list(c.groups)
        G = self.G = max(hg) + 1
        self.rank, self.size = ranks(hg), [hg.count(g) for g in range(G)]
        P = c.P
        self.q_start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
        self.N = int(self.q_start[-1])
        self.max_rows = self.N + extra_rows
        self.max_q = max(1, int(T.max()))
        need = np.array([[-(-(int(kv[b, [h for h in range(c.Hkv) if hg[h] == g]].max()) + int(T[b])) // P)
                          for b in range(self.B)] for g in range(G)])
        self.need = need
        self.stride = [max(1, int(need[g].max())) for g in range(G)]
        self.pages = [int(need[g].sum()) + spare for g in range(G)]
        self.tables, self.k, self.v = [], [], []
        for g in range(G):
            ids = r.permutation(self.pages[g]).astype(np.int32)
            t = np.full((self.B, self.stride[g]), -1, np.int32)
            at = 0
            for b in range(self.B):
                t[b, :need[g, b]] = ids[at:at + need[g, b]]
                at += need[g, b]
            self.tables.append(t)
            rows = self.pages[g] * self.size[g] * P
            self.k.append(np.full((rows, c.D), fill, np.float32))
            self.v.append(np.full((rows, c.D), fill, np.float32))
        for b in range(self.B):
            for h in range(c.Hkv):
                at = self.rows_of(b, h, np.arange(int(kv[b, h] + T[b])))
                self.k[hg[h]][at] = synth.normal(r, (at.size, c.D), c.dtype)
                self.v[hg[h]][at] = synth.normal(r, (at.size, c.D), c.dtype)
        self.q = synth.round_to(c.spread * synth.normal(r, (self.max_rows, self.Hq, c.D), "f32"),
                                c.dtype)
        self.see = [visible(r, c.mask, int(t)) for t in T]
        self.scale = 1.0 / math.sqrt(c.D)

    def rows_of(self, b, h, t):
        g = self.hg[h]
        page = self.tables[g][b, t // self.c.P].astype(np.int64)
        return slot_of(page, self.rank[h], t, self.size[g], self.c.P, self.c.token_major)

    def slots(self):
        s = np.full((self.max_rows, self.Hkv), -1, np.int64)
        for b in range(self.B):
            for h in range(self.Hkv):
                t = self.kv[b, h] + np.arange(self.T[b])
                s[self.q_start[b]:self.q_start[b + 1], h] = self.rows_of(b, h, t)
        return s

    def words(self, max_q=None):
        """uint32 mask words [max_rows][W], bits past T random (they are ignored)."""
        W = ((max_q or self.max_q) + 31) // 32
        m = self.r.integers(0, 1 << 32, size=(self.max_rows, W), dtype=np.uint64)
        for b in range(self.B):
            for i in range(int(self.T[b])):
                row = self.q_start[b] + i
                for j in range(int(self.T[b])):
                    bit = np.uint64(1 << (j % 32))
                    m[row, j // 32] = (m[row, j // 32] | bit) if self.see[b][i, j] else \
                        (m[row, j // 32] & ~bit)
        return m.astype(np.uint32)

    # ---- device side
    def upload(self):
        c = self.c
        self.dk = [to_dev(a, c.dtype) for a in self.k]
        self.dv = [to_dev(a, c.dtype) for a in self.v]
        self.dt = [torch.from_numpy(t).cuda() for t in self.tables]
        self.cache = kvx.Cache(self.B, self.Hq, self.Hkv, c.D, c.P, self.G,
                               kvx.KVX_BF16 if c.dtype == "bf16" else kvx.KVX_F32, self.hg, self.dk,
                               self.dv, self.pages, self.dt, self.stride,
                               layout=kvx.KVX_LAYOUT_TOKEN_MAJOR if c.token_major
                               else kvx.KVX_LAYOUT_HEAD_MAJOR)
        self.dkv = torch.from_numpy(self.kv.astype(np.int32)).cuda()
        self.dqs = torch.from_numpy(self.q_start).cuda()
        self.dmask = None if c.mask == "chain" else \
            torch.from_numpy(self.words().view(np.int32)).cuda()
        if c.fused:
            wide = torch.full((self.max_rows, self.Hq * c.D + 24), float("nan"),
                              dtype=torch.bfloat16 if c.dtype == "bf16" else torch.float32,
                              device="cuda")
            self.dq = wide[:, 8:8 + self.Hq * c.D]
            self.dq.copy_(to_dev(self.q, c.dtype).view(self.max_rows, -1))
        else:
            self.dq = to_dev(self.q, c.dtype)
        self.out = torch.full((self.max_rows, self.Hq, c.D), -7.0, device="cuda")
        n = kvx.kvx_tree_attn_workspace_bytes(self.cache, min(self.max_q, kvx.KVX_MAX_TREE))
        self.ws = torch.zeros(-(-n // 4), dtype=torch.int32, device="cuda")
        return self

    def attend(self, stream=None, max_q=None):
        kvx.kvx_tree_attn(self.cache, self.dq, self.dqs, self.max_rows, max_q or self.max_q,
                          self.dkv, self.dmask, 0.0, self.out, self.ws, stream=stream)

    def run(self):
        self.attend()
        torch.cuda.synchronize()
        return self.out.cpu().numpy()

    def status(self):
        return kvx.kvx_workspace_status(self.ws)

    # ---- references
    def reference(self):
        """(out, tol) [N][Hq][D] in float64: the definition, and the bound on the library's error
        derived below."""
        c = self.c
        out = np.zeros((self.N, self.Hq, c.D))
        tol = np.zeros_like(out)
        for b in range(self.B):
            T = int(self.T[b])
            for h in range(self.Hkv):
                n = int(self.kv[b, h])
                at = self.rows_of(b, h, np.arange(n + T))
                k = self.k[self.hg[h]][at].astype(np.float64)
                v = self.v[self.hg[h]][at].astype(np.float64)
                for i in range(T):
                    see = np.concatenate([np.ones(n, bool), self.see[b][i]])
                    if not see.any():
                        continue
                    for j in range(c.g):
                        q = self.q[self.q_start[b] + i, h * c.g + j].astype(np.float64)
                        s = self.scale * (k[see] @ q)
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        row = self.q_start[b] + i, h * c.g + j
                        out[row] = p @ v[see]
                        mag = p @ np.abs(v[see])
                        tol[row] = error_bound(c, int(see.sum()), s, self.scale *
                                               float((np.abs(k[see]) @ np.abs(q)).max())) * mag
        return out, tol


def error_bound(c: Case, n, s, s_abs):
    """Bound on |out - exact| relative to sum_t p_t |v_t|, first order in the roundings.

    u = 2^-24 is half a step of fp32. The scores: D products and sums, each off by at
    most u (2u for tensor-core sums, which may truncate) of the sum of magnitudes s_abs;
    scaling to log2 units and subtracting the maximum: 3u of the largest |s - max| and of
    |s|. An error e of a score is a relative error e of its weight; the hardware exp2
    adds 2^-22. Weights enter the sum and the weighted sum, hence twice. bf16 caches: each
    weight is a bf16 high part and a bf16 residual, off by 2^-9 * 2^-9. Sums over n
    keys: 2u for each addition of a running sum (at most n + 64 with the merges), for the
    weighted sum and the normaliser.
    """
    u = 2.0 ** -24
    far = float(np.max(np.abs(s))) + float(np.max(s.max() - s))
    score = 2 * u * (c.D + 2) * s_abs + 3 * u * far
    weight = score + 2.0 ** -22
    split = 2.0 ** -18 if c.dtype == "bf16" else 0.0
    return 2 * weight + split + 2 * 2 * u * (n + 64) + 4 * u


def check(setup: Setup, got):
    """Largest |got - exact| / tol; rows past the last sequence must be as they were."""
    ref, tol = setup.reference()
    assert np.all(got[setup.N:] == -7.0)
    err = np.abs(got[:setup.N].astype(np.float64) - ref)
    assert np.all(np.isfinite(got[:setup.N]))
    bad = err > tol
    assert not bad.any(), (float(err.max()), np.argwhere(bad)[:4].tolist())
    return float(err.max(initial=0.0))
