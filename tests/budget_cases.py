"""Inputs and plain 64-bit references for the calls that keep a paged cache within a memory budget:
attention with windows, sinks and accumulated weights, eviction, 4-bit caches.

Test infrastructure only; a `Budget` is a `Setup` of tree_cases (pools with NaN in unused slots) with windows,
weight pools and, for "q4", pools in the library's 4-bit page format, made by NumPy.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

import synth
from paged_non_uniform_gb300 import kvx
from tree_cases import Case, Setup

ALL = 2 ** 31 - 1


@dataclass
class BCase(Case):
    mask: str = "chain"
    sinks: tuple = ()     # per KV head, () : NULL
    window: tuple = ()    # per KV head, () : NULL
    q4: bool = False

    @property
    def name(self):
        return (f"{'q4' if self.q4 else self.dtype}-D{self.D}-g{self.g}-P{self.P}-"
                f"{'tok' if self.token_major else 'head'}-kv{self.kv[0][0]}x{len(self.kv)}-T{max(self.T)}-"
                f"s{self.sinks}-w{self.window}").replace(" ", "")


def bf16(x):
    """float32 rounded to bf16 (nearest even; no NaN handling needed here)."""
    with np.errstate(invalid="ignore", over="ignore"):
        return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(x, np.float32)))


def quantise(x):
    """The header's rule in float32: codes uint8 [..., D], step and lo float32 [..., D / 64]."""
    x = np.asarray(x, np.float32)
    f = x.reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    with np.errstate(all="ignore"):
        lo, hi = f.min(-1), f.max(-1)
        rng = (hi - lo).astype(np.float32)
        bad = ~np.isfinite(rng)
        step = bf16(np.where(bad, 0, rng / np.float32(15)))
        c = np.rint((f - lo[..., None]) / step[..., None])
        c = np.where((step == 0)[..., None], 0, np.minimum(c, 15)).astype(np.uint8)
    return c.reshape(x.shape), step, np.where(bad, np.float32(np.nan), lo).astype(np.float32)


def values(codes, step, lo):
    """lo + step * code in float64 (exact)."""
    c = codes.reshape(codes.shape[:-1] + (codes.shape[-1] // 64, 64)).astype(np.float64)
    return (lo[..., None].astype(np.float64) + step[..., None].astype(np.float64) * c).reshape(codes.shape)


def pack_pool(codes, step, lo, P):
    """Pool bytes of rows [N][D] in row order: per block of P rows the codes, then {step, lo}."""
    N, D = codes.shape
    w = codes.reshape(N, D // 8, 8).astype(np.uint32)
    words = sum(w[:, :, i] << np.uint32(4 * i) for i in range(8)).astype("<u4")
    place = [2 * (j % 8) + j // 8 if D == 128 else j for j in range(D // 8)]
    stored = np.empty_like(words)
    stored[:, place] = words
    par = np.stack([synth.f32_to_bf16_bits(step), synth.f32_to_bf16_bits(lo)], -1).astype("<u2")
    code_bytes = stored.view(np.uint8).reshape(N // P, P * (D // 2))
    par_bytes = par.reshape(N, -1).view(np.uint8).reshape(N // P, P * (D // 16))
    return np.concatenate([code_bytes, par_bytes], 1).reshape(-1)


def unpack_pool(buf, D, P):
    """(codes, step, lo) of all rows of a pool's bytes."""
    b = buf.reshape(-1, P * (D // 2 + D // 16))
    N = b.shape[0] * P
    stored = np.ascontiguousarray(b[:, :P * D // 2]).reshape(N, -1).view("<u4")
    place = [2 * (j % 8) + j // 8 if D == 128 else j for j in range(D // 8)]
    words = stored[:, place]
    codes = np.stack([(words >> np.uint32(4 * i)) & 15 for i in range(8)], -1).reshape(N, D).astype(np.uint8)
    par = synth.bf16_bits_to_f32(np.ascontiguousarray(b[:, P * D // 2:]).reshape(N, -1).view("<u2"))
    par = par.reshape(N, -1, 2)
    return codes, par[..., 0], par[..., 1]


class Budget(Setup):
    def __init__(self, c: BCase, spare=3, extra_rows=2, junk=False):
        super().__init__(c, spare, extra_rows)
        r = np.random.default_rng(c.seed + 1)
        self.w = [r.random(k.shape[0]).astype(np.float32) for k in self.k]
        self.sinks = np.array(c.sinks or [0] * c.Hkv, np.int64)
        self.window = np.array(c.window or [ALL] * c.Hkv, np.int64)
        if c.q4:
            self.qk = [quantise(np.nan_to_num(a)) for a in self.k]
            self.qv = [quantise(np.nan_to_num(a)) for a in self.v]
            self.bk = [pack_pool(*a, c.P) for a in self.qk]
            self.bv = [pack_pool(*a, c.P) for a in self.qv]
            used = [np.zeros(a.shape[0], bool) for a in self.k]
            for b in range(self.B):
                for h in range(c.Hkv):
                    used[self.hg[h]][self.rows_of(b, h, np.arange(int(self.kv[b, h] + self.T[b])))] = True
            for a, (codes, step, lo), u in ((p, q, u) for ps, qs in ((self.bk, self.qk), (self.bv, self.qv))
                                            for p, q, u in zip(ps, qs, used)):
                self.spoil(a, ~u)

    def spoil(self, buf, rows):
        """Fills the parameters of rows of a 4-bit pool with NaN and their codes with ones."""
        c = self.c
        b = buf.reshape(-1, c.P * (c.D // 2 + c.D // 16))
        blk, off = np.nonzero(np.asarray(rows).reshape(-1, c.P))
        for i, o in zip(blk, off):
            b[i, o * c.D // 2:(o + 1) * c.D // 2] = 0xff
            at = c.P * c.D // 2 + o * c.D // 16
            b[i, at:at + c.D // 16] = 0xff

    def kv_values(self, h, at):
        """K and V rows as attention sees them, float64, and the magnitudes that their sums pass through."""
        g = self.hg[h]
        if not self.c.q4:
            k, v = self.k[g][at].astype(np.float64), self.v[g][at].astype(np.float64)
            return k, v, np.abs(k), np.abs(v)
        out, mags = [], []
        for codes, step, lo in (self.qk[g], self.qv[g]):
            s, l = (np.repeat(a[at].astype(np.float64), 64, -1) for a in (step, lo))
            out.append(l + s * codes[at])
            mags.append((s, l))
        (sk, lk), (sv, lv) = mags
        return out[0], out[1], np.abs(lk) + 23 * sk, 7.5 * sv + np.abs(lv + 7.5 * sv)

    def upload(self):
        c = self.c
        super().upload()
        if c.q4:
            self.dk, self.dv = ([torch.from_numpy(a.copy()).cuda() for a in p] for p in (self.bk, self.bv))
            self.cache = kvx.Cache(self.B, self.Hq, self.Hkv, c.D, c.P, self.G, kvx.KVX_Q4, self.hg, self.dk,
                                   self.dv, self.pages, self.dt, self.stride)
        self.dw = [torch.from_numpy(a).cuda() for a in self.w]

        def small(x):
            return torch.from_numpy(np.array(x, np.int32)).cuda() if x else None

        self.dsinks, self.dwindow = small(c.sinks), small(c.window)
        n = kvx.kvx_window_attn_workspace_bytes(self.cache, min(self.max_q, kvx.KVX_MAX_TREE), True)
        self.ws = torch.zeros(-(-n // 4), dtype=torch.int32, device="cuda")
        return self

    def attend(self, stream=None, max_q=None, weigh=False):
        kvx.kvx_window_attn(self.cache, self.dq, self.dqs, self.max_rows, max_q or self.max_q, self.dkv,
                            self.dsinks, self.dwindow, 0.0, self.out, self.dw if weigh else None, self.ws,
                            stream=stream)

    def run(self, weigh=False):
        self.attend(weigh=weigh)
        torch.cuda.synchronize()
        return self.out.cpu().numpy()

    def sees(self, b, h, i):
        n, T = int(self.kv[b, h]), int(self.T[b])
        t, pos = np.arange(n + T), n + i
        return (t <= pos) & ((t < max(0, self.sinks[h])) | (t > pos - max(0, self.window[h])))

    def reference(self):
        """out, tol [N][Hq][D] and weights, tolerances (per group), float64."""
        c = self.c
        out, tol = np.zeros((self.N, self.Hq, c.D)), np.zeros((self.N, self.Hq, c.D))
        w = [a.astype(np.float64) for a in self.w]
        wt = [np.zeros_like(a) for a in w]
        for b in range(self.B):
            T = int(self.T[b])
            for h in range(self.Hkv):
                n = int(self.kv[b, h])
                at = self.rows_of(b, h, np.arange(n + T))
                k, v, km, vm = self.kv_values(h, at)
                acc, err = np.zeros(n + T), np.zeros(n + T)
                for i in range(T):
                    see = self.sees(b, h, i)
                    if not see.any():
                        continue
                    for j in range(c.g):
                        q = self.q[self.q_start[b] + i, h * c.g + j].astype(np.float64)
                        s = self.scale * (k[see] @ q)
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        rel = bound(c, int(see.sum()), s, self.scale * float((km[see] @ np.abs(q)).max()))
                        row = self.q_start[b] + i, h * c.g + j
                        out[row] = p @ v[see]
                        tol[row] = rel * (p @ vm[see])
                        acc[see] += p
                        err[see] += rel * p
                if T:
                    g = self.hg[h]
                    w[g][at[n:]] = 0
                    w[g][at] += acc
                    wt[g][at] = err + 2.0 ** -24 * (T * c.g + 2) * (np.abs(w[g][at]) + acc)
        return out, tol, w, wt

    def check(self, got, weights=None):
        ref, tol, w, wt = self.reference()
        assert np.all(got[self.N:] == -7.0)
        assert np.all(np.isfinite(got[:self.N]))
        err = np.abs(got[:self.N].astype(np.float64) - ref)
        assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(err > tol)[:4].tolist())
        if weights is not None:
            for g, a in enumerate(weights):
                e = np.abs(a.cpu().numpy().astype(np.float64) - w[g])
                assert np.all(e <= wt[g]), (g, float((e - wt[g]).max()), np.argwhere(e > wt[g])[:4].tolist())


def bound(c: BCase, n, s, s_abs):
    """Bound on |out - exact| relative to sum_t p_t |v_t|, as tree_cases.error_bound derives it, but for the
    weights' parts: three bf16 parts leave (2^-9)^3 = 2^-27 of a weight. Two fp16 parts leave 2^-11 * 2^-11
    = 2^-22; below fp16's normal range a part is off by 2^-25 in units in which the largest step times weight 1
    is at least 2^11, that is by 2^-36 of the largest term for each of n tokens. s_abs and the magnitudes of
    V are those that the sums pass through (`kv_values`); two more roundings per group of 64 elements in
    the scores (step * sum, lo * sum) are within the D + 2 of the bound."""
    u = 2.0 ** -24
    far = float(np.max(np.abs(s))) + float(np.max(s.max() - s))
    score = 2 * u * (c.D + 2) * s_abs + 3 * u * far
    weight = score + 2.0 ** -22
    split = 2.0 ** -22 + n * 2.0 ** -36 if c.q4 else 2.0 ** -27 if c.dtype == "bf16" else 0.0
    return 2 * weight + split + 2 * 2 * u * (n + 64) + 4 * u


# ---------------------------------------------------------------- eviction
def ref_evict(w, n, budget, sinks, recent):
    """Old indices of the tokens that stay, in order. w: the head's weights in token order."""
    m = min(n, budget)
    if m == n:
        return np.arange(n)
    r = min(m, recent)
    f = min(m - r, sinks)
    mid = np.asarray(w[f:n - r], np.float64)
    key = np.where(np.isnan(mid), -np.inf, mid)
    order = np.lexsort((np.arange(mid.size), np.isnan(mid), -key))  # NaN after -inf
    best = np.sort(order[:m - r - f]) + f
    return np.concatenate([np.arange(f), best, np.arange(n - r, n)]).astype(np.int64)
