"""Rows of 4-bit caches: quantised by the append, read back; and rows of the other types read back."""
import numpy as np
import pytest
import torch

import synth
from budget_cases import BCase, Budget, bf16, quantise, unpack_pool, values
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu


def special_rows(D, n, seed=0):
    """bf16 rows whose groups are ordinary, shifted, constant, tiny, huge, subnormal, full of exact halves of
    a step, or hold NaN and infinities."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, D)).astype(np.float32)
    for i in range(n):
        kind = i % 12
        g = x[i].reshape(-1, 64)
        if kind == 1:
            g += 40
        elif kind == 2:
            g[:] = r.standard_normal()
        elif kind == 3:
            g *= 2.0 ** -100
        elif kind == 4:
            g *= 2.0 ** 120
        elif kind == 5:
            g *= 2.0 ** -131
        elif kind == 6:  # steps of 1, values on quarters
            g[:] = r.integers(0, 61, g.shape) / 4
            g[:, :2] = 0, 15
        elif kind == 7:
            g[0, 5] = np.nan
        elif kind == 8:
            g[-1, 9] = np.inf
        elif kind == 9:
            g[:, 3], g[:, 4] = 3e38, -3e38
        elif kind == 10:
            g[:] = np.where(r.random(g.shape) < 0.5, 0.0, -0.0)
        elif kind == 11:
            g[:, ::3] *= 1e-6
    return bf16(x)


@pytest.mark.parametrize("D,P", [(128, 16), (64, 8), (128, 128), (64, 64)])
def test_append_and_read(D, P):
    c = BCase("bf16", D, 3, 2, (0, 1, 0), kv=((40, 7, 0), (5, 9, 100)), T=(60, 37), q4=True, P=P)
    s = Budget(c).upload()
    rows = [special_rows(D, s.max_rows * 3, seed).reshape(s.max_rows, 3, D) for seed in (1, 2)]
    dk, dv = (torch.from_numpy(synth.f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16).cuda() for x in rows)
    wide = torch.zeros((s.max_rows, 3 * D + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, :3 * D] = dk.view(s.max_rows, -1)
    slots = s.slots()
    slots[3, 1] = -1
    dslots = torch.from_numpy(slots).cuda()
    kvx.kvx_append_kv(s.cache, wide[:, :3 * D], dv, s.dqs, dslots, s.max_rows, s.ws)
    ko, vo = (torch.full((s.max_rows, 3, D), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kvx.kvx_read_kv(s.cache, s.dqs, dslots, s.max_rows, ko, vo, s.ws)
    torch.cuda.synchronize()
    assert s.status() == 0
    live = (np.arange(s.max_rows) < s.N)[:, None] & (slots >= 0)
    for x, before, pool, out in ((rows[0], s.bk, s.dk, ko), (rows[1], s.bv, s.dv, vo)):
        want = [unpack_pool(b, D, P) for b in before]
        codes, step, lo = quantise(x)
        for h in range(3):
            at, sel = slots[live[:, h], h], live[:, h]
            for a, new in zip(want[s.hg[h]], (codes, step, lo)):
                a[at] = new[sel, h]
        for g, (wc, ws, wl) in enumerate(want):
            gc, gs, gl = unpack_pool(pool[g].cpu().numpy(), D, P)
            assert np.array_equal(gc, wc)
            assert np.array_equal(gs, ws, equal_nan=True) and np.array_equal(gl, wl, equal_nan=True)
        with np.errstate(invalid="ignore", over="ignore"):
            ref = np.where(live[..., None], bf16(values(codes, step, lo).astype(np.float32)), np.float32(-7.0))
        got = out.float().cpu().numpy()
        assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("dtype,D,tok", [("bf16", 128, False), ("bf16", 64, True), ("f32", 128, True), ("f32", 64, False)])
def test_read_of_other_types(dtype, D, tok):
    c = BCase(dtype, D, 2, 2, (0, 1), kv=((40, 7), (5, 9)), T=(6, 3), token_major=tok)
    s = Budget(c).upload()
    slots = s.slots()
    slots[2, 0], slots[4, 1] = -1, s.pages[1] * s.size[1] * c.P
    out = [torch.full((s.max_rows, 2 * D + 8), -7.0, dtype=s.dk[0].dtype, device="cuda") for _ in range(2)]
    kvx.kvx_read_kv(s.cache, s.dqs, torch.from_numpy(slots).cuda(), s.max_rows, *(o[:, :2 * D] for o in out), s.ws)
    torch.cuda.synchronize()
    assert s.status() == kvx.KVX_DEV_BAD_BLOCK
    slots[4, 1] = -1
    for o, pools in zip(out, (s.k, s.v)):
        ref = np.full((s.max_rows, 2, D), -7.0, np.float32)
        for h in range(2):
            ok = (np.arange(s.max_rows) < s.N) & (slots[:, h] >= 0)
            ref[ok, h] = pools[s.hg[h]][slots[ok, h]]
        assert np.array_equal(o[:, :2 * D].float().cpu().numpy().reshape(ref.shape), ref)
        assert (o[:, 2 * D:] == -7).all()


def test_rows_past_the_buffers():
    c = BCase("bf16", 128, 1, 2, (0,), kv=((4,),), T=(5,), q4=True)
    s = Budget(c).upload()
    s.dqs[1] = s.max_rows + 1
    dslots = torch.from_numpy(s.slots()).cuda()
    x = torch.zeros((s.max_rows, 128), dtype=torch.bfloat16, device="cuda")
    kvx.kvx_append_kv(s.cache, x, x, s.dqs, dslots, s.max_rows, s.ws)
    assert s.status() == kvx.KVX_DEV_BAD_LENGTH
    kvx.kvx_append_kv(s.cache, None, None, s.dqs, None, 0, s.ws)
    kvx.kvx_read_kv(s.cache, s.dqs, None, 0, None, None, s.ws)
    torch.cuda.synchronize()
