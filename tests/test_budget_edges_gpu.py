"""Windowed attention and eviction where numbers or surroundings are unusual: scores of any size, a second
CUDA context of the same device."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from budget_cases import BCase, Budget
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
KINDS = [("bf16", False), ("f32", False), ("bf16", True)]


def large(dtype, q4, T, g, sign):
    """Queries times 2^40: every row's weight is on its largest score, to the last bit."""
    s = Budget(BCase(dtype, 128, 1, g, (0,), kv=((300,),), T=(T,), sinks=(3,), window=(150,), q4=q4, seed=7))
    s.q = s.q * np.float32(sign * 2.0 ** 40)
    out, _, w, _ = s.reference()
    # the second largest score is far enough behind, beside fp32 sums of 130 products
    at = s.rows_of(0, 0, np.arange(300 + T))
    k, _, km, _ = s.kv_values(0, at)
    for i in range(T):
        see = s.sees(0, 0, i)
        for j in range(g):
            q = s.q[s.q_start[0] + i, j].astype(np.float64)
            x = np.sort(s.scale * (k[see] @ q))
            assert x[-1] - x[-2] > 300 + 2 * 2.0 ** -24 * 130 * s.scale * (km[see] @ np.abs(q)).max()
    return s, out, w


@pytest.mark.parametrize("dtype,q4", KINDS)
@pytest.mark.parametrize("T,g,sign", [(1, 4, 1), (1, 4, -1), (3, 5, 1)])
def test_large_scores_choose_one_token(dtype, q4, T, g, sign):
    s, out, w = large(dtype, q4, T, g, sign)
    s.upload()
    got = s.run(weigh=True)[:s.N]
    # one weight of 1: what is left are the roundings of 4-bit values (2^-22 of 15 steps) and of the output
    top = np.abs(s.kv_values(0, s.rows_of(0, 0, np.arange(300 + T)))[3]).max()
    assert np.all(np.abs(got - out) <= 2.0 ** -20 * top)
    for a, b in zip(s.dw, w):
        assert np.all(np.abs(a.cpu().numpy() - b) <= 2.0 ** -22 * (1 + np.abs(b)))
    assert s.status() == 0


@pytest.mark.parametrize("dtype,q4", KINDS)
def test_scores_next_to_the_lowest_number(dtype, q4):
    """All scores are -1.8 * 2^127, in powers of two: equal weights, the output is the mean of V."""
    n = 70
    c = BCase(dtype, 128, 1, 4, (0,), kv=((n,),), T=(1,), seed=5)
    s = Budget(c)
    for a in s.k:
        a[:] = 0
        a[:, 0] = -1.796875 * 2.0 ** 63
    s.q[:] = 0
    s.q[:, :, 0] = 2.0 ** 64
    if q4:  # made again, from the changed rows
        keep_k, keep_v, keep_q = s.k, s.v, s.q
        s = Budget(BCase(dtype, 128, 1, 4, (0,), kv=((n,),), T=(1,), seed=5, q4=True))
        from budget_cases import pack_pool, quantise
        s.q = keep_q
        s.qk = [quantise(a) for a in keep_k]
        s.bk = [pack_pool(*a, c.P) for a in s.qk]
    s.upload()
    kvx.kvx_window_attn(s.cache, s.dq, s.dqs, s.max_rows, s.max_q, s.dkv, None, None, 0.6931472, s.out, None, s.ws)
    torch.cuda.synchronize()
    _, v, _, vm = s.kv_values(0, s.rows_of(0, 0, np.arange(n + 1)))
    # weights are equal to the bit; sums of n + 1 terms and parts of at least 22 bits remain
    tol = (2.0 ** -22 + 2 * (n + 64) * 2.0 ** -24) * vm.mean(0)
    assert np.all(np.abs(s.out.cpu().numpy()[0] - v.mean(0)) <= tol)


CHILD = '''
import ctypes, sys
import numpy as np, torch
sys.path[:0] = [{here!r}, {root!r}]
from paged_non_uniform_gb300 import kvx
from budget_cases import BCase, Budget

cuda = ctypes.CDLL("libcuda.so.1")
def ok(rc):
    assert rc == 0, rc

s = Budget(BCase({dtype!r}, {D}, 2, 4, (0, 0), kv=((900, 40), (7, 300)), T=({T}, 2), sinks=(3, 0), window=(200, 50),
                 q4={q4}, seed=3)).upload()
case = s.c
kind = kvx.KVX_Q4 if {q4} else kvx.KVX_BF16 if {dtype!r} == "bf16" else kvx.KVX_F32
budget = torch.tensor([[100, 30], [9, 128]], dtype=torch.int32, device="cuda")
ws2 = torch.zeros(kvx.kvx_evict_workspace_bytes(s.cache), dtype=torch.uint8, device="cuda")
host = [t.detach().cpu().contiguous() for t in (s.dk[0], s.dv[0], s.dt[0], s.dkv, s.dqs, s.dsinks, s.dwindow, s.dw[0],
                                                s.dq, budget, s.out, s.ws, ws2)]
want = s.run(weigh=True)              # in the context that torch uses
kvx.kvx_evict(s.cache, s.dkv, budget, 2, 5, s.dw, s.dw, s.dkv, ws2)
torch.cuda.synchronize()
bits = lambda t: t.detach().cpu().contiguous().view(torch.uint8).numpy()
after = [bits(t) for t in (s.dk[0], s.dv[0], s.dw[0], s.dkv)]

ctx = ctypes.c_void_p()
ok(cuda.cuCtxCreate_v2(ctypes.byref(ctx), 0, torch.cuda.current_device()))
at = []
for t in host:
    p = ctypes.c_uint64()
    ok(cuda.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(t.nbytes)))
    ok(cuda.cuMemcpyHtoD_v2(p, ctypes.c_void_p(t.data_ptr()), ctypes.c_size_t(t.nbytes)))
    at.append(p.value)
k, v, table, kv, qs, sinks, window, w, q, bud, out, ws, wse = at
cache = kvx.Cache(2, s.Hq, 2, {D}, case.P, 1, kind, [0, 0], [k], [v], s.pages, [table], s.stride)
kvx.kvx_window_attn(cache, q, qs, s.max_rows, s.max_q, kv, sinks, window, 0.0, out, [w], ws, host[11].nbytes, stream=0)
kvx.kvx_evict(cache, kv, bud, 2, 5, [w], [w], kv, wse, host[12].nbytes, stream=0)
ok(cuda.cuCtxSynchronize())
def back(a, t):
    got = torch.empty_like(t)
    ok(cuda.cuMemcpyDtoH_v2(ctypes.c_void_p(got.data_ptr()), ctypes.c_uint64(a), ctypes.c_size_t(got.nbytes)))
    return got
assert np.array_equal(back(out, host[10]).numpy(), want)
for a, t, b in zip((k, v, w, kv), (host[0], host[1], host[7], host[3]), after):
    assert np.array_equal(bits(back(a, t)), b)
ok(cuda.cuCtxDestroy_v2(ctx))
print("same bits")
'''


@pytest.mark.parametrize("dtype,D,T,q4", [("bf16", 128, 1, False), ("bf16", 64, 8, False), ("f32", 128, 2, False),
                                          ("bf16", 128, 1, True)])
def test_calls_in_a_second_context(dtype, D, T, q4):
    code = CHILD.format(here=HERE, root=os.path.dirname(HERE), dtype=dtype, D=D, T=T, q4=q4)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr
