"""Calls in a second CUDA context of the same device: what a kernel needs set once is set in each."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = '''
import ctypes, sys
import numpy as np, torch
sys.path[:0] = [{here!r}, {root!r}]
from paged_non_uniform_gb300 import kvx
from tree_cases import Case, Setup

cuda = ctypes.CDLL("libcuda.so.1")
def ok(rc):
    assert rc == 0, rc

s = Setup(Case({dtype!r}, {D}, 2, 4, (0, 0), kv=((900, 40), (7, 300)), T=(5, 9), seed=3)).upload()
case = s.c
want = s.run()                       # in the context that torch uses
host = [t.detach().cpu().contiguous() for t in (s.dk[0], s.dv[0], s.dt[0], s.dkv, s.dqs, s.dmask, s.dq,
                                                torch.full_like(s.out, -7.0), torch.zeros_like(s.ws))]

ctx = ctypes.c_void_p()
ok(cuda.cuCtxCreate_v2(ctypes.byref(ctx), 0, torch.cuda.current_device()))
at = []
for t in host:
    p = ctypes.c_uint64()
    ok(cuda.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(t.nbytes)))
    ok(cuda.cuMemcpyHtoD_v2(p, ctypes.c_void_p(t.data_ptr()), ctypes.c_size_t(t.nbytes)))
    at.append(p.value)
k, v, table, kv, qs, mask, q, out, ws = at
cache = kvx.Cache(2, s.Hq, 2, {D}, 16, 1, kvx.KVX_BF16 if {dtype!r} == "bf16" else kvx.KVX_F32, [0, 0], [k], [v],
                  s.pages, [table], s.stride)
for _ in range(2):
    kvx.kvx_tree_attn(cache, q, qs, s.max_rows, s.max_q, kv, mask, 0.0, out, ws, host[8].nbytes, stream=0)
ok(cuda.cuCtxSynchronize())
got = torch.empty_like(host[7])
ok(cuda.cuMemcpyDtoH_v2(ctypes.c_void_p(got.data_ptr()), ctypes.c_uint64(out), ctypes.c_size_t(got.nbytes)))
assert np.array_equal(got.numpy(), want)
ok(cuda.cuCtxDestroy_v2(ctx))
s.out.fill_(-7.0)
assert np.array_equal(s.run(), want)  # and back
print("same bits")
'''


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_attention_in_a_second_context(dtype, D):
    code = CHILD.format(here=HERE, root=os.path.dirname(HERE), dtype=dtype, D=D)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr
