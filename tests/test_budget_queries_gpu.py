"""Windowed attention with queries and scales at the ends of their ranges."""
import numpy as np
import pytest
import torch

from budget_cases import BCase, Budget, pack_pool, quantise
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu

KINDS = [("bf16", False), ("f32", False), ("bf16", True)]


def run(s, scale):
    s.scale = scale or s.scale
    s.upload()
    kvx.kvx_window_attn(s.cache, s.dq, s.dqs, s.max_rows, s.max_q, s.dkv, s.dsinks, s.dwindow, scale, s.out, s.dw,
                        s.ws)
    torch.cuda.synchronize()
    assert s.status() == 0
    s.check(s.out.cpu().numpy(), s.dw)


@pytest.mark.parametrize("dtype,q4", KINDS)
@pytest.mark.parametrize("T,g", [(1, 4), (3, 5)])
@pytest.mark.parametrize("scale", [0.0, 1e-8, 1e-30, 2.0 ** -126, 1e-44])
def test_rows_of_zeros_weigh_all_alike(dtype, q4, T, g, scale):
    """Zero rows, and rows of the smallest numbers, beside ordinary ones; tiles that the rows see in part."""
    s = Budget(BCase(dtype, 128, 1, g, (0,), kv=((300,),), T=(T,), sinks=(3,), window=(150,), q4=q4, seed=11))
    s.q[:, 0] = 0
    s.q[:, 1] *= np.float32(2.0 ** -120)
    if T > 1:
        s.q[1] = 0
    run(s, scale)


@pytest.mark.parametrize("dtype,q4", KINDS)
def test_small_queries_at_a_large_scale(dtype, q4):
    """2^-110 * 2^70 * 2^38: scores of a few units, which the queries' own range must not lose."""
    c = BCase(dtype, 128, 1, 4, (0,), kv=((200,),), T=(2,), sinks=(3,), window=(150,), q4=q4, seed=12)
    s = Budget(c)
    s.q = s.q * np.float32(2.0 ** -110)
    s.k = [k * np.float32(2.0 ** 70) for k in s.k]
    if q4:
        s.qk = [quantise(np.nan_to_num(k)) for k in s.k]
        s.bk = [pack_pool(*a, c.P) for a in s.qk]
    run(s, 2.0 ** 38)
