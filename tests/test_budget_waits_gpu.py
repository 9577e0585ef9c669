"""What the memory-budget calls leave behind when a wait runs out (the library's own hook, with short limits)."""
import numpy as np
import pytest
import torch

from budget_cases import BCase, Budget, ref_evict, unpack_pool
from paged_non_uniform_gb300 import kvx
from test_evict_gpu import Evict

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,q4,T", [("bf16", False, 1), ("bf16", False, 9), ("bf16", True, 1)])
def test_weights_stay_when_attention_gives_up(dtype, q4, T):
    s = Budget(BCase(dtype, 128, 1, 4, (0,), kv=((500,),), T=(T,), q4=q4)).upload()
    # scores of an earlier call that no sum may show
    n = kvx.kvx_window_attn_workspace_bytes(s.cache, s.max_q, False) // 4
    s.ws[n:].view(torch.float32).fill_(1e30)
    s.cache.inject_stall(1, 5_000_000)
    s.attend(weigh=True)
    torch.cuda.synchronize()
    assert s.status() & kvx.KVX_DEV_TIMEOUT
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(s.dw, s.w))
    s.cache.inject_stall(-1, 2_000_000_000)
    s.ws.zero_()
    s.check(s.run(weigh=True), s.dw)
    assert s.status() == 0


@pytest.mark.parametrize("dtype,q4,in_place", [("bf16", False, True), ("f32", False, False), ("bf16", True, True)])
def test_eviction_that_gives_up_leaves_out_only_what_it_waited_for(dtype, q4, in_place):
    """One long head of 313 units (64 places each) and, with empty heads between, short ones of one unit, which
    waits for nobody. Block 0 does not say that it has read its first unit, one of the long head's: some of that head's
    units stay unwritten, whole, and nothing else does. (The head's last unit nobody waits for.)"""
    D, P, sinks, recent = 64, 64, 4, 16
    kv = ((40000, 0, 0, 0),) + ((0,) * 4,) * 155 + ((100, 70, 300, 65),) * 100
    budget = ((20000, 40, 50, 64),) + ((64, 60, 33, 1),) * 255
    s = Evict(BCase(dtype, D, 4, 1, (0, 1, 1, 1), kv=kv, T=(0,) * 256, q4=q4, P=P), budget)
    s.upload()

    def contents(w):
        """K, V and weight of every row, as numbers."""
        out = []
        for g in range(s.G):
            if q4:
                kv = [np.concatenate(unpack_pool(p[g].cpu().numpy(), D, P), 1) for p in (s.dk, s.dv)]
            else:
                kv = [p[g].double().cpu().numpy() for p in (s.dk, s.dv)]
            out.append(np.concatenate(kv + [w[g].double().cpu().numpy()[:, None]], 1))
        return out

    w = s.dw if in_place else s.dout
    before = contents(w)
    s.cache.inject_stall(0, 20_000_000)
    s.evict(sinks, recent, in_place)
    torch.cuda.synchronize()
    s.cache.inject_stall(-1, 2_000_000_000)
    status = kvx.kvx_workspace_status(s.ews)
    assert status in (0, kvx.KVX_DEV_TIMEOUT)
    assert np.array_equal(s.kv_out.cpu().numpy(), np.minimum(kv, budget))
    after = contents(w)
    for b in range(256):
        for h in range(4):
            n, m, g = kv[b][h], min(kv[b][h], budget[b][h]), s.hg[h]
            at = s.rows_of(b, h, np.arange(n))
            keep = ref_evict(s.w[g][at], n, m, sinks, recent)
            want, was, got = before[g][at[keep]], before[g][at[:m]], after[g][at[:m]]
            if not in_place:  # (copied weights wait for nothing)
                want[:, -1] = was[:, -1] = s.w[g][at[keep]]
            left = [c for c in range(0, m, 64) if not np.array_equal(got[c:c + 64], want[c:c + 64], equal_nan=True)]
            assert not left or (b, h) == (0, 0), (b, h, left)
            assert bool(left) == bool(status) or (b, h) != (0, 0)
            for c in left:
                assert np.array_equal(got[c:c + 64], was[c:c + 64], equal_nan=True)
            assert np.array_equal(after[g][at[m:]], before[g][at[m:]], equal_nan=True)
