"""What the memory-budget calls leave behind when a wait runs out (the library's own hook, with short limits)."""
import numpy as np
import pytest
import torch

from budget_cases import BCase, Budget
from paged_non_uniform_gb300 import kvx

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
