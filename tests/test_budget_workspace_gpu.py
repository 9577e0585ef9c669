"""The workspace of weighing attention: what the header says that it takes."""
import pytest

from budget_cases import BCase, Budget
from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,q4", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("g,max_q", [(1, 1), (4, 1), (5, 1), (5, 7), (3, 4), (4, 32), (8, 128), (7, 2)])
def test_scores_take_what_the_header_says(dtype, q4, g, max_q):
    s = Budget(BCase(dtype, 64, 3, g, (0, 1, 1), kv=((900, 30, 3), (5, 70, 60)), T=(1, 1), q4=q4)).upload()
    most = 32 if dtype == "f32" else next((r for r in (4, 8, 16) if r >= max_q * g), 16 if q4 else 32)
    T = most // g
    rows = -(-min(T, max_q) * g // 4) * 4
    room = -(-max(s.stride) * s.c.P // 64) * 64
    scores = 4 * -(-max_q // T) * rows * room * 2 * 3
    row_ml = 8 * 2 * max_q * 3 * g
    plain, weigh = (kvx.kvx_window_attn_workspace_bytes(s.cache, max_q, w) for w in (False, True))
    # three arrays, each rounded up to 256 bytes; the small one has a number a block (at most three an SM)
    assert 0 <= weigh - plain - scores - row_ml <= 3 * 256 + 4 * 3 * 160
