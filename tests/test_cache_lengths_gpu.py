"""What the cache calls make of lengths out of range, and how they report them."""
import numpy as np
import pytest
import torch

from paged_non_uniform_gb300 import kvx
from tree_cases import Case, Setup

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("end,rows,status", [(4, 4, 0), (3, 3, 0), (0, 0, 0), (-1, 0, kvx.KVX_DEV_BAD_LENGTH),
                                             (-2 ** 31, 0, kvx.KVX_DEV_BAD_LENGTH),
                                             (5, 4, kvx.KVX_DEV_BAD_LENGTH),
                                             (2 ** 31 - 1, 4, kvx.KVX_DEV_BAD_LENGTH)])
def test_append_reports_a_row_count_out_of_range(end, rows, status):
    s = Setup(Case(kv=((40, 7),), T=(4,)), extra_rows=0).upload()
    new = torch.ones(4, 2 * 128, dtype=torch.bfloat16, device="cuda")
    want = [bits(x[0]).clone() for x in (s.dk, s.dv)]
    slots = s.slots()
    at = dev(slots[:rows].reshape(-1))
    one = int(bits(new)[0, 0])
    for w in want:
        w[at] = one
    kvx.kvx_append_kv(s.cache, new, new, torch.tensor([0, end], dtype=torch.int32, device="cuda"), dev(slots),
                      4, s.ws)
    torch.cuda.synchronize()
    assert s.status() == status
    for x, w in zip((s.dk, s.dv), want):
        assert torch.equal(bits(x[0]), w)
