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


@pytest.mark.parametrize("dtype,D,Hkv", [("bf16", 128, 20), ("f32", 64, 5), ("f32", 128, 9), ("bf16", 64, 33)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_keeps_heads_whose_length_is_out_of_range(dtype, D, Hkv, in_place):
    """Negative lengths and lengths that do not fit the page table with the new rows keep their rows and
    come back as they are; the sequence's other heads, in the same and in other blocks, move on. Lengths
    that just fit are good."""
    groups = tuple(h % 3 for h in range(Hkv))
    s = Setup(Case(dtype, D, Hkv, 1, groups, kv=((40,) * Hkv, (21,) * Hkv), T=(5, 4))).upload()
    kv = s.kv.astype(np.int32)
    stride = np.array([s.stride[g] for g in groups]) * 16
    good = np.ones(kv.shape, bool)
    for h, n in ((0, -1), (2, -2 ** 31), (4, stride[4] - 4), (Hkv - 1, 2 ** 31 - 1)):
        kv[0, h], good[0, h] = n, False
    kv[1, 1] = stride[1] - 4  # fits: 4 new rows
    want = [[bits(x).clone() for x in pool] for pool in (s.dk, s.dv)]
    for b, path in enumerate(([1, 4], [0, 3])):
        for h in range(Hkv):
            if good[b, h]:
                of, to = s.rows_of(b, h, s.kv[b, h] + np.array(path)), s.rows_of(b, h, s.kv[b, h] + np.arange(2))
                for pool in want:
                    pool[groups[h]][dev(to)] = pool[groups[h]][dev(of)]
    d_kv = dev(kv)
    out = d_kv if in_place else torch.full_like(d_kv, -7)
    kvx.kvx_tree_commit(s.cache, s.dqs, dev(s.slots()), s.max_rows, dev(np.array([[1, 4], [0, 3]], np.int32)),
                        dev(np.array([2, 2], np.int32)), d_kv, out, s.ws)
    torch.cuda.synchronize()
    assert s.status() == kvx.KVX_DEV_BAD_LENGTH
    assert np.array_equal(out.cpu().numpy(), kv + 2 * good)
    for pool, ref in zip((s.dk, s.dv), want):
        for x, w in zip(pool, ref):
            assert torch.equal(bits(x), w)


def test_commit_in_place_with_many_heads_again_and_again():
    """Lengths advance in place, by every block for its own heads: 64 heads are 8 blocks a sequence."""
    Hkv = 64
    s = Setup(Case("f32", 128, Hkv, 1, (0,) * Hkv, P=128, kv=((30,) * Hkv,) * 3, T=(6, 3, 4))).upload()
    kv = s.dkv.clone()
    path = dev(np.array([[0, 2], [1, 2], [0, 1]], np.int32))
    acc, slots = dev(np.array([2, 1, 0], np.int32)), dev(s.slots())
    for i in range(1, 30):
        kvx.kvx_tree_commit(s.cache, s.dqs, slots, s.max_rows, path, acc, kv, kv, s.ws)
        want = s.kv + i * np.array([2, 1, 0])[:, None]
        if i % 7 == 0:
            torch.cuda.synchronize()
            assert np.array_equal(kv.cpu().numpy(), want), i
    torch.cuda.synchronize()
    assert np.array_equal(kv.cpu().numpy(), want) and s.status() == 0
