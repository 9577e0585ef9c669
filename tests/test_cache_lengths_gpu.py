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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_at_the_longest_heads(dtype):
    """Heads next to 2^31 tokens, all in one page that the table repeats: positions stay in int32 up to the
    stated limit, past it a head is left out. The keys are zero, so that every weight is 1 and the sums are
    whole numbers below 2^24 in each piece; V[r][d] is 1 where r % 64 = d, so the output is 1/64 up to one
    page in 2^24, the division and the merge of at most 304 pieces (one rounding of 2^-24 each, of sum
    and normaliser)."""
    P, D, pages = 128, 64, 2 ** 24 - 1  # 2^31 - 128 tokens fit the table
    limit = 2 ** 31 - 1 - 4096
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.zeros(1, pages, **i32)
    k = torch.zeros(P, D, dtype=tt, device="cuda")
    v = torch.eye(D, dtype=tt, device="cuda").repeat(2, 1).contiguous()
    cache = kvx.Cache(1, 1, 1, D, P, 1, kvx.KVX_BF16 if dtype == "bf16" else kvx.KVX_F32, [0], [k], [v], [1],
                      [table], [pages])
    q = torch.ones(3, 1, D, dtype=tt, device="cuda")
    ws = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(cache, 3) // 4, **i32)
    for T, n, good in ((1, limit - 1, True), (3, limit - 3, True), (1, limit, False), (3, limit - 2, False),
                       (1, 2 ** 31 - 129, False), (2, 2 ** 31 - 130, False)):
        out = torch.full((3, 1, D), -7.0, device="cuda")
        kvx.kvx_tree_attn(cache, q, torch.tensor([0, T], **i32), 3, 3, torch.tensor([[n]], **i32), None, 0.0,
                          out, ws)
        torch.cuda.synchronize()
        assert kvx.kvx_workspace_status(ws) == (0 if good else kvx.KVX_DEV_BAD_LENGTH), (T, n)
        kvx.kvx_workspace_clear(ws)
        assert bool((out[T:] == -7.0).all())
        if good:
            err = (out[:T].double() * 64 - 1).abs().max().item()
            assert err <= 2.0 ** -23 + (2 * 304 + 2) * 2.0 ** -24, (T, n, err)
        else:
            assert bool((out == -7.0).all()), (T, n)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_have_no_influence(dtype, bad):
    """Query rows from q_start[B] on may share a load with the last sequence's; whatever they hold, the
    outputs keep their bits."""
    s = Setup(Case(dtype, 128, 2, 4, (0, 0), kv=((300, 20), (7, 140)), T=(5, 3)), extra_rows=9).upload()
    want = s.run()
    s.dq[s.N:] = bad
    s.out.fill_(-7.0)
    assert np.array_equal(s.run(), want) and np.all(want[s.N:] == -7.0)
    assert s.status() == 0
