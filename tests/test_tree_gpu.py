"""Tree attention on the GPU against the 64-bit definition."""
import numpy as np
import pytest
import torch

from paged_non_uniform_gb300 import kvx
from tree_cases import Case, Setup, check, to_dev

pytestmark = pytest.mark.gpu

CASES = [
    # the smallest: one token, one head, one cached token; nothing cached at all
    Case(Hkv=1, g=1, groups=(0,), kv=((1,),), T=(1,), mask="chain"),
    Case(Hkv=1, g=1, groups=(0,), kv=((0,),), T=(1,), mask="self"),
    Case("f32", 64, 2, 2, (0, 1), kv=((37, 20), (100, 20)), T=(5, 8)),
    Case("f32", 128, 2, 3, (0, 0), P=8, token_major=True, kv=((200, 63), (64, 1)), T=(33, 2)),
    Case("f32", 64, 1, 8, (0,), P=128, kv=((700,), (0,)), T=(9, 4), mask="empty"),
    # bf16: every head dim, GQA factor, page size and layout meets odd lengths
    Case("bf16", 64, 2, 1, (0, 0), P=8, kv=((130, 5), (127, 128)), T=(7, 1)),
    Case("bf16", 128, 2, 2, (0, 1), P=8, token_major=True, kv=((129, 300), (1, 0)), T=(16, 3)),
    Case("bf16", 128, 4, 4, (0, 1, 1, 0), P=16, kv=((700, 70, 33, 1), (333, 200, 1, 64)), T=(16, 5)),
    Case("bf16", 128, 3, 5, (2, 0, 1), P=32, kv=((255, 257, 256), (31, 32, 33)), T=(26, 48)),
    Case("bf16", 64, 1, 7, (0,), P=64, token_major=True, kv=((1000,), (63,), (65,)), T=(18, 64, 19)),
    Case("bf16", 128, 1, 8, (0,), P=128, kv=((500,), (0,)), T=(16, 17), mask="empty"),
    # 128 drafts: several row groups; masks of four words
    Case("bf16", 128, 2, 8, (0, 0), kv=((300, 129),), T=(128,)),
    Case("bf16", 64, 1, 3, (0,), kv=((90,), (91,)), T=(128, 100), mask="full"),
    # sequences without new rows, heads without a cache, rows that see nothing
    Case("bf16", 128, 2, 4, (0, 0), kv=((50, 0), (0, 0), (900, 3), (5, 5)), T=(0, 4, 0, 2),
         mask="empty"),
    Case("bf16", 128, 1, 2, (0,), kv=((0,), (0,)), T=(70, 33), mask="empty"),
    # one long head cut into many pieces
    Case("bf16", 128, 1, 4, (0,), kv=((9000,),), T=(16,)),
    Case("bf16", 64, 1, 2, (0,), P=64, kv=((20001,),), T=(65,), mask="chain"),
    Case("f32", 64, 1, 2, (0,), kv=((5000,),), T=(3,), mask="chain"),
    # single tokens: a decode step with device lengths
    Case("bf16", 128, 4, 4, (0, 0, 1, 1), kv=((900, 800, 10, 100),) * 5, T=(1,) * 5, mask="chain"),
    # query rows as slices; a peaked softmax
    Case("bf16", 128, 2, 4, (0, 0), kv=((300, 200),), T=(11,), fused=True),
    Case("f32", 64, 2, 2, (0, 0), kv=((100, 90),), T=(6,), fused=True),
    Case("bf16", 128, 2, 4, (0, 0), kv=((600, 200),), T=(12,), spread=8.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.name)
def test_matches_definition(case):
    s = Setup(case).upload()
    check(s, s.run())
    assert s.status() == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    r = np.random.default_rng(seed + 700)
    Hkv = int(r.integers(1, 5))
    G = int(r.integers(1, Hkv + 1))
    hg = np.concatenate([np.arange(G), r.integers(0, G, Hkv - G)])
    r.shuffle(hg)
    B = int(r.integers(1, 6))
    case = Case("f32" if seed % 4 == 3 else "bf16", int(r.choice([64, 128])), Hkv,
                int(r.integers(1, 9)), tuple(int(x) for x in hg), int(r.choice([8, 16, 32, 64, 128])),
                bool(r.integers(0, 2)),
                tuple(tuple(int(x) for x in r.integers(0, 600, Hkv)) for _ in range(B)),
                tuple(int(x) for x in r.integers(0, int(r.choice([3, 20, 70])), B)),
                str(r.choice(["tree", "empty", "chain", "full"])), seed)
    s = Setup(case).upload()
    check(s, s.run())
    assert s.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_rows_have_no_influence(dtype, bad):
    """NaN and infinities in a draft's K and V reach only the rows that see it: the others' bits
    are those of a run with ordinary values there."""
    case = Case(dtype, 128, 2, 4, (0, 1), kv=((140, 5), (0, 250)), T=(20, 9), mask="tree", seed=5)
    s = Setup(case)
    draft = 3
    ref = Setup(case).upload()
    want = ref.run()
    for b in range(s.B):
        for h in range(s.Hkv):
            at = s.rows_of(b, h, np.array([s.kv[b, h] + draft]))
            s.k[s.hg[h]][at] = bad
            s.v[s.hg[h]][at] = bad
    s.upload()
    got = s.run()
    for b in range(s.B):
        for i in range(int(s.T[b])):
            row = s.q_start[b] + i
            if s.see[b][i, draft]:
                assert not np.isfinite(got[row]).any(), (b, i)
            else:
                assert np.array_equal(got[row], want[row]), (b, i)
    assert s.status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_infinite_value_of_a_seen_draft_stays_in_its_dims(bad):
    """A non-finite element of one seen draft's V makes that output element non-finite for the rows
    that see it, and no other element."""
    case = Case("bf16", 128, 1, 4, (0,), kv=((140,),), T=(20,), mask="tree", seed=6)
    want = Setup(case).upload().run()
    s = Setup(case)
    at = s.rows_of(0, 0, np.array([140 + 2]))
    s.v[0][at, 77] = bad
    got = s.upload().run()
    for i in range(20):
        hit = np.zeros(128, bool)
        hit[77] = s.see[0][i, 2]
        assert np.array_equal(got[i][:, ~hit], want[i][:, ~hit]), i
        if hit.any():
            x = got[i][:, 77]
            assert np.all(np.isnan(x) if np.isnan(bad) else x == bad), (i, x)


def test_physical_page_order_does_not_matter():
    case = Case("bf16", 128, 2, 4, (0, 0), kv=((700, 300), (90, 1000)), T=(16, 3), seed=7)
    a = Setup(case)
    want = Setup(case).upload().run()
    perm = a.r.permutation(a.pages[0]).astype(np.int32)
    rows = a.size[0] * case.P
    for pool in (a.k, a.v):
        p = pool[0].reshape(a.pages[0], rows, -1)
        moved = np.empty_like(p)
        moved[perm] = p
        pool[0] = moved.reshape(-1, case.D)
    a.tables[0] = np.where(a.tables[0] >= 0, perm[np.maximum(a.tables[0], 0)], -1).astype(np.int32)
    assert np.array_equal(a.upload().run(), want)


def test_repeated_calls_and_shared_workspace():
    """The counters return to zero: calls of two shapes take turns in one workspace and give the
    same bits every time."""
    a = Setup(Case("bf16", 128, 1, 4, (0,), kv=((6000,),), T=(16,), seed=8)).upload()
    b = Setup(Case("bf16", 128, 2, 2, (0, 0), kv=((3000, 90), (1, 700)), T=(5, 40), seed=9)).upload()
    big = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.int32, device="cuda")
    a.ws = b.ws = big
    wa, wb = a.run().copy(), b.run().copy()
    for _ in range(20):
        a.attend()
        b.attend()
    torch.cuda.synchronize()
    assert np.array_equal(a.out.cpu().numpy(), wa) and np.array_equal(b.out.cpu().numpy(), wb)
    check(a, wa)
    check(b, wb)


def test_other_stream_and_graph_replay_with_new_lengths():
    """A captured call reads the lengths at replay: shorter and longer heads, ended sequences."""
    case = Case("bf16", 128, 2, 4, (0, 0), kv=((2000, 900), (300, 20), (50, 60)), T=(16, 9, 1), seed=10)
    s = Setup(case).upload()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.attend()
    side.synchronize()
    check(s, s.out.cpu().numpy())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.attend()
    for kv, T in ((case.kv, case.T), (((1500, 3), (300, 20), (0, 9)), (16, 9, 1)),
                  (((100, 900), (20, 7), (50, 60)), (4, 0, 1))):
        n = Setup(Case("bf16", 128, 2, 4, (0, 0), kv=kv, T=T, seed=10))
        s.kv, s.T = n.kv, n.T
        s.q_start, s.N, s.see = n.q_start, n.N, n.see
        s.dkv.copy_(torch.from_numpy(n.kv.astype(np.int32)))
        s.dqs.copy_(torch.from_numpy(n.q_start))
        words = np.zeros((s.max_rows, 1), np.uint32)
        for b in range(3):
            for i in range(T[b]):
                for j in range(T[b]):
                    words[n.q_start[b] + i, 0] |= np.uint32(int(n.see[b][i, j]) << j)
        s.dmask.copy_(torch.from_numpy(words.view(np.int32)))
        s.out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        # lengths shrank inside the pages already filled: every token read is a filled one
        check(s, s.out.cpu().numpy())
    assert s.status() == 0


def test_agrees_with_plan_decode_for_single_tokens():
    """One new row a sequence is a decode step: kvx_decode_attn over n + 1 kept tokens."""
    case = Case("bf16", 128, 2, 4, (0, 1), kv=((300, 80), (41, 7)), T=(1, 1), mask="chain", seed=11)
    s = Setup(case, extra_rows=0).upload()
    got = s.run()
    n = (s.kv + 1).astype(np.int32)
    L = n.max(1).astype(np.int32)
    plan = kvx.kvx_plan_create(2, 8, 2, 128, 16, 2, kvx.KVX_BF16, n, L, s.hg)
    kvx.kvx_plan_upload(plan)
    ws = torch.zeros(plan.workspace_bytes() // 4 + 64, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 8, 128, device="cuda")
    kvx.kvx_decode_attn(plan, s.dq, s.dk, s.dv, s.pages, s.dt, s.stride,
                        torch.from_numpy(n.reshape(-1)).cuda(), torch.from_numpy(L).cuda(), 0.0, out, ws)
    torch.cuda.synchronize()
    _, tol = s.reference()
    assert np.all(np.abs(out.cpu().numpy() - got) <= 2 * tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_skip_their_sequence(dtype):
    """Row starts, row counts and cached lengths out of range: that sequence's rows (that head's
    outputs) are left as they were, the others are computed, and the status says so."""
    case = Case(dtype, 64, 2, 2, (0, 1), kv=((40, 30), (20, 10), (33, 5)), T=(4, 4, 4), seed=12)
    ref, tol = Setup(case).reference()

    def outcome(kv=None, q_start=None, max_q=None):
        s = Setup(case).upload()
        if kv is not None:
            s.dkv.copy_(torch.tensor(kv, dtype=torch.int32))
        if q_start is not None:
            s.dqs.copy_(torch.tensor(q_start, dtype=torch.int32))
        s.attend(max_q=max_q)
        torch.cuda.synchronize()
        out = s.out.cpu().numpy()
        assert s.status() == kvx.KVX_DEV_BAD_LENGTH
        fine = np.zeros(out.shape[:2], bool)
        fine[:12] = np.all(np.abs(out[:12] - ref) <= tol, axis=2)
        kept = np.all(out == -7.0, axis=2)
        assert np.all(fine | kept)
        return fine[:12].reshape(3, 4, 2, 2).all(axis=(1, 3)), kept[:12].reshape(3, 4, 2, 2).all(axis=(1, 3))

    fine, kept = outcome(kv=[[40, 30], [-1, 10], [33, 10 ** 9]])
    assert fine.tolist() == [[True, True], [False, True], [True, False]] and np.array_equal(kept, ~fine)
    fine, kept = outcome(q_start=[0, 4, 8, 1000])
    assert fine.tolist() == [[True, True]] * 2 + [[False, False]] and np.array_equal(kept, ~fine)
    fine, kept = outcome(q_start=[-4, 4, 8, 12])
    assert fine.tolist() == [[False, False]] + [[True, True]] * 2 and np.array_equal(kept, ~fine)


def test_too_many_rows_for_max_q_are_skipped():
    case = Case("bf16", 64, 1, 2, (0,), kv=((40,), (20,)), T=(9, 4), mask="chain", seed=13)
    s = Setup(case).upload()
    s.attend(max_q=8)
    torch.cuda.synchronize()
    out = s.out.cpu().numpy()
    ref, tol = s.reference()
    assert np.all(out[:9] == -7.0) and np.all(np.abs(out[9:13] - ref[9:]) <= tol[9:])
    assert s.status() == kvx.KVX_DEV_BAD_LENGTH


@pytest.mark.parametrize("page", [-5, 10 ** 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_read_zeros(dtype, page):
    case = Case(dtype, 128, 1, 2, (0,), kv=((100,),), T=(4,), mask="chain", seed=14)
    s = Setup(case)
    at = s.rows_of(0, 0, np.arange(32, 48))
    s.k[0][at] = 0
    s.v[0][at] = 0
    ref = s.reference()
    s.tables[0][0, 2] = page
    s.upload()
    got = s.run()
    assert np.all(np.abs(got[:4] - ref[0]) <= ref[1])
    assert s.status() == kvx.KVX_DEV_BAD_PAGE


def test_pool_past_32_bit_offsets():
    """Pages at the far end of pools larger than 4 GiB."""
    case = Case("bf16", 128, 1, 4, (0,), P=64, kv=((150,),), T=(5,), seed=15)
    s = Setup(case)
    far = (5 << 30) // (64 * 256)
    want = Setup(case).upload().run()
    s.upload()
    pools = []
    for small in (s.dk[0], s.dv[0]):
        big = torch.empty((far + s.pages[0]) * 64 * 128, dtype=torch.bfloat16, device="cuda")
        big[far * 64 * 128:] = small.reshape(-1)
        pools.append(big)
    table = [s.dt[0] + far * (s.dt[0] >= 0).int()]
    s.cache = kvx.Cache(1, 4, 1, 128, 64, 1, kvx.KVX_BF16, [0], pools[:1], pools[1:],
                        [far + s.pages[0]], table, s.stride)
    assert np.array_equal(s.run(), want)
    assert s.status() == 0


def test_binding_refuses_tensors_that_do_not_fit():
    s = Setup(Case(kv=((40, 7),), T=(5,))).upload()
    good = dict(cache=s.cache, q=s.dq, q_start=s.dqs, max_rows=s.max_rows, max_q=5, kv_len=s.dkv,
                mask=s.dmask, scale=0.0, out=s.out, workspace=s.ws)
    kvx.kvx_tree_attn(**good)
    for change in (dict(q=s.dq.float()), dict(q=s.dq[:, :4]), dict(q=s.dq.transpose(1, 2)),
                   dict(q=s.dq.cpu()), dict(kv_len=s.dkv.long()), dict(out=s.out[:-1]),
                   dict(out=s.out.half()), dict(mask=s.dmask[:1]), dict(q_start=s.dqs[:1]),
                   dict(max_rows=s.max_rows + 1), dict(workspace=s.ws[:64])):
        with pytest.raises(kvx.KvxError) as e:
            kvx.kvx_tree_attn(**{**good, **change})
        assert e.value.status == kvx.KVX_EINVAL, change.keys()
    torch.cuda.synchronize()
    check(s, s.out.cpu().numpy())


def test_guard_bands():
    """Output and workspace sit between canary bands, which stay intact."""
    s = Setup(Case("bf16", 128, 2, 4, (0, 1), kv=((5000, 70), (1, 333)), T=(16, 40), seed=16)).upload()
    band = 4096

    def guarded(t):
        whole = torch.full((2 * band + t.numel() * 4,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = whole[band:-band].view(t.dtype).view(t.shape)
        inner.copy_(t)
        return inner, whole

    s.out, out_w = guarded(s.out)
    n = kvx.kvx_tree_attn_workspace_bytes(s.cache, s.max_q)
    s.ws, ws_w = guarded(s.ws[:n // 4])
    check(s, s.run())
    for w in (out_w, ws_w):
        w = w.cpu().numpy()
        assert np.all(w[:band] == 0xA5) and np.all(w[-band:] == 0xA5)


@pytest.mark.parametrize("T,D", [(3, 64), (40, 64), (40, 128)])
def test_long_items_leave_tensor_memory_in_time(T, D):
    """One head of 1.4 M keys: every block works on 36 tiles of it (72 with 160 rows, which are two row
    groups), so that its output is folded into the fp32 sum twice or four times. The tensor cores
    truncate what they add: 16 additions to an output element a tile, each off by at most 2^-23 of the sum
    so far, over the 16 tiles between folds; the folds and the merge round like fp32."""
    n, g = 1_400_000, 4
    P, len_ = 128, 1_400_000 + T
    pages = -(-len_ // P)
    gen = torch.Generator(device="cuda").manual_seed(T)
    k = torch.empty(pages * P, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    v = torch.empty(pages * P, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    v += 0.5  # sums that grow
    q = torch.empty(T, g, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    table = torch.randperm(pages, generator=gen, device="cuda").int().view(1, -1)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = kvx.Cache(1, g, 1, D, P, 1, kvx.KVX_BF16, [0], [k], [v], [pages], [table], [pages])
    ws = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(cache, T) // 4, **i32)
    out = torch.zeros(T, g, D, device="cuda")
    for _ in range(2):
        kvx.kvx_tree_attn(cache, q, torch.tensor([0, T], **i32), T, T, torch.tensor([[n]], **i32), None, 0.0,
                          out, ws)
    torch.cuda.synchronize()
    at = (table.long().view(-1, 1) * P + torch.arange(P, device="cuda")).view(-1)[:len_]
    kd, vd = k[at].double(), v[at].double()
    x = q.view(T * g, D).double() @ kd.T / D ** 0.5
    row = torch.arange(T * g, device="cuda") // g
    x[:, n:] = x[:, n:].masked_fill(torch.arange(T, device="cuda") > row[:, None], -float("inf"))
    p = torch.softmax(x, 1)
    want, mag = p @ vd, p @ vd.abs()
    far = float((x.amax(1) - x[:, :n].amin(1)).max()) + float(x[:, :n].abs().max())
    s_abs = float((q.view(T * g, D).double().abs() @ kd.abs().T).max()) / D ** 0.5
    u = 2.0 ** -24
    weight = 2 * u * (D + 2) * s_abs + 3 * u * far + 2.0 ** -22
    # truncation between folds 2u * 16 * 16; a sum of l over 128 keys of a tile by four chains, tiles and
    # pieces: (32 + 72 + 152) u; folds and merge (5 + 152) u of output and sum
    tol = (2 * weight + 2.0 ** -18 + 2 * u * 256 + (256 + 2 * 157) * u) * mag
    err = (out.view(T * g, D).double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol).max()))
    assert kvx.kvx_workspace_status(ws) == 0


def batch_reference(kp, vp, tables, kv, q_start, q, see, scale, P):
    """float64 attention of every sequence and head on the GPU: pools [pages][P][D] of one head group of
    one head each, tables [Hkv][B][stride]; see[b]: bool [T][T]."""
    Hkv, g = len(kp), q.shape[1] // len(kp)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for b in range(kv.shape[0]):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        if r0 == r1:
            continue
        hide = torch.from_numpy(~see[b]).cuda()
        for h in range(Hkv):
            n = int(kv[b, h])
            t = torch.arange(n + r1 - r0, device="cuda")
            rows = tables[h][b][t // P].long() * P + t % P
            k, v = kp[h].view(-1, kp[h].shape[-1])[rows].double(), vp[h].view(-1, vp[h].shape[-1])[rows].double()
            x = torch.einsum("tgd,ld->tgl", q[r0:r1, h * g:(h + 1) * g].double(), k) * scale
            x[:, :, n:] = x[:, :, n:].masked_fill(hide[:, None], -float("inf"))
            p = torch.nan_to_num(torch.softmax(x, -1))  # rows that see nothing
            out[r0:r1, h * g:(h + 1) * g] = p @ v
            mag[r0:r1, h * g:(h + 1) * g] = p @ v.abs()
    return out, mag


@pytest.mark.parametrize("dtype,g,tmax,hi", [("bf16", 4, 8, 700), ("bf16", 5, 48, 5000), ("bf16", 8, 128, 900),
                                             ("bf16", 2, 1, 3000), ("f32", 3, 20, 800)])
def test_many_ragged_sequences(dtype, g, tmax, hi):
    """Batches in which every block has several items of unlike lengths, cut at any tile: 60 sequences
    x 4 heads with budgets of their own, some sequences without rows, some heads without a cache."""
    r = np.random.default_rng(tmax)
    B, Hkv, D, P = 60, 4, 128, 16
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(tmax)
    kv = r.integers(0, hi + 1, (B, Hkv))
    kv[r.random((B, Hkv)) < 0.05] = 0
    T = r.integers(0, tmax + 1, B)
    q_start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
    N = int(q_start[-1])
    stride = -(-(hi + tmax) // P)
    kp = [torch.empty(B * stride, P, D, dtype=tt, device="cuda").normal_(generator=gen) for _ in range(Hkv)]
    vp = [torch.empty(B * stride, P, D, dtype=tt, device="cuda").normal_(generator=gen) for _ in range(Hkv)]
    tables = [torch.randperm(B * stride, generator=gen, device="cuda").int().view(B, stride) for _ in range(Hkv)]
    q = torch.empty(N, Hkv * g, D, dtype=tt, device="cuda").normal_(generator=gen)
    W = (tmax + 31) // 32
    see = [np.tril(r.random((t, t)) < 0.4) for t in T]  # (rows that see no draft among them)
    words = np.zeros((N, W), np.uint32)
    for b in range(B):
        for i in range(T[b]):
            for j in np.flatnonzero(see[b][i]):
                words[q_start[b] + i, j // 32] |= np.uint32(1 << (j % 32))
    cache = kvx.Cache(B, Hkv * g, Hkv, D, P, Hkv, kvx.KVX_BF16 if dtype == "bf16" else kvx.KVX_F32,
                      list(range(Hkv)), kp, vp, [B * stride] * Hkv, tables, [stride] * Hkv)
    ws = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(cache, tmax) // 4, dtype=torch.int32, device="cuda")
    out = torch.full((N, Hkv * g, D), float("nan"), device="cuda")
    args = (cache, q, torch.from_numpy(q_start).cuda(), N, tmax, torch.from_numpy(kv.astype(np.int32)).cuda(),
            torch.from_numpy(words.view(np.int32)).cuda(), 0.0, out, ws)
    kvx.kvx_tree_attn(*args)
    torch.cuda.synchronize()
    first = out.clone()
    for _ in range(5):
        kvx.kvx_tree_attn(*args)
    torch.cuda.synchronize()
    assert torch.equal(out, first)  # equal inputs give equal bits
    assert kvx.kvx_workspace_status(ws) == 0
    want, mag = batch_reference(kp, vp, tables, kv, q_start, q, see, D ** -0.5, P)
    # error_bound of tree_cases with |s| <= 8 (128-dim dot products of N(0, 1), scaled; largest of 10^7
    # draws below 6), s_abs <= 14 (mean 7.2, deviation 0.6), at most hi + 128 keys
    u = 2.0 ** -24
    weight = 2 * u * 130 * 14 + 3 * u * 24 + 2.0 ** -22
    tol = (2 * weight + 2.0 ** -18 + 4 * u * (hi + 192) + 4 * u) * mag
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol.clamp(min=1e-30)).max()))


def test_wait_that_runs_out_is_reported():
    """A block whose first K tile never arrives gives up after the limit: the call ends with
    KVX_DEV_TIMEOUT, and the next call on a cleared workspace is right."""
    s = Setup(Case("bf16", 128, 2, 4, (0, 0), kv=((3000, 700), (900, 20)), T=(16, 9), seed=17)).upload()
    want = s.run().copy()
    s.cache.inject_stall(1, 20_000_000)
    s.attend()
    torch.cuda.synchronize()
    assert s.status() & kvx.KVX_DEV_TIMEOUT
    s.cache.inject_stall(-1, 2_000_000_000)
    kvx.kvx_workspace_clear(s.ws)
    assert np.array_equal(s.run(), want)
    assert s.status() == 0


def test_calls_on_two_streams_at_once():
    """Two caches' attention in two streams, each with a workspace of its own and its call repeated back
    to back: the outputs are those of each alone, bit for bit."""
    sets = [Setup(Case("bf16", 128, 4, 4, (0, 1, 1, 0), kv=((3000, 700, 900, 10),) * 8, T=(16, 5) * 4,
                       seed=31)).upload(),
            Setup(Case("bf16", 64, 2, 8, (0, 0), kv=((2000, 2000),) * 12, T=(40, 1, 33) * 4,
                       seed=32)).upload()]
    want = [s.run().copy() for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in sets:
        s.out.fill_(-7.0)
    torch.cuda.synchronize()
    for _ in range(50):
        for s, st in zip(sets, streams):
            s.attend(stream=st.cuda_stream)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert np.array_equal(s.out.cpu().numpy(), w)
        assert s.status() == 0
