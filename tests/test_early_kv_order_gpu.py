"""kvx_decode_attn with early K/V loads behind the calls that write pages and page tables.

The load warps of such a decode call read page ids and K/V pages before the launch's
dependency wait, so a call before it that writes several pages of a head has to hold its
dependents back. Each sequence of calls is made back to back with two sets of rows in
turn; every output has to equal, bit for bit, that of the same decode without early
loads after the device has finished the calls before it."""
import numpy as np
import pytest
import torch

from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu

B, HKV, G, D, P = 3, 2, 4, 128, 16
HQ = HKV * G
N0, T = 640, 200  # cached tokens; new rows: 12.5 pages of every head
PAGES_OF = 60     # pages of a sequence
ROUNDS = 20


class Cache:
    def __init__(self, token_major):
        gen = self.gen = torch.Generator(device="cuda").manual_seed(5)
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = self.pages = B * PAGES_OF
        self.k, self.v = (self.normal(pages * HKV * P, D) for _ in range(2))
        self.table = torch.randperm(pages, generator=gen, device="cuda").int().view(B, PAGES_OF)
        self.layout = kvx.KVX_LAYOUT_TOKEN_MAJOR if token_major else kvx.KVX_LAYOUT_HEAD_MAJOR
        self.cache = kvx.Cache(B, HQ, HKV, D, P, 1, kvx.KVX_BF16, [0] * HKV, [self.k], [self.v], [pages],
                               [self.table], [PAGES_OF], layout=self.layout)
        self.kv = torch.full((B, HKV), N0, **i32)
        self.q_start = torch.arange(B + 1, **i32) * T
        self.rows = B * T
        row = torch.arange(self.rows, device="cuda")
        t = N0 + row % T
        page = self.table[row // T, t // P].long()[:, None]
        h = torch.arange(HKV, device="cuda")[None]
        off = (t % P)[:, None]
        self.slots = ((page * P + off) * HKV + h if token_major else (page * HKV + h) * P + off).contiguous()
        self.new = [[self.normal(self.rows, HKV * D) for _ in range(2)] for _ in range(2)]
        self.q = self.normal(B, HQ, D)
        self.ws = torch.zeros(64, **i32)

    def normal(self, *shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(generator=self.gen)

    def append(self, d):
        kvx.kvx_append_kv(self.cache, *self.new[d], self.q_start, self.slots, self.rows, self.ws)

    def plan(self, tokens):
        """A decode over `tokens` tokens of every head: (plan, call)."""
        n = np.full((B, HKV), tokens, np.int32)
        plan = kvx.kvx_plan_create(B, HQ, HKV, D, P, 1, kvx.KVX_BF16, n, n[:, 0], [0] * HKV,
                                   layout=self.layout)
        kvx.kvx_plan_upload(plan)
        ws = torch.zeros(plan.workspace_bytes() // 4 + 64, dtype=torch.int32, device="cuda")
        budget, length = torch.from_numpy(n.reshape(-1)).cuda(), torch.from_numpy(n[:, 0].copy()).cuda()

        def decode(out):
            kvx.kvx_decode_attn(plan, self.q, [self.k], [self.v], [self.pages], [self.table], [PAGES_OF],
                                budget, length, 0.0, out, ws)
        self.decode_ws = ws
        return plan, decode


def compare(c, tokens, before, graph):
    """`before(d)`: the calls before the decode, with the rows of set d."""
    plan, decode = c.plan(tokens)
    want = []
    for d in range(2):
        before(d)
        torch.cuda.synchronize()
        out = torch.zeros(B, HQ, D, device="cuda")
        decode(out)
        torch.cuda.synchronize()
        want.append(out)
    assert not torch.equal(*want)
    plan.set_early_kv(True)
    outs = torch.full((ROUNDS, 2, B, HQ, D), float("nan"), device="cuda")

    def all_rounds():
        for r in range(ROUNDS):
            for d in range(2):
                before(d)
                decode(outs[r, d])

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            all_rounds()
        captured.replay()
    else:
        all_rounds()
    torch.cuda.synchronize()
    for d in range(2):
        assert torch.equal(outs[:, d], want[d].expand_as(outs[:, d])), d
    assert kvx.kvx_workspace_status(c.ws) == 0 and kvx.kvx_workspace_status(c.decode_ws) == 0


CASES = pytest.mark.parametrize("token_major,graph", [(False, False), (True, False), (False, True)])


@CASES
def test_append_then_early_decode(token_major, graph):
    c = Cache(token_major)
    compare(c, N0 + T, c.append, graph)


@CASES
def test_append_then_attention_then_early_decode(token_major, graph):
    """The kernels in between let their dependents start early; the append has to be over all the same."""
    c = Cache(token_major)
    i32 = dict(dtype=torch.int32, device="cuda")
    few, kv = torch.arange(B + 1, **i32), torch.full((B, HKV), 20, **i32)
    q, out = c.normal(B, HQ, D), torch.zeros(B, HQ, D, device="cuda")
    ws = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(c.cache, 1) // 4, **i32)

    def before(d):
        c.append(d)
        kvx.kvx_tree_attn(c.cache, q, few, B, 1, kv, None, 0.0, out, ws)

    compare(c, N0 + T, before, graph)
    assert kvx.kvx_workspace_status(ws) == 0


@CASES
def test_commit_then_early_decode(token_major, graph):
    """A branch of 70 rows out of 140: its rows move within five pages."""
    c = Cache(token_major)
    path = (2 * torch.arange(70, dtype=torch.int32, device="cuda") + 1).expand(B, 70).contiguous()
    acc = torch.full((B,), 70, dtype=torch.int32, device="cuda")
    kv_out = torch.zeros_like(c.kv)

    def before(d):
        c.append(d)
        kvx.kvx_tree_commit(c.cache, c.q_start, c.slots, c.rows, path, acc, c.kv, kv_out, c.ws)

    compare(c, N0 + 70, before, graph)


@CASES
def test_build_tables_then_early_decode(token_major, graph):
    """Both halves of the free list in turn: the same call writes other page ids into the tables."""
    c = Cache(token_major)
    i32 = dict(dtype=torch.int32, device="cuda")
    held = N0 // P
    c.table[:, held:] = 0  # (page ids that the calls replace)
    need = -(-(N0 + T) // P) - held
    pool = torch.randperm(c.pages, generator=c.gen, device="cuda").int()
    lists = [torch.cat([pool[:B * need], pool[:c.pages - B * need]]),
             torch.cat([pool[-B * need:], pool[:c.pages - B * need]])]
    free = [x.contiguous() for x in lists]
    count, count_out = torch.full((1,), B * need, **i32), torch.zeros(1, **i32)
    have, have_out = torch.full((1, B), held, **i32), torch.zeros(1, B, **i32)
    new, qs = torch.full((B,), T, **i32), torch.zeros(B + 1, **i32)
    slots = torch.zeros_like(c.slots)

    def before(d):
        kvx.kvx_build_tables(c.cache, c.kv, new, have, have_out, [free[d]], count, count_out, c.rows, qs,
                             slots, c.ws)

    compare(c, N0 + T, before, graph)
