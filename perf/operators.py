"""Cases of the operators that make one speculative-decoding step over the
non-uniform paged KV cache: page tables and slot maps built on the GPU from
request lengths, the scatter of new K/V rows into pages, attention for a tree of
drafted tokens over the cache, and the compaction of the accepted branch.

A case is a dict of plain values:
  op        "tables", "append", "tree" or "commit"
  B, Hq, Hkv, D, P, groups, layout, dtype   the cache's shape; `groups` counts the KV heads of each
            head group, `layout` is "head" or "token" (page layout)
  lo, hi    cached tokens of a sequence, log-uniform in [lo, hi]
  keep      "full" (every head keeps all), "mix" (a quarter of the heads keep all, the others 10-50 %) or
            "half" (half keep all, half 12.5 %)
  tmin, tmax   new rows of a sequence, uniform in [tmin, tmax] (log-uniform for prompts)

`run` in its plain form is elementary torch in 32 bits; with `own` it makes the
library's calls.
"""
from __future__ import annotations

import math
import zlib

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    tiny = dict(B=2, Hq=4, Hkv=2, D=64, P=16, groups="1,1", layout="head", dtype="f32")
    q4 = dict(B=16, Hq=32, Hkv=8, D=128, P=16, groups="2,3,3", layout="head", dtype="bf16")
    q32 = dict(Hq=40, Hkv=8, D=128, P=32, groups="2,2,2,2", layout="head", dtype="bf16")
    rm = dict(B=256, Hq=32, Hkv=8, D=128, P=16, groups="8", layout="token", dtype="bf16")
    return [
        # between two verify steps of a batch: most sequences grow by their drafts, some end, one starts
        dict(name="tables_step", op="tables", lo=8192, hi=32768, keep="mix", tmin=4, tmax=16, **q4),
        # a wave of prompts admitted at once (the movement workload's 256 sequences)
        dict(name="tables_prompts", op="tables", lo=0, hi=0, keep="full", tmin=512, tmax=16384, **rm),
        # drafted tokens of a batch of 16 written into the pages
        dict(name="append_step", op="append", lo=512, hi=2048, keep="mix", tmin=16, tmax=16, **q4),
        # prompts of a prefill written into token-major pages
        dict(name="append_prompts", op="append", lo=0, hi=0, keep="full", tmin=64, tmax=1024, **rm),
        # the smallest call: two short sequences in fp32
        dict(name="tree_tiny", op="tree", lo=37, hi=100, keep="full", tmin=5, tmax=8, **tiny),
        # one interactive user, a short chat, a tree of 16 drafts
        dict(name="tree_one_user", op="tree", lo=1500, hi=2500, keep="full", tmin=16, tmax=16, **{**q4, "B": 1}),
        # the decode benchmark's layer with 16 drafts a sequence (64 query rows a KV head)
        dict(name="tree_qwen3_4b", op="tree", lo=8192, hi=32768, keep="mix", tmin=16, tmax=16, **q4),
        # ragged trees (1..48 drafts, 5 query heads a KV head: up to 240 query rows), bimodal budgets
        dict(name="tree_ragged_32b", op="tree", B=32, lo=1000, hi=32000, keep="half", tmin=1, tmax=48, **q32),
        # KV-RM blocks (token-major), short histories, many sequences: 8 drafts each
        dict(name="tree_many_short", op="tree", lo=100, hi=1000, keep="full", tmin=1, tmax=8, **rm),
        # long context: 8 x 122k tokens, 24 drafts
        dict(name="tree_long", op="tree", lo=121000, hi=123000, keep="full", tmin=24, tmax=24,
             **{**q4, "B": 8, "groups": "8"}),
        # accepted branches of a batch of 16
        dict(name="commit_step", op="commit", lo=200, hi=1000, keep="mix", tmin=16, tmax=16, **q4),
        # accepted branches of 256 sequences with wide trees, token-major
        dict(name="commit_wide", op="commit", lo=100, hi=400, keep="full", tmin=24, tmax=64, **rm),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    cuts, left = [], Hkv
    while left:
        cuts.append(rng.randint(1, left))
        left -= cuts[-1]
    c = dict(op=rng.choice(["tables", "append", "tree", "tree", "tree", "commit"]), Hq=Hkv * g, Hkv=Hkv,
             D=rng.choice([64, 128, 128]), P=rng.choice([8, 16, 16, 32, 64, 128]),
             groups=",".join(map(str, cuts)), layout=rng.choice(["head", "token"]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), keep=rng.choice(["full", "mix", "half"]))
    if c["op"] == "tree":
        small = c["dtype"] == "f32"  # fp32 caches are the small end of the range
        c["hi"] = _log(rng, 20, 3000 if small else 60000)
        c["lo"] = _log(rng, max(1, c["hi"] // 20), c["hi"])
        c["tmax"] = _log(rng, 1, max(1, min(128, (64 if small else 512) // g)))
        most = 8000 if small else min(500000, 90000000 // (c["tmax"] * g))
        c["B"] = _log(rng, 1, max(1, min(64, most // c["hi"])))
    elif c["op"] == "tables":
        c["lo"], c["hi"] = 0, 0
        c["tmax"] = _log(rng, 1, 8000)
        c["B"] = _log(rng, 1, max(1, min(1000, 1000000 // c["tmax"])))
        if rng.random() < 0.6:
            c["tmax"] = min(c["tmax"], 64)
            c["hi"] = _log(rng, 20, 30000)
            c["lo"] = _log(rng, 1, c["hi"])
    elif c["op"] == "append":
        c["lo"], c["hi"] = 0, 0
        c["tmax"] = _log(rng, 1, 2000)
        c["B"] = _log(rng, 1, max(1, min(256, 60000 // c["tmax"])))
    else:
        c["hi"] = _log(rng, 1, 600)
        c["lo"] = _log(rng, 1, c["hi"])
        c["tmax"] = _log(rng, 1, 128)
        c["B"] = _log(rng, 1, 128)
    c["tmin"] = _log(rng, 1, c["tmax"])
    return c


# ---------------------------------------------------------------- inputs
def _sizes(case):
    return [int(x) for x in case["groups"].split(",")]


def _lengths(case):
    """What the case fixes and a seed only reorders: cached tokens a head [B][Hkv] (heads by falling
    budget), new rows [B], and pages held before the call [G][B]. Sizes, and so the work, are the case's."""
    r = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    B, Hkv, P = case["B"], case["Hkv"], case["P"]
    L = np.zeros(B, np.int64)
    if case["hi"] > 0:
        L = np.round(np.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"]), B))).astype(np.int64)
    if case["keep"] == "full":
        rho = np.ones(Hkv)
    elif case["keep"] == "half":
        rho = np.where(np.arange(Hkv) < (Hkv + 1) // 2, 1.0, 0.125)
    else:
        rho = np.sort(r.uniform(0.1, 0.5, Hkv))[::-1].copy()
        rho[: max(1, Hkv // 4)] = 1.0
    kv = np.maximum(np.ceil(L[:, None] * rho[None]), (L > 0)[:, None]).astype(np.int32)
    if case["op"] in ("tables", "append") and case["hi"] == 0:
        new = np.round(np.exp(r.uniform(math.log(case["tmin"]), math.log(case["tmax"]), B))).astype(np.int32)
    else:
        new = r.integers(case["tmin"], case["tmax"] + 1, B).astype(np.int32)
    ends = np.cumsum([0] + _sizes(case))

    def tokens():
        return np.stack([kv[:, a:z].max(1) for a, z in zip(ends[:-1], ends[1:])]).astype(np.int64)

    held = tokens() + new[None]
    if case["op"] == "tables":
        # the step before had its own drafts, some of which were rejected; a tenth of the sequences end
        # now, a tenth start
        held = tokens() + r.integers(0, case["tmax"] + 1, B)[None]
        held[tokens() == 0] = 0
        if case["hi"] > 0:
            fate = r.random(B)
            end, start = fate < 0.1, fate > 0.9
            kv[end | start] = 0
            new[end] = 0
            held[:, start] = 0
    need = -(-(tokens() + new[None]) // P)
    return kv, new, -(-held // P), need


def _tree(r, T):
    """Parents of a random tree of T drafts in topological order (-1: a child of the cached token)."""
    return np.array([r.integers(-1, i) if i else -1 for i in range(T)])


def prepare(case, seed):
    r = np.random.default_rng([int(seed), 17])
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) + 1)
    op, B, Hq, Hkv, D, P = case["op"], case["B"], case["Hq"], case["Hkv"], case["D"], case["P"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    sizes = _sizes(case)
    G = len(sizes)

    kv_len, new_len, need_old, need_new = _lengths(case)
    seqs, heads = r.permutation(B), r.permutation(Hkv)
    kv_len, new_len = kv_len[seqs][:, heads], new_len[seqs]
    need_old, need_new = need_old[:, seqs], need_new[:, seqs]
    grp = np.repeat(np.arange(G, dtype=np.int32), sizes)[heads]  # heads of like budgets share a group
    row = np.array([np.sum(grp[:h] == grp[h]) for h in range(Hkv)])
    N = int(new_len.sum())
    max_rows = N + 3  # the caller's row buffers are a little larger than this step's rows
    stride = int(max(need_old.max(), need_new.max(), 1)) + 2
    pages = int(np.maximum(need_old, need_new).sum(1).max()) + 5
    tables = np.full((G, B, stride), -1, np.int32)
    free = np.full((G, pages), -1, np.int32)
    n_free = np.zeros(G, np.int32)
    for g in range(G):
        ids = r.permutation(pages).astype(np.int32)
        tables[g][np.arange(stride)[None] < need_old[g][:, None]] = ids[: need_old[g].sum()]
        rest = ids[need_old[g].sum():]
        free[g, : rest.size] = rest
        n_free[g] = rest.size
    cu = np.concatenate([[0], np.cumsum(new_len)]).astype(np.int32)

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    s = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, G=G, sizes=sizes, layout=case["layout"], max_rows=max_rows,
             pages=pages, stride=stride, tables=up(tables), kv_len=up(kv_len), new_len=up(new_len),
             q_start=up(cu), grp=up(grp.astype(np.int64)), row=up(row.astype(np.int64)),
             gsize=up(np.array(sizes)[grp].astype(np.int64)), head_group=grp, case=dict(case))
    # one buffer holds the pools of all groups, [pages][heads of the group][P][D] one after the other
    rows_of = [pages * n * P for n in sizes]
    base = np.concatenate([[0], np.cumsum(rows_of)])
    s["base_g"] = base
    s["base"] = up(base[:-1][grp].astype(np.int64))
    total = int(base[-1])
    if op == "tables":
        s.update(free=up(free), free_in=up(n_free), pages_in=up(need_old.astype(np.int32)),
                 pages_out=torch.zeros((G, B), dtype=torch.int32, device=dev),
                 free_out=torch.zeros(G, dtype=torch.int32, device=dev),
                 cu_out=torch.zeros(B + 1, dtype=torch.int32, device=dev),
                 slots=torch.full((max_rows, Hkv), -7, dtype=torch.int64, device=dev),
                 masks=up(np.stack([grp == g for g in range(G)])))
        s["k"] = s["v"] = None
    else:
        s["k"] = torch.empty((total, D), dtype=dt, device=dev).normal_(generator=gen)
        s["v"] = torch.empty((total, D), dtype=dt, device=dev).normal_(generator=gen)
        s["slots"] = _slots(s, max_rows)
    if op == "append":
        # K and V of the new rows as a fused projection leaves them: slices of one row
        fused = torch.empty((max_rows, (Hq + 2 * Hkv) * D), dtype=dt, device=dev).normal_(generator=gen)
        s["k_new"] = fused[:, Hq * D:(Hq + Hkv) * D]
        s["v_new"] = fused[:, (Hq + Hkv) * D:]
    if op == "tree":
        T = case["tmax"]
        W = (T + 31) // 32
        mask = np.zeros((max_rows, W), np.uint32)
        for b in range(B):
            par = _tree(r, int(new_len[b]))
            for i in range(int(new_len[b])):
                m = mask[cu[b] + par[i]] if par[i] >= 0 else np.zeros(W, np.uint32)
                mask[cu[b] + i] = m
                mask[cu[b] + i, i // 32] |= np.uint32(1 << (i % 32))
        s.update(q=torch.empty((max_rows, Hq, D), dtype=dt, device=dev).normal_(generator=gen), T=T, W=W,
                 mask=up(mask.view(np.int32)), out=torch.zeros((max_rows, Hq, D), device=dev),
                 span=int((kv_len + new_len[:, None]).max()), scale=1.0 / math.sqrt(D))
    if op == "commit":
        T = case["tmax"]
        depth = min(T, 12)
        path = np.zeros((B, depth), np.int32)
        acc = np.zeros(B, np.int32)
        for b in range(B):
            par = _tree(r, int(new_len[b]))
            at, up_path = int(r.integers(0, new_len[b])), []
            while at >= 0:
                up_path.append(at)
                at = int(par[at])
            p = up_path[::-1][:depth]
            acc[b] = len(p)
            path[b, : len(p)] = p
        s.update(path=up(path), n_acc=up(acc), depth=depth,
                 kv_out=torch.zeros((B, Hkv), dtype=torch.int32, device=dev))
    if own:
        _handles(s, dt)
    return s


def _handles(s, dt):
    """What a program keeps from step to step: the cache handle and the workspace."""
    from paged_non_uniform_gb300 import kvx
    if s["k"] is None:  # the table call reads no pool: any device address serves
        dummy = torch.zeros(64, dtype=torch.int32, device="cuda")
        kp = vp = [dummy] * s["G"]
        s["dummy"] = dummy
    else:
        cut = s["base_g"]
        kp = [s["k"][cut[g]:cut[g + 1]] for g in range(s["G"])]
        vp = [s["v"][cut[g]:cut[g + 1]] for g in range(s["G"])]
    s["cache"] = kvx.Cache(s["B"], s["Hq"], s["Hkv"], s["D"], s["P"], s["G"],
                           kvx.KVX_BF16 if dt == torch.bfloat16 else kvx.KVX_F32, s["head_group"], kp, vp,
                           [s["pages"]] * s["G"], [s["tables"][g] for g in range(s["G"])],
                           [s["stride"]] * s["G"],
                           layout=kvx.KVX_LAYOUT_TOKEN_MAJOR if s["layout"] == "token" else kvx.KVX_LAYOUT_HEAD_MAJOR)
    nbytes = kvx.KVX_WS_HEADER_BYTES
    if s["op"] == "tree":
        nbytes = kvx.kvx_tree_attn_workspace_bytes(s["cache"], s["T"])
    s["ws"] = torch.zeros(-(-nbytes // 4), dtype=torch.int32, device="cuda")
    if s["op"] == "tables":
        s["free_list"] = [s["free"][g] for g in range(s["G"])]


# ---------------------------------------------------------------- plain forms
def _slots(s, max_rows, tables=None, q_start=None):
    """Slot map: [max_rows][Hkv] pool rows of the new tokens (rows behind the last sequence: 0)."""
    tables = s["tables"] if tables is None else tables
    q_start = (s["q_start"] if q_start is None else q_start).long()
    at = torch.arange(max_rows, device="cuda")
    b = (torch.searchsorted(q_start, at, right=True) - 1).clamp(max=s["B"] - 1)
    t = s["kv_len"].long()[b] + (at - q_start[b])[:, None]
    live = (at < q_start[-1])[:, None]
    t = torch.where(live, t, 0)
    page = tables[s["grp"][None], b[:, None], t // s["P"]].long()
    P, n, r = s["P"], s["gsize"][None], s["row"][None]
    slot = (page * P + t % P) * n + r if s["layout"] == "token" else (page * n + r) * P + t % P
    return torch.where(live, slot, 0)


def _plain_tables(s):
    P, G, B = s["P"], s["G"], s["B"]
    tokens = torch.where(s["masks"][:, None], s["kv_len"][None], 0).amax(2) + s["new_len"][None]
    need = (tokens.long() + P - 1) // P
    have = s["pages_in"].long()
    rel, alloc = (have - need).clamp(min=0), (need - have).clamp(min=0)
    rel_end, alloc_end = rel.cumsum(1), alloc.cumsum(1)
    R, A = rel_end[:, -1], alloc_end[:, -1]
    F = s["free_in"].long()
    j = torch.arange(s["stride"], device="cuda")[None, None]
    # released pages go on the stack in order (a dummy column takes what is not released)
    gone = (j >= need[..., None]) & (j < have[..., None])
    at = torch.where(gone, F[:, None, None] + (rel_end - rel)[..., None] + j - need[..., None], s["pages"])
    stack = torch.cat([s["free"], s["free"][:, :1]], 1).scatter(1, at.reshape(G, -1), s["tables"].reshape(G, -1))[:, :-1]
    # new pages come off its top
    fresh = (j >= have[..., None]) & (j < need[..., None])
    k = (alloc_end - alloc)[..., None] + j - have[..., None]
    pop = torch.where(fresh, (F + R)[:, None, None] - 1 - k, 0)
    tables = torch.where(fresh, stack.gather(1, pop.reshape(G, -1)).view(G, B, -1), s["tables"])
    q_start = torch.cat([s["new_len"].new_zeros(1), s["new_len"].cumsum(0).int()])
    slots = _slots(s, s["max_rows"], tables, q_start)
    live = torch.arange(s["max_rows"], device="cuda")[:, None] < q_start[-1]
    return {"tables": tables, "free": stack, "free_count": (F + R - A).int(), "pages": need.int(),
            "q_start": q_start, "slots": torch.where(live, slots, s["slots"])}


def _plain_append(s):
    live = torch.arange(s["max_rows"], device="cuda") < s["q_start"][-1]
    dst = (s["base"][None] + s["slots"])[live].reshape(-1)
    s["k"][dst] = s["k_new"][live].reshape(-1, s["D"])
    s["v"][dst] = s["v_new"][live].reshape(-1, s["D"])
    return {"k": s["k"], "v": s["v"]}


def _plain_tree(s):
    B, Hkv, D, P, T = s["B"], s["Hkv"], s["D"], s["P"], s["T"]
    g = s["Hq"] // Hkv
    n = s["kv_len"].long()
    t = torch.arange(s["span"], device="cuda")
    live = t < (n + s["new_len"][:, None].long())[..., None]  # [B][Hkv][span]
    page = s["tables"][s["grp"][None, :, None], torch.arange(B, device="cuda")[:, None, None], (t // P)[None, None]].long()
    size, row = s["gsize"][None, :, None], s["row"][None, :, None]
    slot = (page * P + t % P) * size + row if s["layout"] == "token" else (page * size + row) * P + t % P
    at = torch.where(live, s["base"][None, :, None] + slot, 0)
    k, v = s["k"][at].float(), s["v"][at].float()
    i = torch.arange(T, device="cuda")
    rows = (s["q_start"][:-1, None].long() + i).clamp(max=s["max_rows"] - 1)  # [B][T]
    q = s["q"][rows].float().view(B, T, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, D)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    # a draft is seen by the rows whose mask has its bit
    d = torch.arange(32 * s["W"], device="cuda")
    bits = ((s["mask"][rows][..., d // 32] >> (d % 32)) & 1).bool()  # [B][T][32 W]
    draft = (t - n[..., None])[:, :, None].expand(B, Hkv, T, -1)
    seen = bits[:, None].expand(B, Hkv, T, -1).gather(3, draft.clamp(0, 32 * s["W"] - 1)) | (draft < 0)
    seen = seen & live[:, :, None]
    x = x.view(B, Hkv, T, g, -1).masked_fill_(~seen[:, :, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    x = (x / x.sum(-1, keepdim=True).clamp(min=1e-30)).view(B, Hkv, T * g, -1)
    o = (x @ v).view(B, Hkv, T, g, D).permute(0, 2, 1, 3, 4).reshape(B, T, s["Hq"], D)
    out = torch.zeros_like(s["out"])
    have = i[None] < s["new_len"][:, None]
    out[rows[have]] = o[have]
    return out


def _plain_commit(s):
    j = torch.arange(s["depth"], device="cuda")
    first, T = s["q_start"][:-1, None].long(), s["new_len"][:, None].long()
    dst = torch.minimum(j[None], T - 1)
    src = torch.where(j[None] < s["n_acc"][:, None], s["path"].long(), dst)  # what is not accepted stays
    to = (s["base"][None, None] + s["slots"][first + dst]).reshape(-1)
    of = (s["base"][None, None] + s["slots"][first + src]).reshape(-1)
    s["k"][to], s["v"][to] = s["k"][of], s["v"][of]
    return {"k": s["k"], "v": s["v"], "kv_len": s["kv_len"] + s["n_acc"][:, None]}


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "tree": _plain_tree,
                "commit": _plain_commit}[s["op"]](s)
    from paged_non_uniform_gb300 import kvx
    c, ws = s["cache"], s["ws"]
    if s["op"] == "tables":
        kvx.kvx_build_tables(c, s["kv_len"], s["new_len"], s["pages_in"], s["pages_out"], s["free_list"],
                             s["free_in"], s["free_out"], s["max_rows"], s["cu_out"], s["slots"], ws)
        return {"tables": s["tables"], "free": s["free"], "free_count": s["free_out"], "pages": s["pages_out"],
                "q_start": s["cu_out"], "slots": s["slots"]}
    if s["op"] == "append":
        kvx.kvx_append_kv(c, s["k_new"], s["v_new"], s["q_start"], s["slots"], s["max_rows"], ws)
        return {"k": s["k"], "v": s["v"]}
    if s["op"] == "tree":
        kvx.kvx_tree_attn(c, s["q"], s["q_start"], s["max_rows"], s["T"], s["kv_len"], s["mask"], s["scale"],
                          s["out"], ws)
        return s["out"]
    kvx.kvx_tree_commit(c, s["q_start"], s["slots"], s["max_rows"], s["path"], s["n_acc"], s["kv_len"],
                        s["kv_out"], ws)
    return {"k": s["k"], "v": s["v"], "kv_len": s["kv_out"]}


# ---------------------------------------------------------------- the work of a pass
def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    kv, new, held, need = _lengths(case)
    N, G = int(new.sum()), len(_sizes(case))
    if case["op"] == "tables":
        # lengths, counts in and out, moved page ids read and written, the slot map
        moved = int(np.abs(need - held).sum())
        return {"bytes": 4 * B * Hkv + 8 * G * B + 8 * B + 8 * moved + 8 * N * Hkv, "flops": 0}
    if case["op"] == "append":
        return {"bytes": N * Hkv * (8 + 4 * D * es), "flops": 0}
    if case["op"] == "commit":
        # the mean depth of a random node of a random recursive tree of T drafts is about ln T
        a = float(np.minimum(12.0, 0.6 + np.log(new)).mean())
        return {"bytes": B * Hkv * (a * 4 * D * es + 8 * a + 8) + 4 * B * (a + 2), "flops": 0}
    tokens = kv.sum(1) + Hkv * new  # of all heads
    return {"bytes": int(tokens.sum()) * 2 * D * es + N * Hq * D * (es + 4) + 4 * N * ((case["tmax"] + 31) // 32)
            + 4 * B * (Hkv + 1), "flops": 4 * D * (Hq // Hkv) * int((tokens * new).sum())}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits or in whole numbers. The table
    call's outputs are whole numbers and the copies of append and commit move bits, so only the attention's
    outputs have a 64-bit value of their own; the copies' are the rows themselves."""
    global own
    if case["op"] == "tables":
        return None
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    B, Hkv, D, P = s["B"], s["Hkv"], s["D"], s["P"]
    grp, row = s["head_group"], s["row"].cpu().numpy()
    n, cu, tables = s["kv_len"].cpu().numpy(), s["q_start"].cpu().numpy(), s["tables"].cpu().numpy()

    def where(b, h, t):
        g = grp[h]
        page = tables[g, b, t // P].astype(np.int64)
        if s["layout"] == "token":
            return s["base_g"][g] + (page * P + t % P) * s["sizes"][g] + row[h]
        return s["base_g"][g] + (page * s["sizes"][g] + row[h]) * P + t % P

    if case["op"] == "tree":
        gq = s["Hq"] // Hkv
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        masks = s["mask"].cpu().numpy().view(np.uint32)
        for b in range(B):
            T = int(cu[b + 1] - cu[b])
            bit = np.array([[(int(masks[cu[b] + i, j // 32]) >> (j % 32)) & 1 for j in range(T)] for i in range(T)])
            hide = torch.from_numpy(bit == 0).cuda()[:, None]
            for h in range(Hkv):
                m = int(n[b, h])
                at = torch.from_numpy(where(b, h, np.arange(m + T))).cuda()
                k, v = s["k"][at].double(), s["v"][at].double()
                q = s["q"][cu[b]:cu[b + 1], h * gq:(h + 1) * gq].double()
                x = torch.einsum("tgd,ld->tgl", q, k) / math.sqrt(D)
                x[:, :, m:] = x[:, :, m:].masked_fill(hide, -math.inf)
                out[cu[b]:cu[b + 1], h * gq:(h + 1) * gq] = torch.einsum("tgl,ld->tgd", torch.softmax(x, -1), v)
        return out
    dst, src = [], []
    if case["op"] == "append":
        k_new, v_new = s["k_new"].reshape(-1, Hkv, D), s["v_new"].reshape(-1, Hkv, D)
        for b in range(B):
            t = np.arange(cu[b + 1] - cu[b])
            for h in range(Hkv):
                at = torch.from_numpy(where(b, h, n[b, h] + t)).cuda()
                s["k"][at], s["v"][at] = k_new[cu[b]:cu[b + 1], h], v_new[cu[b]:cu[b + 1], h]
        return {"k": s["k"], "v": s["v"]}
    path, acc = s["path"].cpu().numpy(), s["n_acc"].cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            dst.append(where(b, h, n[b, h] + np.arange(acc[b])))
            src.append(where(b, h, n[b, h] + path[b, :acc[b]].astype(np.int64)))
    dst, src = torch.from_numpy(np.concatenate(dst)).cuda(), torch.from_numpy(np.concatenate(src)).cuda()
    s["k"][dst], s["v"][dst] = s["k"][src].clone(), s["v"][src].clone()
    return {"k": s["k"], "v": s["v"], "kv_len": None}
