"""Cases of the operators that keep a paged cache within a memory budget: attention with a sliding
window and sink tokens, the same with the accumulation of each cached token's attention weight, eviction
by those weights, and caches held in 4 bits (rows quantised into their pages and read back, attention over
them).

A case is a dict of plain values:
  op        "window", "weigh", "q4", "rows" or "evict"
  B, Hq, Hkv, D, P, groups, layout, dtype   the cache's shape; `groups` counts the KV heads of each
            head group, `layout` is "head" or "token" (page layout), `dtype` "bf16", "f32" or "q4"
  lo, hi    cached tokens of a sequence, log-uniform in [lo, hi]
  keep      "full" (every head keeps all), "mix" (a quarter of the heads keep all, the others 10-50 %) or
            "half" (half keep all, half 12.5 %): tokens cached, for "evict" tokens that stay
  tmin, tmax   new rows of a sequence, uniform in [tmin, tmax] (log-uniform for "rows")
  sinks, window, wide   tokens seen by heads with a window (window 0: no head has one); the first `wide`
            heads see everything. For "evict" the first tokens and the last tokens that stay in any case

`run` in its plain form is elementary torch in 32 bits; with `own` it makes the library's calls.
"""
from __future__ import annotations

import math
import zlib

import numpy as np
import torch

own = False

ALL = 2 ** 31 - 1  # the window of a head that sees everything


# ---------------------------------------------------------------- the cases
def listed():
    tiny = dict(B=2, Hq=4, Hkv=2, D=64, P=16, groups="1,1", layout="head", dtype="f32")
    q4b = dict(B=16, Hq=32, Hkv=8, D=128, P=16, groups="2,3,3", layout="head", dtype="bf16")
    q32 = dict(Hq=40, Hkv=8, D=128, P=32, groups="2,2,2,2", layout="head", dtype="bf16")
    rm = dict(Hq=32, Hkv=8, D=128, P=16, groups="8", layout="token", dtype="bf16")
    no = dict(sinks=0, window=0, wide=0)
    return [
        # the smallest call: two short fp32 sequences, 4 sinks and 16 recent tokens in one of two heads
        dict(name="window_tiny", op="window", lo=37, hi=100, keep="full", tmin=1, tmax=3, sinks=4, window=16, wide=1,
             **tiny),
        # one interactive user, one token, every head streaming over 1024 tokens
        dict(name="window_one_user", op="window", lo=1500, hi=2500, keep="full", tmin=1, tmax=1, sinks=4, window=1024,
             wide=0, **{**q4b, "B": 1}),
        # the decode benchmark's layer: a quarter of the heads see all, the others stream over 4096 tokens
        dict(name="window_step", op="window", lo=8192, hi=32768, keep="full", tmin=1, tmax=1, sinks=4, window=4096,
             wide=2, **q4b),
        # a step with up to 8 drafts a sequence, 5 query heads a KV head, odd window, ragged lengths
        dict(name="window_drafts", op="window", B=32, lo=1000, hi=32000, keep="full", tmin=1, tmax=8, sinks=5,
             window=1000, wide=4, **q32),
        # a decode step that accumulates weights for a later eviction, unequal budgets
        dict(name="weigh_step", op="weigh", lo=8192, hi=32768, keep="mix", tmin=1, tmax=1, **no, **q4b),
        # the last 32 rows of a prompt vote on what stays of it
        dict(name="weigh_observe", op="weigh", B=4, lo=8000, hi=16000, keep="full", tmin=32, tmax=32, **no, **rm),
        # the decode benchmark's layer with a cache in 4 bits
        dict(name="q4_step", op="q4", lo=8192, hi=32768, keep="mix", tmin=1, tmax=1, **no, **{**q4b, "dtype": "q4"}),
        # long context in 4 bits: 8 x 122k tokens
        dict(name="q4_long", op="q4", lo=121000, hi=123000, keep="full", tmin=1, tmax=1, **no,
             **{**q4b, "dtype": "q4", "B": 8, "groups": "8"}),
        # a step's rows quantised into their pages and read back
        dict(name="rows_step", op="rows", lo=512, hi=2048, keep="mix", tmin=16, tmax=16, **no, **{**q4b, "dtype": "q4"}),
        # prompts of a prefill quantised into pages, and read back as the attention over the prompt sees them
        dict(name="rows_prompts", op="rows", lo=0, hi=0, keep="full", tmin=64, tmax=1024, **no,
             **{**q4b, "dtype": "q4", "B": 128}),
        # prompts cut down to unequal budgets after the prefill
        dict(name="evict_prompts", op="evict", lo=8192, hi=32768, keep="mix", tmin=0, tmax=0, sinks=4, window=64, wide=0,
             **q4b),
        # a periodic eviction: 64 sequences at 10 to 50 % budgets of short histories, token-major blocks
        dict(name="evict_step", op="evict", B=64, lo=1000, hi=2500, keep="half", tmin=0, tmax=0, sinks=4, window=32,
             wide=0, **rm),
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
    op = rng.choice(["window", "window", "weigh", "q4", "q4", "rows", "evict"])
    c = dict(op=op, Hq=Hkv * g, Hkv=Hkv, D=rng.choice([64, 128, 128]), P=rng.choice([8, 16, 16, 32, 64, 128]),
             groups=",".join(map(str, cuts)), layout=rng.choice(["head", "token"]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), keep=rng.choice(["full", "mix", "half"]),
             sinks=0, window=0, wide=0)
    if op in ("q4", "rows"):
        c.update(dtype="q4", layout="head")
    if op == "rows":
        c["lo"], c["hi"] = 0, 0
        c["tmax"] = _log(rng, 1, 2000)
        c["B"] = _log(rng, 1, max(1, min(256, 30000 // c["tmax"])))
        c["tmin"] = _log(rng, 1, c["tmax"])
        return c
    small = c["dtype"] == "f32"  # fp32 caches are the small end of the range
    c["hi"] = _log(rng, 20, 6000 if small else 60000)
    c["lo"] = _log(rng, max(1, c["hi"] // 20), c["hi"])
    if op == "evict":
        c["tmin"] = c["tmax"] = 0
        c["B"] = _log(rng, 1, max(1, min(64, 400000 // c["hi"])))
        c["sinks"], c["window"] = rng.choice([0, 1, 4, 17]), _log(rng, 1, 200)
        return c
    c["tmax"] = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, min(128, (64 if small else 256) // g)))
    c["tmin"] = _log(rng, 1, c["tmax"])
    most = 16000 if small else min(500000, 60000000 // (c["tmax"] * g))
    c["B"] = _log(rng, 1, max(1, min(64, most // c["hi"])))
    if op == "window" or rng.random() < 0.3:
        c["sinks"], c["window"], c["wide"] = rng.choice([0, 1, 4, 17, 200]), _log(rng, 1, 10000), rng.randint(0, Hkv)
    return c


# ---------------------------------------------------------------- inputs
def _sizes(case):
    return [int(x) for x in case["groups"].split(",")]


def _lengths(case):
    """What the case fixes and a seed only reorders: cached tokens a head [B][Hkv], new rows [B], and for
    "evict" the tokens that stay [B][Hkv] (heads by falling budget)."""
    r = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    B, Hkv = case["B"], case["Hkv"]
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
    if case["op"] == "rows":
        new = np.round(np.exp(r.uniform(math.log(case["tmin"]), math.log(case["tmax"]), B))).astype(np.int32)
    else:
        new = r.integers(case["tmin"], case["tmax"] + 1, B).astype(np.int32)
    if case["op"] == "evict":
        return np.repeat(L[:, None], Hkv, 1).astype(np.int32), new, kv
    return kv, new, kv


def _windows(case):
    """Window of each head (heads by falling budget)."""
    w = np.full(case["Hkv"], ALL, np.int64)
    if case["window"]:
        w[case["wide"]:] = case["window"]
    return w


def _row_bytes(case):
    return {"bf16": 2 * case["D"], "f32": 4 * case["D"], "q4": case["D"] // 2 + case["D"] // 16}[case["dtype"]]


def _q4_pack(x):
    """(codes uint8 [..., D / 2], parameters uint8 [..., D / 16]) of rows [..., D]: every 64 elements have a
    bf16 step and a bf16 minimum, an element is 4 bits. Eight bytes hold eight elements of the first 64 and
    eight of the second (D 64: four bytes hold eight elements), lowest bits first."""
    D = x.shape[-1]
    f = x.float().unflatten(-1, (D // 64, 64))
    lo = f.amin(-1)
    step = ((f.amax(-1) - lo) / 15).bfloat16()
    s = step.float()[..., None]
    c = ((f - lo[..., None]) / torch.where(s == 0, 1.0, s)).round().clamp(max=15).to(torch.uint8)
    c = c.unflatten(-1, (8, 4, 2)).movedim(-4, -3)  # [..., 8 units, halves, 4 bytes, 2]
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-3), torch.stack([step, lo.bfloat16()], -1).view(torch.uint8).flatten(-2)


def _q4_views(pool, D, P):
    """The codes [blocks][P][D / 2] and parameters [blocks][P][D / 16] of a pool: a head's P rows of a page are a
    block."""
    b = pool.view(-1, P * (D // 2 + D // 16))
    return b[:, : P * D // 2].unflatten(1, (P, D // 2)), b[:, P * D // 2:].unflatten(1, (P, D // 16))


def _q4_values(pool, at, D, P):
    """Rows `at` of a 4-bit pool as the fp32 values that they stand for."""
    codes, params = _q4_views(pool, D, P)
    c = codes[at // P, at % P].unflatten(-1, (8, D // 64, 4))
    c = torch.stack([c & 15, c >> 4], -1).movedim(-3, -4).flatten(-3)  # [..., halves, 64]
    p = params[at // P, at % P].view(torch.bfloat16).unflatten(-1, (D // 64, 2)).float()
    return (p[..., 1:] + p[..., :1] * c).flatten(-2)


def prepare(case, seed):
    r = np.random.default_rng([int(seed), 23])
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) + 1)
    op, B, Hq, Hkv, D, P = case["op"], case["B"], case["Hq"], case["Hkv"], case["D"], case["P"]
    q4 = case["dtype"] == "q4"
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    sizes = _sizes(case)
    G = len(sizes)

    kv_len, new_len, stay = _lengths(case)
    seqs, heads = r.permutation(B), r.permutation(Hkv)
    kv_len, new_len, stay = kv_len[seqs][:, heads], new_len[seqs], stay[seqs][:, heads]
    grp = np.repeat(np.arange(G, dtype=np.int32), sizes)[heads]  # heads of like budgets share a group
    row = np.array([np.sum(grp[:h] == grp[h]) for h in range(Hkv)])
    need = np.stack([-(-(kv_len[:, grp == g].max(1) + new_len) // P) for g in range(G)])
    N = int(new_len.sum())
    max_rows = N + 3  # the caller's row buffers are a little larger than this step's rows
    stride = int(max(need.max(), 1)) + 2
    pages = int(need.sum(1).max()) + 5
    tables = np.full((G, B, stride), -1, np.int32)
    for g in range(G):
        tables[g][np.arange(stride)[None] < need[g][:, None]] = r.permutation(pages)[: need[g].sum()]
    cu = np.concatenate([[0], np.cumsum(new_len)]).astype(np.int32)

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    def normal(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=gen)

    s = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, G=G, sizes=sizes, layout=case["layout"], max_rows=max_rows,
             pages=pages, stride=stride, tables=up(tables), kv_len=up(kv_len), new_len=up(new_len), q4=q4,
             q_start=up(cu), grp=up(grp.astype(np.int64)), row=up(row.astype(np.int64)), rb=_row_bytes(case),
             gsize=up(np.array(sizes)[grp].astype(np.int64)), head_group=grp, case=dict(case))
    # one buffer holds the pools of all groups, [pages][heads of the group][P][D] one after the other
    base = np.concatenate([[0], np.cumsum([pages * n * P for n in sizes])])
    s["base_g"] = base
    s["base"] = up(base[:-1][grp].astype(np.int64))
    total = int(base[-1])
    if q4:
        for name in ("k", "v"):
            pool = torch.empty(total * s["rb"], dtype=torch.uint8, device=dev)
            codes, params = _q4_views(pool, D, P)
            for i in range(0, codes.shape[0], 1 << 16):  # (in parts: small temporaries)
                codes[i:i + (1 << 16)], params[i:i + (1 << 16)] = _q4_pack(normal(*codes[i:i + (1 << 16)].shape[:2], D))
            s[name] = pool
    else:
        s["k"], s["v"] = normal(total, D), normal(total, D)
    if op == "rows":
        # K and V of the new rows as a fused projection leaves them: slices of one row
        fused = normal(max_rows, (Hq + 2 * Hkv) * D)
        s["k_new"] = fused[:, Hq * D:(Hq + Hkv) * D]
        s["v_new"] = fused[:, (Hq + Hkv) * D:]
        s["k_out"] = torch.zeros((max_rows, Hkv * D), dtype=dt, device=dev)
        s["v_out"] = torch.zeros((max_rows, Hkv * D), dtype=dt, device=dev)
        s["slots"] = _slots(s)
    elif op == "evict":
        # what attention has left: a few tokens with most of the weight, some that were never looked at
        w = torch.exp(2 * normal(total, dtype=torch.float32) - 4)
        w[torch.rand(total, device=dev, generator=gen) < 0.1] = 0
        s.update(budget=up(stay), weights=w, weights_out=torch.zeros_like(w), kv_out=torch.zeros_like(s["kv_len"]),
                 sinks=case["sinks"], recent=case["window"], span=int(kv_len.max()), most=int(stay.max()))
    else:
        s.update(q=normal(max_rows, Hq, D), T=case["tmax"], out=torch.zeros((max_rows, Hq, D), device=dev),
                 span=int((kv_len + new_len[:, None]).max()), scale=1.0 / math.sqrt(D))
        s["sinks"] = torch.full((Hkv,), case["sinks"], dtype=torch.int32, device=dev)
        s["window"] = up(_windows(case)[heads].astype(np.int32))
        s["limited"] = bool(case["window"])
        if op == "weigh":
            s["weights"] = torch.rand(total, device=dev, generator=gen)
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program keeps from step to step: the cache handle and the workspace."""
    from paged_non_uniform_gb300 import kvx
    width = s["rb"] if s["q4"] else 1  # of a pool's row
    cut = s["base_g"]

    def parts(x, width=1):
        return [x[cut[g] * width:cut[g + 1] * width] for g in range(s["G"])]

    dtype = {"bf16": kvx.KVX_BF16, "f32": kvx.KVX_F32, "q4": kvx.KVX_Q4}[case["dtype"]]
    s["cache"] = kvx.Cache(s["B"], s["Hq"], s["Hkv"], s["D"], s["P"], s["G"], dtype, s["head_group"],
                           parts(s["k"], width), parts(s["v"], width), [s["pages"]] * s["G"],
                           [s["tables"][g] for g in range(s["G"])], [s["stride"]] * s["G"],
                           layout=kvx.KVX_LAYOUT_TOKEN_MAJOR if s["layout"] == "token" else kvx.KVX_LAYOUT_HEAD_MAJOR)
    nbytes = kvx.KVX_WS_HEADER_BYTES
    if s["op"] == "evict":
        nbytes = kvx.kvx_evict_workspace_bytes(s["cache"])
        s["w_in"], s["w_out"] = parts(s["weights"]), parts(s["weights_out"])
    elif s["op"] != "rows":
        nbytes = kvx.kvx_window_attn_workspace_bytes(s["cache"], s["T"], s["op"] == "weigh")
        s["w_in"] = parts(s["weights"]) if s["op"] == "weigh" else None
    s["ws"] = torch.zeros(-(-nbytes // 4), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plain forms
def _pool_rows(s, t):
    """Rows of the buffers that hold tokens t [B][Hkv][...] of every head."""
    P = s["P"]
    shape = (1, s["Hkv"]) + (1,) * (t.dim() - 2)
    b = torch.arange(s["B"], device="cuda").view((s["B"],) + (1,) * (t.dim() - 1))
    page = s["tables"][s["grp"].view(shape), b, t // P].long()
    n, r = s["gsize"].view(shape), s["row"].view(shape)
    slot = (page * P + t % P) * n + r if s["layout"] == "token" else (page * n + r) * P + t % P
    return s["base"].view(shape) + slot


def _slots(s):
    """Slot map: [max_rows][Hkv] pool rows of the new tokens (rows behind the last sequence: 0)."""
    q_start = s["q_start"].long()
    at = torch.arange(s["max_rows"], device="cuda")
    b = (torch.searchsorted(q_start, at, right=True) - 1).clamp(max=s["B"] - 1)
    live = (at < q_start[-1])[:, None]
    t = torch.where(live, s["kv_len"].long()[b] + (at - q_start[b])[:, None], 0)
    page = s["tables"][s["grp"][None], b[:, None], t // s["P"]].long()
    slot = (page * s["gsize"][None] + s["row"][None]) * s["P"] + t % s["P"]
    return torch.where(live, slot, 0)


def _plain_attention(s):
    B, Hkv, D, T = s["B"], s["Hkv"], s["D"], s["T"]
    g = s["Hq"] // Hkv
    n = s["kv_len"].long()
    t = torch.arange(s["span"], device="cuda")
    live = t < (n + s["new_len"][:, None].long())[..., None]  # [B][Hkv][span]
    at = _pool_rows(s, torch.where(live, t, 0))
    at = torch.where(live, at, at[..., :1])
    if s["q4"]:
        k, v = _q4_values(s["k"], at, D, s["P"]), _q4_values(s["v"], at, D, s["P"])
    else:
        k, v = s["k"][at].float(), s["v"][at].float()
    i = torch.arange(T, device="cuda")
    rows = (s["q_start"][:-1, None].long() + i).clamp(max=s["max_rows"] - 1)  # [B][T]
    have = i[None] < s["new_len"][:, None]
    q = s["q"][rows].float().view(B, T, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, D)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    pos = (n[..., None] + i)[..., None]  # [B][Hkv][T][1]
    seen = (t <= pos) & have[:, None, :, None]
    if s["limited"]:
        seen &= (t < s["sinks"].view(1, Hkv, 1, 1)) | (t > pos - s["window"].view(1, Hkv, 1, 1).long())
    x = x.view(B, Hkv, T, g, -1).masked_fill_(~seen[:, :, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (x.view(B, Hkv, T * g, -1) @ v).view(B, Hkv, T, g, D).permute(0, 2, 1, 3, 4).reshape(B, T, s["Hq"], D)
    out = torch.zeros_like(s["out"])
    out[rows[have]] = o[have]
    if s["op"] != "weigh":
        return out
    # new tokens start at zero
    w = torch.where(t < n[..., None], s["weights"][at], 0) + x.sum((2, 3))
    s["weights"][at[live]] = w[live]
    return {"out": out, "weights": s["weights"]}


def _plain_rows(s):
    D = s["D"]
    live = torch.arange(s["max_rows"], device="cuda") < s["q_start"][-1]
    at = (s["base"][None] + s["slots"])[live]
    out = {}
    for name in ("k", "v"):
        codes, params = _q4_views(s[name], D, s["P"])
        new = s[name + "_new"][live].view(-1, s["Hkv"], D)
        codes[at // s["P"], at % s["P"]], params[at // s["P"], at % s["P"]] = _q4_pack(new)
        rows = _q4_values(s[name], at, D, s["P"]).to(s[name + "_out"].dtype)
        s[name + "_out"][live] = rows.flatten(1)
        out[name] = s[name + "_out"]
    return out


def _plain_evict(s):
    n, m = s["kv_len"].long(), torch.minimum(s["kv_len"], s["budget"]).long()
    last = torch.minimum(m, torch.full_like(m, s["recent"]))
    first = torch.minimum(m - last, torch.full_like(m, s["sinks"]))
    t = torch.arange(s["span"], device="cuda")
    live = t < n[..., None]
    at = _pool_rows(s, torch.where(live, t, 0))
    w = torch.where(live, s["weights"][at], -math.inf)
    w = torch.where((t < first[..., None]) | ((t >= (n - last)[..., None]) & live), math.inf, w)
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., : s["most"]]  # of equal weights the lower index first
    stays = torch.arange(s["most"], device="cuda") < m[..., None]
    src = torch.where(stays, order, s["span"]).sort(-1).values
    to, of = at[..., : s["most"]][stays], at.gather(2, src.clamp(max=s["span"] - 1))[stays]
    s["k"][to], s["v"][to] = s["k"][of], s["v"][of]
    s["weights_out"][to] = s["weights"][of]
    return {"k": s["k"], "v": s["v"], "weights": s["weights_out"], "kv_len": m.int()}


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return {"rows": _plain_rows, "evict": _plain_evict}.get(s["op"], _plain_attention)(s)
    from paged_non_uniform_gb300 import kvx
    c, ws = s["cache"], s["ws"]
    if s["op"] == "rows":
        kvx.kvx_append_kv(c, s["k_new"], s["v_new"], s["q_start"], s["slots"], s["max_rows"], ws)
        kvx.kvx_read_kv(c, s["q_start"], s["slots"], s["max_rows"], s["k_out"], s["v_out"], ws)
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "evict":
        kvx.kvx_evict(c, s["kv_len"], s["budget"], s["sinks"], s["recent"], s["w_in"], s["w_out"], s["kv_out"], ws)
        return {"k": s["k"], "v": s["v"], "weights": s["weights_out"], "kv_len": s["kv_out"]}
    sinks, window = (s["sinks"], s["window"]) if s["limited"] else (None, None)
    kvx.kvx_window_attn(c, s["q"], s["q_start"], s["max_rows"], s["T"], s["kv_len"], sinks, window, s["scale"],
                        s["out"], s["w_in"], ws)
    return {"out": s["out"], "weights": s["weights"]} if s["op"] == "weigh" else s["out"]


# ---------------------------------------------------------------- the work of a pass
def work(case):
    B, Hq, Hkv, D, rb = case["B"], case["Hq"], case["Hkv"], case["D"], _row_bytes(case)
    kv, new, stay = _lengths(case)
    N = int(new.sum())
    if case["op"] == "rows":
        return {"bytes": N * Hkv * (8 + 2 * (rb + 4 * D)), "flops": 0}
    if case["op"] == "evict":
        n = np.minimum(kv, stay)
        moved = int(n[stay < kv].sum())  # nearly every row that stays gets another place
        return {"bytes": 4 * int(kv.sum() + n.sum()) + moved * 4 * rb + 12 * B * Hkv, "flops": 0}
    kv = kv.astype(np.int64)
    w = _windows(case)[None]
    first = np.maximum(kv - w + 1, 0)  # of the first row's window
    seen = np.minimum(first, case["sinks"]) + kv + new[:, None] - first  # keys that some row sees
    if case["tmin"] == 0:
        seen = np.where(new[:, None] > 0, seen, 0)
    es = 4 if case["dtype"] == "f32" else 2
    each = 0.0  # (row, key) pairs
    for i in range(int(new.max())):
        pos = kv + i
        a = np.maximum(pos - w + 1, 0)
        each += float(((np.minimum(a, case["sinks"]) + pos + 1 - a) * (new[:, None] > i)).sum())
    extra = 8 * int(seen.sum()) if case["op"] == "weigh" else 0
    return {"bytes": int(seen.sum()) * 2 * rb + N * Hq * D * (es + 4) + 4 * B * (Hkv + 1) + extra,
            "flops": int(4 * D * (Hq // Hkv) * each)}


# ---------------------------------------------------------------- 64-bit values
def _exact_q4(pool, at, D, P):
    """Rows `at` of a 4-bit pool in 64 bits, from the page format byte by byte."""
    block = P * (D // 2 + D // 16)
    word = torch.arange(D, device="cuda") // 8  # of the elements: 8 to a 32-bit word
    word = 2 * (word % 8) + word // 8 if D == 128 else word
    nib = torch.arange(D, device="cuda") % 8
    start = (at // P * block)[:, None]
    byte = pool[start + (at % P * (D // 2))[:, None] + 4 * word + nib // 2]
    code = (byte >> (4 * (nib % 2)).to(torch.uint8)) & 15
    at16 = (at // P * (block // 2) + P * D // 4 + at % P * (D // 32))[:, None] + 2 * (torch.arange(D, device="cuda") // 64)
    half = pool.view(torch.bfloat16)
    return half[at16 + 1].double() + half[at16].double() * code.double()


def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits or in whole numbers."""
    global own
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
        at = (page * P + t % P) * s["sizes"][g] + row[h] if s["layout"] == "token" else \
            (page * s["sizes"][g] + row[h]) * P + t % P
        return torch.from_numpy(s["base_g"][g] + at).cuda()

    if case["op"] == "rows":
        out = {}
        for name in ("k", "v"):
            x = s[name + "_new"].double().reshape(-1, Hkv, D // 64, 64)
            lo = x.min(-1, keepdim=True).values
            step = ((x.max(-1, keepdim=True).values - lo) / 15).float().bfloat16().double()
            val = (lo + step * ((x - lo) / step).round().clamp(0, 15)).reshape(-1, Hkv * D)
            val[int(cu[-1]):] = 0
            out[name] = val
        return out
    if case["op"] == "evict":
        budget = s["budget"].cpu().numpy()
        kv_out = np.minimum(n, budget)
        k, v, w, w_out = (s[x].clone() for x in ("k", "v", "weights", "weights_out"))
        for b in range(B):
            for h in range(Hkv):
                m, L = int(kv_out[b, h]), int(n[b, h])
                r = min(m, s["recent"])
                f = min(m - r, s["sinks"])
                at = where(b, h, np.arange(L))
                mid = w[at[f:L - r]].cpu().numpy().astype(np.float64)
                best = np.lexsort((np.arange(mid.size), -mid))[: m - r - f] + f
                src = np.sort(np.concatenate([np.arange(f), best, np.arange(L - r, L)]))
                src = torch.from_numpy(src).cuda()
                k[at[:m]], v[at[:m]], w_out[at[:m]] = s["k"][at[src]], s["v"][at[src]], w[at[src]]
        return {"k": k, "v": v, "weights": w_out, "kv_len": torch.from_numpy(kv_out)}
    gq = s["Hq"] // Hkv
    sinks, window = s["sinks"].cpu().numpy(), s["window"].cpu().numpy().astype(np.int64)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["op"] == "weigh" else None
    for b in range(B):
        T = int(cu[b + 1] - cu[b])
        for h in range(Hkv):
            m = int(n[b, h])
            at = where(b, h, np.arange(m + T))
            k, v = (_exact_q4(s[x], at, D, P) if s["q4"] else s[x][at].double() for x in ("k", "v"))
            q = s["q"][cu[b]:cu[b + 1], h * gq:(h + 1) * gq].double()
            x = torch.einsum("tgd,ld->tgl", q, k) / math.sqrt(D)
            for i in range(T):
                x[i, :, m + i + 1:] = -math.inf
                begin = m + i - int(window[h]) + 1
                if begin > sinks[h]:
                    x[i, :, int(sinks[h]):begin] = -math.inf
            p = torch.softmax(x, -1)
            out[cu[b]:cu[b + 1], h * gq:(h + 1) * gq] = torch.einsum("tgl,ld->tgd", p, v)
            if weights is not None:
                weights[at[m:]] = 0
                weights[at] += p.sum((0, 1))
    return {"out": out, "weights": weights} if weights is not None else out
