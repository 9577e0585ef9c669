"""Accuracy of tree attention's sums over long heads, with exact weights."""
import numpy as np
import pytest
import torch

from paged_non_uniform_gb300 import kvx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g,T", [(128, 4, 16), (64, 8, 3), (128, 5, 30)])
def test_long_sums_leave_tensor_memory_in_time(D, g, T):
    """64 heads of 400,000 tokens are about 650 tiles a block (more where a head has two row groups): a sum
    that stayed in the tensor cores, which truncate, is off by 3e-4 to 6e-4.

    The queries are zero, so that every weight is exactly 1 and its residual 0, and the normaliser is a
    whole number below 2^24 in each piece: only the weighted sums round. The values are positive and
    spread over 16 binary orders, so that their sums need more bits than fp32 has. u = 2^-24:
      * between two folds, 16 tiles make 8 additions of 16 products each to an output element (those of
        the residuals add 0), each truncated by at most 2u of the sum so far: 128 * 2u of the final sum
      * folds: one fp32 fma each, at most ceil(tiles / 16) + 1 of an item, of which no block has more
        than the tiles of its part, 64 heads * row groups * 3126 tiles / 304 blocks + 1
      * merge: at most 8 pieces of a head, each with a weight of 1, in sum and normaliser; the
        reciprocal and the product with it: 2 * 8 + 3 u
    """
    B, Hkv, P, n, pages = 8, 8, 128, 400_000, 96
    gen = torch.Generator(device="cuda").manual_seed(D + T)
    i32 = dict(dtype=torch.int32, device="cuda")
    stride = -(-(n + T) // P)
    table = torch.randint(0, pages, (B, stride), generator=gen, **i32)
    k = torch.empty(pages * Hkv * P, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    v = torch.exp2(-16 * torch.rand(pages * Hkv * P, D, generator=gen, device="cuda")).bfloat16()
    cache = kvx.Cache(B, Hkv * g, Hkv, D, P, 1, kvx.KVX_BF16, [0] * Hkv, [k], [v], [pages], [table], [stride])
    q = torch.zeros(B * T, Hkv * g, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B * T, Hkv * g, D, device="cuda")
    ws = torch.zeros(kvx.kvx_tree_attn_workspace_bytes(cache, T) // 4, **i32)
    kvx.kvx_tree_attn(cache, q, torch.arange(B + 1, **i32) * T, B * T, T, torch.full((B, Hkv), n, **i32), None,
                      0.0, out, ws)
    torch.cuda.synchronize()
    assert kvx.kvx_workspace_status(ws) == 0
    # the mean of the values that a row sees: whole pages by their counts, then the last keys one by one
    vd = v.double().view(pages, Hkv, P, D)
    page_sum = vd.sum(2)
    whole = n // P
    groups = 1 if T * g <= 128 else 2
    u = 2.0 ** -24
    tiles = -(-64 * groups * stride // 304) + 1
    tol = (128 * 2 + -(-tiles // 16) + 1 + 2 * 8 + 3) * u
    worst = 0.0
    for b in range(B):
        count = torch.bincount(table[b, :whole].long(), minlength=pages).double()
        base = torch.einsum("p,phd->hd", count, page_sum)
        t = torch.arange(whole * P, n + T, device="cuda")
        tail = vd[table[b].long()[t // P], :, t % P].cumsum(0)  # [keys][Hkv][D]
        for i in range(T):
            want = (base + tail[n + i - whole * P]) / (n + i + 1)
            got = out[b * T + i].double().view(Hkv, g, D)
            worst = max(worst, float(((got - want[:, None]) / want[:, None]).abs().max()))
    assert worst <= tol, (worst, tol)
    print(f"largest relative error {worst:.2e} of {tol:.2e}")
