"""Refusals of the calls that keep a cache within a memory budget, what their binding checks, rules of their
sources, and their references by hand (host only; made-up device addresses serve)."""
import os

import numpy as np
import pytest

from test_cache_cpu import A, OnDevice, kvx, make, refused  # noqa: F401
from test_sources_cpu import CSRC, kernels

Q4 = 4
WINDOW = dict(q=A, q_start=A, max_rows=4, max_q=2, kv_len=A, sinks=A, window=A, scale=0.0, out=A, weights=None,
              workspace=A, workspace_bytes=1 << 40, stream=0)
READ = dict(q_start=A, slots=A, max_rows=4, k_out=A, v_out=A, workspace=A, workspace_bytes=256, stream=0)
EVICT = dict(kv_len=A, budget=A, sinks=1, recent=2, weights=[A, A], weights_out=[A, A], kv_len_out=A, workspace=A,
             workspace_bytes=1 << 40, stream=0)


def test_q4_caches(kvx):
    make(kvx, dtype=Q4).destroy()
    refused(kvx, kvx.KVX_EUNSUPPORTED, make, kvx, dtype=Q4, layout=1)
    for dtype in (2, 3, 5, -1):
        refused(kvx, kvx.KVX_EUNSUPPORTED, make, kvx, dtype=dtype)
    c = make(kvx, dtype=Q4)
    U = kvx.KVX_EUNSUPPORTED
    refused(kvx, U, kvx.kvx_tree_attn_workspace_bytes, c, 4)
    refused(kvx, U, kvx.kvx_tree_attn, c, A, A, 4, 2, A, None, 0.0, A, A, 1 << 40, 0)
    refused(kvx, U, kvx.kvx_tree_commit, c, A, A, 4, A, A, A, A, A, 2, 256, 0)
    refused(kvx, U, kvx.kvx_plan_create, 1, 4, 1, 128, 16, 1, Q4, [[64]], [64], [0], num_ctas=4)


@pytest.mark.parametrize("name,good,changes", [
    ("kvx_window_attn", WINDOW, [dict(max_rows=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(q=A + 8),
                                 dict(out=A + 4), dict(sinks=A + 2), dict(window=A + 1), dict(workspace=A + 64),
                                 dict(workspace_bytes=255), dict(weights=[A]),
                                 dict(weights=[A, None]), dict(weights=[A, A + 2])]),
    ("kvx_read_kv", READ, [dict(max_rows=-1), dict(k_out=A + 8), dict(v_out=A + 2), dict(workspace_bytes=0),
                           dict(workspace=A + 128), dict(slots=A + 4), dict(q_start=A + 2)]),
    ("kvx_evict", EVICT, [dict(sinks=-1), dict(recent=-1), dict(weights=[A]), dict(weights_out=[A, None]),
                          dict(weights=[A, A + 1]), dict(weights_out=[A, 2 * A]), dict(workspace_bytes=1024),
                          dict(workspace=A + 8), dict(kv_len=A + 2), dict(budget=A + 1), dict(kv_len_out=A + 2)]),
])
@pytest.mark.parametrize("dtype", [0, 1, Q4])
def test_argument_refusals(kvx, dtype, name, good, changes):
    c, call = make(kvx, dtype=dtype), getattr(kvx, name)
    for change in changes:
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, **change})
    for key in good:  # every pointer is needed, but the windows
        if good[key] == A and key not in ("workspace", "sinks", "window"):
            refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, key: 0})


def test_ranges(kvx):
    c = make(kvx)
    for max_q in (0, -1, kvx.KVX_MAX_TREE + 1):
        refused(kvx, kvx.KVX_ERANGE, kvx.kvx_window_attn, c, **{**WINDOW, "max_q": max_q})
        refused(kvx, kvx.KVX_ERANGE, kvx.kvx_window_attn_workspace_bytes, c, max_q, False)
    refused(kvx, kvx.KVX_ERANGE, kvx.kvx_window_attn, c, **{**WINDOW, "max_rows": (1 << 30) + 1})
    refused(kvx, kvx.KVX_ERANGE, kvx.kvx_read_kv, c, **{**READ, "max_rows": (1 << 30) + 1})
    assert kvx.lib.kvx_window_attn_workspace_bytes(c.handle, 2, 2, None) == kvx.KVX_EINVAL
    # page tables for more than 2^32 chunks of 64 tokens
    big = make(kvx, B=4096, Hq=64, Hkv=64, G=1, hg=(0,) * 64, pages=(9,), stride=(1 << 16,), P=64)
    refused(kvx, kvx.KVX_ERANGE, kvx.kvx_evict_workspace_bytes, big)
    refused(kvx, kvx.KVX_ERANGE, kvx.kvx_evict, big, **{**EVICT, "weights": [A], "weights_out": [A]})


def test_row_strides(kvx):
    for dtype, item in ((0, 4), (1, 2), (Q4, 2)):
        c = make(kvx, dtype=dtype)
        for stride in (2 * 64 - 16 // item, 2 * 64 + 1, -128, 0, 2 ** 40 // item):
            for k, v in ((stride, 128), (128, stride)):
                assert kvx.lib.kvx_read_kv(c.handle, A, A, 4, A, k, A, v, A, 256, None) == kvx.KVX_EINVAL
        for stride in (8 * 64 - 16 // item, 8 * 64 + 1):
            assert kvx.lib.kvx_window_attn(c.handle, A, stride, A, 4, 2, A, None, None, 0.0, A, None, A, 1 << 40,
                                           None) == kvx.KVX_EINVAL


def test_null_cache(kvx):
    c = make(kvx)
    c.destroy()
    for name, good in (("kvx_window_attn", WINDOW), ("kvx_read_kv", READ), ("kvx_evict", EVICT)):
        refused(kvx, kvx.KVX_EINVAL, getattr(kvx, name), c, **good)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_window_attn_workspace_bytes, c, 4, False)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_evict_workspace_bytes, c)


def test_tensors_of_another_device(kvx):
    pytest.importorskip("torch")
    E = kvx.KVX_EINVAL
    c = make(kvx, kp=[OnDevice(1), A], tables=[A, OnDevice(1)])
    c.current_device = lambda: 0  # another device is current
    for name, good in (("kvx_window_attn", WINDOW), ("kvx_read_kv", READ), ("kvx_evict", EVICT)):
        refused(kvx, E, getattr(kvx, name), c, **good)
    c.pools_fit, c.current_device = True, lambda: 1
    for name, good, keys in (("kvx_window_attn", WINDOW, ("q_start", "kv_len", "sinks", "window", "out", "q")),
                             ("kvx_read_kv", READ, ("q_start", "slots", "k_out", "v_out")),
                             ("kvx_evict", EVICT, ("kv_len", "budget", "kv_len_out"))):
        for key in keys:
            refused(kvx, E, getattr(kvx, name), c, **{**good, key: OnDevice(0)})
    refused(kvx, E, kvx.kvx_evict, c, **{**EVICT, "weights": [A, OnDevice(0)]})
    refused(kvx, E, kvx.kvx_window_attn, c, **{**WINDOW, "weights": [OnDevice(0), A]})


def test_binding_checks_sizes_and_types(kvx):
    torch = pytest.importorskip("torch")
    from test_cache_binding_cpu import Dev
    E = kvx.KVX_EINVAL
    rows = 9 * 16  # of a group: one head
    good_pool = lambda **k: Dev(rows * 36, dtype=torch.uint8, **k)  # noqa: E731  (D 64: 36 bytes a row)
    c = make(kvx, dtype=Q4, kp=[good_pool()] * 2, vp=[good_pool()] * 2, tables=[Dev(2, 4)] * 2)
    c.current_device = lambda: 1
    assert c.pools_fit
    for bad in (Dev(rows * 36 - 1, dtype=torch.uint8), Dev(rows * 36, dtype=torch.bfloat16),
                good_pool(contiguous=False)):
        s = make(kvx, dtype=Q4, kp=[bad] + [good_pool()], vp=[good_pool()] * 2, tables=[Dev(2, 4)] * 2)
        s.current_device = lambda: 1
        for name, good in (("kvx_window_attn", WINDOW), ("kvx_read_kv", READ), ("kvx_evict", EVICT)):
            refused(kvx, E, getattr(kvx, name), s, **good)
    for bad in (Dev(rows - 1, dtype=torch.float32), Dev(rows, dtype=torch.int32),
                Dev(rows, dtype=torch.float32, contiguous=False), Dev(rows, dtype=torch.bfloat16)):
        refused(kvx, E, kvx.kvx_evict, c, **{**EVICT, "weights": [bad, A]})
        refused(kvx, E, kvx.kvx_evict, c, **{**EVICT, "weights_out": [A, bad]})
        refused(kvx, E, kvx.kvx_window_attn, c, **{**WINDOW, "weights": [A, bad]})
    refused(kvx, E, kvx.kvx_window_attn, c, **{**WINDOW, "sinks": Dev(1)})
    refused(kvx, E, kvx.kvx_window_attn, c, **{**WINDOW, "window": Dev(2, dtype=torch.int64)})
    refused(kvx, E, kvx.kvx_evict, c, **{**EVICT, "budget": Dev(3)})
    refused(kvx, E, kvx.kvx_read_kv, c, **{**READ, "k_out": Dev(4, 128, dtype=torch.float32)})
    refused(kvx, E, kvx.kvx_read_kv, c, **{**READ, "v_out": Dev(3, 128, dtype=torch.bfloat16)})


def test_no_rows_need_no_row_arrays(kvx):
    c = make(kvx)
    kvx.kvx_read_kv(c, A, None, 0, None, None, A, 256, 0)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_read_kv, c, A, None, 1, None, None, A, 256, 0)


def test_page_writers_hold_their_dependents_back():
    """A decode call with early loads reads pages before its dependency wait: kernels that write them neither
    release their dependents early nor finish before their writes are performed."""
    rows, evict = kernels("q4_rows.cu"), kernels("evict.cu")
    assert set(rows) == {"q4_append_kernel", "read_kernel"}
    assert set(evict) == {"evict_select_kernel", "evict_move_kernel"}
    for body, last in ((rows["q4_append_kernel"], "g.v + po) ="), (evict["evict_move_kernel"], "write(before,")):
        assert "pdl_launch_dependents" not in body
        assert "__threadfence();" in body[body.rindex(last):]
    assert "grp.k" not in evict["evict_select_kernel"] and "grp.v" not in evict["evict_select_kernel"]


@pytest.mark.parametrize("source", ["q4_rows.cu", "evict.cu", "window_mma.cuh", "window_simt.cu", "window_split.cuh",
                                    "window_weigh.cu"])
def test_dependents_read_with_ordinary_loads(source):
    """The non-coherent path is for memory that nobody writes while the grid runs."""
    text = open(os.path.join(CSRC, source)).read()
    assert "__ldg(" not in text and "ld.global.nc" not in text


def test_reference_quantisation_by_hand():
    from budget_cases import pack_pool, quantise, unpack_pool, values
    x = np.zeros((8, 64), np.float32)
    x[0, :3] = 30, 2, 1                     # step 2: codes 15, 1, tie 0.5 -> 0
    x[1, :4] = -15, 15, 1, -1               # step 2, lo -15: 0, 15, 8, 7 and zeros tie 7.5 -> 8
    x[2] = 3                                # constant
    x[3, 7] = np.nan
    codes, step, lo = quantise(x)
    assert step[:4, 0].tolist() == [2, 2, 0, 0] and lo[:3, 0].tolist() == [0, -15, 3] and np.isnan(lo[3, 0])
    assert codes[0, :4].tolist() == [15, 1, 0, 0] and codes[1, :5].tolist() == [0, 15, 8, 7, 8]
    assert values(codes, step, lo)[2].tolist() == [3.0] * 64 and np.isnan(values(codes, step, lo)[3]).all()
    buf = pack_pool(codes, step, lo, 8)
    assert buf.size == 8 * 36 and buf[:2].tolist() == [15 | 1 << 4, 0]
    assert buf[8 * 32:8 * 32 + 4].tolist() == [0x00, 0x40, 0, 0]  # step 2.0, lo 0.0
    again = unpack_pool(buf, 64, 8)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(again, (codes, step, lo)))
    # a row of 128: word 1 (elements 8 .. 15) is stored at place 2, word 8 (64 .. 71) at place 1
    y = np.zeros((8, 128), np.uint8)
    y[0, 8], y[0, 64] = 5, 9
    buf = pack_pool(y, np.ones((8, 2), np.float32), np.zeros((8, 2), np.float32), 8)
    assert buf[8] == 5 and buf[4] == 9


def test_reference_eviction_by_hand():
    from budget_cases import ref_evict
    w = [0, 9, 1, 5, 5, 5, 2, 0, 0]
    assert ref_evict(w, 9, 5, 1, 1).tolist() == [0, 1, 3, 4, 8]
    assert ref_evict(w, 9, 9, 1, 1).tolist() == list(range(9))
    assert ref_evict(w, 9, 0, 1, 1).tolist() == []
    assert ref_evict(w, 9, 2, 4, 5).tolist() == [7, 8]         # recent before sinks
    assert ref_evict(w, 9, 3, 4, 1).tolist() == [0, 1, 8]
    w = [np.nan, -np.inf, np.nan, -0.0, 0.0]
    assert ref_evict(w, 5, 3, 0, 0).tolist() == [1, 3, 4]
    assert ref_evict(w, 5, 1, 0, 0).tolist() == [3]
