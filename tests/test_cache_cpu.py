"""Refusals of the cache calls (host checks; no device work is reached, so
made-up device addresses serve)."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def kvx():
    from paged_non_uniform_gb300 import build
    build.build()
    from paged_non_uniform_gb300 import kvx as k
    return k


A = 1 << 20  # a 16-byte aligned device address that is never read


def make(kvx, B=2, Hq=8, Hkv=2, D=64, P=16, G=2, dtype=1, hg=(0, 1), kp=None, vp=None, pages=(9, 9),
         tables=None, stride=(4, 4), layout=0):
    n = max(G, 1)
    return kvx.Cache(B, Hq, Hkv, D, P, G, dtype, list(hg), kp or [A] * n, vp or [A] * n, list(pages),
                     tables or [A] * n, list(stride), layout=layout)


def refused(kvx, status, call, *a, **k):
    with pytest.raises(kvx.KvxError) as e:
        call(*a, **k)
    assert e.value.status == status, (k, str(e.value))


def test_cache_create_refuses(kvx):
    make(kvx).destroy()
    E, U, R = kvx.KVX_EINVAL, kvx.KVX_EUNSUPPORTED, kvx.KVX_ERANGE
    for status, change in (
            (E, dict(B=0)), (U, dict(B=kvx.KVX_MAX_CACHE_SEQS + 1)), (E, dict(Hq=7)), (U, dict(Hq=18)),
            (U, dict(D=96)), (U, dict(P=12)), (U, dict(P=4)), (U, dict(P=256)), (U, dict(dtype=2)),
            (U, dict(layout=2)), (E, dict(hg=(0, 2))), (E, dict(hg=(0, -1))), (E, dict(hg=(0, 0))),
            (E, dict(hg=(0,))), (E, dict(pages=(9, 0))), (R, dict(pages=(9, 2 ** 31 - 1))),
            (E, dict(stride=(0, 4))), (R, dict(stride=(4, 1 << 28))), (E, dict(kp=[A, A + 8])),
            (E, dict(vp=[A, None])), (E, dict(tables=[A, None])), (E, dict(tables=[A, A + 2])),
            (E, dict(pages=(9,))), (E, dict(kp=[A]))):
        refused(kvx, status, make, kvx, **change)


def test_null_cache_is_refused(kvx):
    c = make(kvx)
    c.destroy()
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_tree_attn, c, A, A, 4, 2, A, None, 0.0, A, A, 1 << 30, 0)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_append_kv, c, A, A, A, A, 4, A, 256, 0)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_tree_attn_workspace_bytes, c, 4)


TABLES = dict(kv_len=A, new_len=A, pages_in=A, pages_out=2 * A, free_pages=[A, A], free_in=A,
              free_out=2 * A, max_rows=4, q_start=A, slots=A, workspace=A, workspace_bytes=256, stream=0)
APPEND = dict(k_new=A, v_new=A, q_start=A, slots=A, max_rows=4, workspace=A, workspace_bytes=256, stream=0)
TREE = dict(q=A, q_start=A, max_rows=4, max_q=2, kv_len=A, mask=None, scale=0.0, out=A, workspace=A,
            workspace_bytes=1 << 40, stream=0)
COMMIT = dict(q_start=A, slots=A, max_rows=4, path=A, n_acc=A, kv_len=A, kv_len_out=A, workspace=A,
              path_stride=2, workspace_bytes=256, stream=0)


@pytest.mark.parametrize("name,good,changes", [
    ("kvx_build_tables", TABLES, [dict(pages_out=A), dict(free_out=A), dict(max_rows=-1),
                                  dict(free_pages=[A]), dict(free_pages=[A, None]),
                                  dict(workspace_bytes=255), dict(workspace=A + 16), dict(slots=A + 4)]),
    ("kvx_append_kv", APPEND, [dict(max_rows=-1), dict(k_new=A + 8), dict(v_new=A + 2),
                               dict(workspace_bytes=0), dict(workspace=A + 128), dict(slots=A + 4)]),
    ("kvx_tree_attn", TREE, [dict(max_rows=-1), dict(scale=-1.0), dict(scale=float("nan")),
                             dict(scale=float("inf")), dict(q=A + 8), dict(out=A + 4), dict(mask=A + 2),
                             dict(workspace=A + 64), dict(workspace_bytes=255)]),
    ("kvx_tree_commit", COMMIT, [dict(max_rows=-1), dict(path_stride=0), dict(workspace_bytes=8),
                                 dict(workspace=A + 8), dict(slots=A + 4)]),
])
def test_argument_refusals(kvx, name, good, changes):
    c, call = make(kvx), getattr(kvx, name)
    for change in changes:
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, **change})
    for key in good:  # every pointer is needed, but the mask
        if good[key] == A and key != "workspace":
            refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, key: 0})


def test_tree_size_range(kvx):
    c = make(kvx)
    for max_q in (0, -1, kvx.KVX_MAX_TREE + 1):
        refused(kvx, kvx.KVX_ERANGE, kvx.kvx_tree_attn, c, **{**TREE, "max_q": max_q})
        refused(kvx, kvx.KVX_ERANGE, kvx.kvx_tree_attn_workspace_bytes, c, max_q)


def test_row_strides_are_checked(kvx):
    """Through the C ABI: a row stride below the row or not a multiple of 16 bytes."""
    for dtype, item in ((kvx.KVX_BF16, 2), (kvx.KVX_F32, 4)):
        c = make(kvx, dtype=dtype)
        for stride in (2 * 64 - 16 // item, 2 * 64 + 1, 2 * 64 + 8 // item, -128, 0):
            for k, v in ((stride, 128), (128, stride)):
                assert kvx.lib.kvx_append_kv(c.handle, A, k, A, v, A, A, 4, A, 256, None) == kvx.KVX_EINVAL
        for stride in (8 * 64 - 16 // item, 8 * 64 + 1):
            assert kvx.lib.kvx_tree_attn(c.handle, A, stride, A, 4, 2, A, None, 0.0, A, A, 1 << 40,
                                         None) == kvx.KVX_EINVAL


def test_binding_refuses_host_tensors(kvx):
    torch = pytest.importorskip("torch")
    c = make(kvx)
    for key in ("kv_len", "q_start", "slots"):
        refused(kvx, kvx.KVX_EINVAL, kvx.kvx_build_tables, c,
                **{**TABLES, key: torch.zeros(64, dtype=torch.int64 if key == "slots" else torch.int32)})
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_append_kv, c, **{**APPEND, "k_new": torch.zeros(4, 128)})


def test_reference_tables_by_hand():
    """The plain reading of the table call itself, on a case worked by hand: sequence 0 gives back a
    page, sequence 1 takes two (the page just released first, then the list's last)."""
    from tree_cases import ref_tables
    tables = [np.array([[5, 6, 7], [8, -1, -1]], np.int32)]
    free = [np.array([1, 2, -1, -1], np.int32)]
    t, pages, f, left, qs, slots = ref_tables([[9], [8]], [2, 12], [0], 1, 8, tables, [[3, 1]], free, [2],
                                              False)
    assert t[0].tolist() == [[5, 6, 7], [8, 7, 2]] and pages.tolist() == [[2, 3]]
    assert f[0].tolist() == [1, 2, 7, -1] and left.tolist() == [1] and qs.tolist() == [0, 2, 14]
    assert slots[:, 0].tolist() == [49, 50] + list(range(56, 64)) + list(range(16, 20))


def test_row_count_limit(kvx):
    c = make(kvx)
    for name, good in (("kvx_build_tables", TABLES), ("kvx_append_kv", APPEND), ("kvx_tree_attn", TREE),
                       ("kvx_tree_commit", COMMIT)):
        refused(kvx, kvx.KVX_ERANGE, getattr(kvx, name), c, **{**good, "max_rows": (1 << 30) + 1})


def test_bf16_pool_limit(kvx):
    """A bf16 pool's pages times the larger of |G| and P / 8 stay in int32 (tensor-map coordinates)."""
    refused(kvx, kvx.KVX_ERANGE, make, kvx, pages=(9, 2 ** 30), P=16)
    make(kvx, pages=(9, 2 ** 30), P=16, dtype=kvx.KVX_F32)
    make(kvx, pages=(9, 2 ** 30 - 2), P=16)


def test_inject_stall_refusals(kvx):
    c = make(kvx)
    for limit in (0, 999_999, 4_000_000_001):
        refused(kvx, kvx.KVX_ERANGE, c.inject_stall, 0, limit)
    c.inject_stall(3, 1_000_000)
    c.inject_stall(-1, 2_000_000_000)
    c.destroy()
    refused(kvx, kvx.KVX_EINVAL, c.inject_stall, 0, 1_000_000)


class OnDevice:
    """Stands in for a dense tensor on a device of the given index."""
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def element_size(self):
        return 4

    def numel(self):
        return 1 << 20

    def data_ptr(self):
        return A


def test_tensors_of_another_device_are_refused(kvx):
    pytest.importorskip("torch")
    E = kvx.KVX_EINVAL
    refused(kvx, E, make, kvx, kp=[OnDevice(0), OnDevice(1)])
    refused(kvx, E, make, kvx, kp=[OnDevice(-1), A])
    c = make(kvx, kp=[OnDevice(1), A], tables=[A, OnDevice(1)])
    c.current_device = lambda: 0  # another device is current
    refused(kvx, E, kvx.kvx_build_tables, c, **TABLES)
    refused(kvx, E, kvx.kvx_append_kv, c, **APPEND)
    refused(kvx, E, kvx.kvx_tree_attn, c, **TREE)
    refused(kvx, E, kvx.kvx_tree_commit, c, **COMMIT)
    c.current_device = lambda: 1
    for key in ("kv_len", "q_start", "free_in", "pages_out"):
        refused(kvx, E, kvx.kvx_build_tables, c, **{**TABLES, key: OnDevice(0)})
    refused(kvx, E, kvx.kvx_build_tables, c, **{**TABLES, "free_pages": [A, OnDevice(0)]})
    refused(kvx, E, kvx.kvx_tree_commit, c, **{**COMMIT, "path": OnDevice(0)})
    refused(kvx, E, kvx.kvx_tree_attn, c, **{**TREE, "mask": OnDevice(0)})
    c.destroy()


def test_no_rows_need_no_row_arrays(kvx):
    c = make(kvx)
    kvx.kvx_append_kv(c, None, None, A, None, 0, A, 256, 0)
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_append_kv, c, None, None, A, None, 1, A, 256, 0)
    c.destroy()
