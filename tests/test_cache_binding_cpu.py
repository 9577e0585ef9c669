"""What the binding's cache calls check of the arrays that they are given. Stand-ins for device
tensors serve, and no call passes every check, so nothing is launched."""
import pytest

from test_cache_cpu import A, APPEND, COMMIT, TABLES, TREE, kvx, make, refused  # noqa: F401

torch = pytest.importorskip("torch")

CALLS = [("kvx_build_tables", TABLES), ("kvx_append_kv", APPEND), ("kvx_tree_attn", TREE),
         ("kvx_tree_commit", COMMIT)]


class Dev:
    """Stands in for a device tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32, device=1, contiguous=True):
        self.shape, self.dtype, self.device, self.dense = shape, dtype, device, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.dense

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def stride(self):
        out = [1]
        for x in self.shape[:0:-1]:
            out.insert(0, out[0] * x)
        return tuple(out)

    def data_ptr(self):
        return A


def on_device_1(kvx, **change):
    """A cache on device 1, which is current. Its tables and pools fit make()'s shape."""
    pool = dict(dtype=torch.bfloat16)
    c = make(kvx, **{**dict(kp=[Dev(9 * 16, 64, **pool)] * 2, vp=[Dev(9 * 16, 64, **pool)] * 2,
                            tables=[Dev(2, 4)] * 2), **change})
    c.current_device = lambda: 1
    return c


@pytest.mark.parametrize("name,good", CALLS)
def test_workspace_is_checked(kvx, name, good):
    """On the cache's device, dense, and no smaller than it is said to be."""
    c, call = on_device_1(kvx), getattr(kvx, name)
    for bad in (Dev(1 << 20, device=0), Dev(1 << 20, contiguous=False), torch.zeros(1 << 10), None, "ws"):
        for nbytes in (None, 256):
            refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "workspace": bad, "workspace_bytes": nbytes})
    for nbytes in (257, -1):
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "workspace": Dev(64), "workspace_bytes": nbytes})
    refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "workspace": A, "workspace_bytes": None})
    refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "workspace": A, "workspace_bytes": -1})
    assert kvx._workspace(c, Dev(64), None) == (A, 256)
    assert kvx._workspace(c, Dev(64), 255) == (A, 255)
    assert kvx._workspace(c, A, 1 << 40) == (A, 1 << 40)


def test_free_lists_hold_the_whole_pool(kvx):
    """The call may push every page: a list with room for fewer ids than the pool has pages is refused."""
    c = on_device_1(kvx, pages=(9, 12), kp=[A, A], vp=[A, A])
    good = {**TABLES, "workspace": Dev(64), "workspace_bytes": None}
    for lists in ([Dev(8), Dev(12)], [Dev(9), Dev(11)], [Dev(9), None], [Dev(9, device=0), Dev(12)]):
        refused(kvx, kvx.KVX_EINVAL, kvx.kvx_build_tables, c, **{**good, "free_pages": lists})


INTS = {"kvx_build_tables": ["kv_len", "new_len", "pages_in", "pages_out", "free_in", "free_out", "q_start"],
        "kvx_append_kv": ["q_start"], "kvx_tree_attn": ["q_start", "kv_len", "mask"],
        "kvx_tree_commit": ["q_start", "path", "n_acc", "kv_len", "kv_len_out"]}


@pytest.mark.parametrize("name,good", CALLS)
def test_element_types_are_checked(kvx, name, good):
    """An array of another type of the same size is refused: lengths and masks are integers, rows have the
    cache's type, the output is fp32."""
    c, call = on_device_1(kvx), getattr(kvx, name)
    good = {**good, "workspace": Dev(1 << 20), "workspace_bytes": None}
    for key in INTS[name]:
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, key: Dev(64, dtype=torch.float32)})
    if name == "kvx_build_tables":
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "free_pages": [Dev(64, dtype=torch.float32)] * 2})
    if "slots" in good:
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "slots": Dev(64, dtype=torch.float64)})
    if name == "kvx_append_kv":
        for key in ("k_new", "v_new"):
            refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, key: Dev(4, 128, dtype=torch.float16)})
    if name == "kvx_tree_attn":
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "q": Dev(4, 512, dtype=torch.int16)})
        refused(kvx, kvx.KVX_EINVAL, call, c, **{**good, "out": Dev(4, 8, 64, dtype=torch.int32)})


def test_accepted_element_types(kvx):
    c = on_device_1(kvx)
    for dtype, kind in ((torch.int32, "int32"), (torch.uint32, "int32"), (torch.int64, "int64"),
                        (torch.float32, "float32")):
        assert kvx._dense(c, Dev(64, dtype=dtype), "x", kind, 64) == A
    assert kvx._rows(c, Dev(4, 2, 64, dtype=torch.bfloat16), "x", 128, 4) == (A, 128)
    f = make(kvx, dtype=kvx.KVX_F32)
    assert kvx._rows(f, Dev(4, 128, dtype=torch.float32), "x", 128, 4) == (A, 128)
    refused(kvx, kvx.KVX_EINVAL, kvx._rows, f, Dev(4, 128, dtype=torch.bfloat16), "x", 128, 4)


def test_page_tables_hold_their_strides(kvx):
    for bad in (Dev(2, 3), Dev(7), Dev(2, 4, dtype=torch.float32), Dev(2, 4, contiguous=False)):
        refused(kvx, kvx.KVX_EINVAL, on_device_1, kvx, tables=[Dev(2, 4), bad])
    on_device_1(kvx, tables=[Dev(2, 4), Dev(9)]).destroy()


@pytest.mark.parametrize("which", ["kp", "vp"])
@pytest.mark.parametrize("dtype,right,wrong", [(1, torch.bfloat16, torch.float16), (0, torch.float32, torch.float64)])
def test_pools_hold_their_pages(kvx, which, dtype, right, wrong):
    """Too few rows, another type, not dense: the calls that touch pools refuse."""
    full = (9 * 16, 64)
    other = {"kp": "vp", "vp": "kp"}[which]
    both = [Dev(*full, dtype=right)] * 2
    fit = on_device_1(kvx, dtype=dtype, **{which: both, other: both})
    assert fit.pools_fit
    raw = [Dev(fit.pool_pages[0] * 16 * 64 * (4 if dtype == 0 else 2), dtype=torch.uint8)] * 2
    assert on_device_1(kvx, dtype=dtype, **{which: raw, other: both}).pools_fit
    for bad in (Dev(9 * 16 - 1, 64, dtype=right), Dev(*full, dtype=wrong),
                Dev(*full, dtype=right, contiguous=False)):
        c = on_device_1(kvx, dtype=dtype, **{which: [Dev(*full, dtype=right), bad], other: both})
        for name, good in CALLS[1:]:
            with pytest.raises(kvx.KvxError, match="pool_pages") as e:
                getattr(kvx, name)(c, **good)
            assert e.value.status == kvx.KVX_EINVAL


def test_arrays_that_are_no_tensors(kvx):
    refused(kvx, kvx.KVX_EINVAL, on_device_1, kvx, kp=["pool", A])


def test_path_without_a_stride(kvx):
    """An address, nothing or a flat tensor has no row stride of its own."""
    c = on_device_1(kvx)
    good = {**COMMIT, "workspace": Dev(64), "workspace_bytes": None, "path_stride": None}
    for path in (A, None, Dev(4)):
        refused(kvx, kvx.KVX_EINVAL, kvx.kvx_tree_commit, c, **{**good, "path": path})


def test_rows_that_are_no_tensors(kvx):
    import numpy as np
    for c in (on_device_1(kvx), make(kvx)):
        for bad in (np.zeros((4, 128), np.float32), [0.0], "rows", None):
            refused(kvx, kvx.KVX_EINVAL, kvx._rows, c, bad, "rows", 128, 4)
