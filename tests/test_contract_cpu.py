"""Limits that the header states, against the library (host calls only)."""
import os
import re

import pytest


@pytest.fixture(scope="module")
def kvx():
    from paged_non_uniform_gb300 import build
    build.build()
    from paged_non_uniform_gb300 import kvx as k
    return k


HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvx.h")


def comment_of(function):
    """The header's comment before a function's declaration, as one line."""
    text = open(HEADER).read()
    text = text[:text.index(f"\nint {function}(")]
    return " ".join(re.sub(r"\n \* ?", "\n", text[text.rindex("/*"):]).split())


def test_stated_stall_limits_are_the_accepted_ones(kvx):
    """1 ms up to the stated number of seconds is accepted, a nanosecond more or less is not."""
    plan = kvx.kvx_plan_create(1, 4, 1, 128, 16, 1, kvx.KVX_BF16, [[64]], [64], [0], num_ctas=4)
    cache = kvx.Cache(1, 4, 1, 128, 16, 1, kvx.KVX_BF16, [0], [1 << 20], [1 << 20], [9], [1 << 20], [4])
    for function, handle in (("kvx_plan_inject_stall", plan.handle), ("kvx_cache_inject_stall", cache.handle)):
        most = int(re.search(r"\(1 ms \.\. (\d+) s", comment_of(function)).group(1)) * 10 ** 9
        call = getattr(kvx.lib, function)
        for ns in (10 ** 6, most):
            assert call(handle, -1, ns) == kvx.KVX_OK, (function, ns)
        for ns in (10 ** 6 - 1, most + 1):
            assert call(handle, -1, ns) == kvx.KVX_ERANGE, (function, ns)


def test_unaligned_integer_arrays_are_refused(kvx):
    """A kernel's load from an address that is not a multiple of its size would fault."""
    from test_cache_cpu import A, APPEND, COMMIT, TABLES, TREE, make, refused
    c = make(kvx)
    for name, good, keys in (
            ("kvx_build_tables", TABLES, ("kv_len", "new_len", "pages_in", "pages_out", "free_in", "free_out",
                                          "q_start")),
            ("kvx_append_kv", APPEND, ("q_start",)), ("kvx_tree_attn", TREE, ("q_start", "kv_len", "mask")),
            ("kvx_tree_commit", COMMIT, ("q_start", "path", "n_acc", "kv_len", "kv_len_out"))):
        for key in keys:
            for off in (1, 2):
                refused(kvx, kvx.KVX_EINVAL, getattr(kvx, name), c, **{**good, key: 4 * A + off})
    refused(kvx, kvx.KVX_EINVAL, kvx.kvx_build_tables, c, **{**TABLES, "free_pages": [A, A + 2]})


def test_row_strides_past_a_tensor_map_are_refused(kvx):
    """2^40 bytes: an argument error, not a failed launch."""
    from test_cache_cpu import A, make
    for dtype, item in ((kvx.KVX_BF16, 2), (kvx.KVX_F32, 4)):
        c = make(kvx, dtype=dtype)
        for stride in (2 ** 40 // item, 2 ** 40, 2 ** 62):
            assert kvx.lib.kvx_tree_attn(c.handle, A, stride, A, 4, 2, A, None, 0.0, A, A, 1 << 40,
                                         None) == kvx.KVX_EINVAL
            assert kvx.lib.kvx_append_kv(c.handle, A, stride, A, 128, A, A, 4, A, 256, None) == kvx.KVX_EINVAL
            assert kvx.lib.kvx_append_kv(c.handle, A, 128, A, stride, A, A, 4, A, 256, None) == kvx.KVX_EINVAL
