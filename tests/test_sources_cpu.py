"""Rules of the cache kernels' sources that a run cannot show to be broken without a race."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_non_uniform_gb300",
                    "csrc")


def kernels(name):
    """{kernel name: its source} of a file: from its __global__ to the next closing brace in column 0."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    return {re.search(r"(\w+)\(const __grid_constant__", part).group(1): part[:part.index("\n}\n")]
            for part in text.split("__global__")[1:]}


@pytest.mark.parametrize("source,names", [("rows.cu", {"append_kernel", "commit_kernel"}),
                                          ("tables.cu", {"tables_kernel"})])
def test_page_writers_hold_their_dependents_back(source, names):
    """A decode call with early loads reads pages and page tables before its dependency wait. Kernels
    that write them must neither release their dependents early nor finish before their writes are
    performed."""
    found = kernels(source)
    assert set(found) == names
    last_write = {"append_kernel": ".v + dst) =", "commit_kernel": "*(uint4 *)(pool", "tables_kernel": "grp.table["}
    for name, body in found.items():
        assert "pdl_launch_dependents" not in body, name
        writes = [m.end() for m in re.finditer(re.escape(last_write[name]), body)]
        assert writes and "__threadfence();" in body[writes[-1]:], name


@pytest.mark.parametrize("source", ["rows.cu", "tables.cu", "tree_mma.cu", "tree_simt.cu", "tree_merge.cu",
                                    "tree_split.cuh"])
def test_dependents_read_with_ordinary_loads(source):
    """The non-coherent path is for memory that nobody writes while the grid runs. These grids may be
    resident while the kernel before them writes their lengths, tables, slots and rows."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    assert "__ldg(" not in text and "ld.global.nc" not in text


def constant(source, name):
    return int(re.search(rf"{name}\s*(?:=|\s)\s*(\d+)", open(os.path.join(CSRC, source)).read()).group(1))


@pytest.mark.parametrize("source,item,D", [("tree_simt.cu", 4, 64), ("tree_simt.cu", 4, 128),
                                           ("tree_mma.cu", 2, 64), ("tree_mma.cu", 2, 128)])
def test_work_of_a_full_device_fits_the_cut(source, item, D):
    """The cut of tree attention counts its units in 32 bits. The most that 288 GB of distinct pages can
    ask for, with the most query heads a KV head, new rows, sequences and heads, stays below."""
    header = os.path.join("..", "..", "include", "kvx.h")
    g, tree = constant(header, "KVX_MAX_GQA"), constant(header, "KVX_MAX_TREE")
    heads = constant(header, "KVX_MAX_CACHE_SEQS") * constant(header, "KVX_MAX_KV_HEADS")
    tile = constant(source, "kTile")
    if source == "tree_simt.cu":
        tokens = constant(source, "kRows") // g
    else:
        box = constant("tree.h", "kTreeBox")
        tokens = 128 // (box * g) * box
    groups = -(-tree // tokens)
    tiles = 288e9 / (2 * tile * D * item) + heads  # the last tile of a head may be partly filled
    units = groups * (constant("tree_split.cuh", "kTileCost") * tiles
                      + constant("tree_split.cuh", "kItemCost") * heads)
    assert units < 2 ** 31, units
