"""Pointers that a kernel would read or write at a misaligned address are refused on
the host (CPU only: no call here reaches CUDA)."""
import ctypes
import os
import shutil

import pytest

from test_nodes_abi import UNSUPPORTED, binding, cache  # noqa: F401

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

PLAN = dict(par=4, nodes=4, ctx=4, table=4, positions=4, slots=8, masks=4, status=4)
ATTN = dict(table=4, masks=4, lse=4, status=4, q=16, out=16)
COMMIT = dict(masks=4, slots=8, last=4, ctx=4, new=4, status=4)
WRITE = dict(k=2, v=2, slots=8, positions=4, q=2, out_q=2, status=4)


def off(pointers):
    """Each pointer in turn off by half of what it needs (from 4 bytes on also by 1)."""
    return [(n, d) for n, a in pointers.items() for d in sorted({a // 2, 1})]


def at(names, bad, by):
    return {n: 0x100000 * (i + 1) + (by if n == bad else 0) for i, n in enumerate(names)}


@pytest.mark.parametrize("bad,by", off(PLAN))
def test_plan(binding, bad, by):  # noqa: F811
    a = at(PLAN, bad, by)
    assert binding.lib().spec_tree_plan(a["par"], a["nodes"], a["ctx"], a["table"], 1, 2, 4, 16, 4, a["positions"], a["slots"],
                                        a["masks"], 0x8000000, 1 << 20, a["status"], None) == UNSUPPORTED


@pytest.mark.parametrize("bad,by", off(ATTN))
def test_attention(binding, bad, by):  # noqa: F811
    a, c = at(ATTN, bad, by), cache(binding)
    assert binding.lib().spec_tree_attention(a["q"], 512, 256, 64, 1, 1, 2, 4, ctypes.addressof(c), a["table"], 4, a["masks"],
                                             0x8000000, 1.0, a["out"], a["lse"], 0x9000000, 1 << 30, a["status"],
                                             None) == UNSUPPORTED


@pytest.mark.parametrize("bad,by", off(COMMIT))
def test_commit(binding, bad, by):  # noqa: F811
    a, c = at(COMMIT, bad, by), cache(binding)
    assert binding.lib().spec_kv_commit(ctypes.addressof(c), 1, a["masks"], a["slots"], a["last"], a["ctx"], 1, 2, a["new"],
                                        a["status"], None) == UNSUPPORTED


@pytest.mark.parametrize("bad,by", off(WRITE))
def test_write(binding, bad, by):  # noqa: F811
    a, c, t = at(WRITE, bad, by), cache(binding), binding._CTable(0x1000, 64, 0, 1.0)
    assert binding.lib().spec_kv_write(ctypes.addressof(c), a["k"], 128, 64, a["v"], 128, 64, 1, 3, a["slots"], a["positions"],
                                       ctypes.addressof(t), a["q"], 2, 128, 64, a["out_q"], 128, 64, a["status"],
                                       None) == UNSUPPORTED
