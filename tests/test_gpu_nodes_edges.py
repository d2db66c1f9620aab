"""The nodes' attention where it can go wrong, for few rows a key head
(k_attn_rows) and for many (the tile kernels): nodes that are not there, values
of very different sizes, queries that are not finite, scales of any sign, strides,
pages far into a cache, other streams, and a step in a CUDA graph."""
import math

import numpy as np
import pytest
import torch

import nodes_common as NC
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding
from test_gpu_nodes import BF, E4, FL, HF, KINDS, attn_case, check_attention, gen, randn

pytestmark = pytest.mark.gpu

# nodes and query heads over 2 key heads: at most 16 rows a key head, and more
FEW_AND_MANY = [(6, 4), (12, 24)]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def slots_of(table, ctx, page, b, tokens):
    """The cache slots of `tokens` of request b."""
    t = np.asarray(tokens)
    return dev(table[b].cpu().numpy()[t // page].astype(np.int64) * page + t % page)


def star_masks(B, N, nodes):
    """Node 0 and its children alone: a node sees node 0 and itself."""
    m = np.array([[(1 << v | 1) if v < nodes[b] else 0 for v in range(N)] for b in range(B)], np.uint32)
    return dev(m.view(np.int32))


# ---------------------------------------------------------------- nodes that are not there

@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
@pytest.mark.parametrize("ctx", [[40, 37, 300], [21000, 9, 30000]])   # whole items, and items joined from parts
def test_nodes_past_the_tree_are_zero_whatever_the_context_holds(ctx, N, Hq, qdt, kind):
    nodes = [N - 2, N - 3, 1]
    q, cache, p, table, ctx, nodes = attn_case(3, N, Hq, 2, 64, 16, qdt, kind, ctx, nodes, 5)
    for b, t, value in ((0, 11, math.nan), (2, 200, math.inf)):
        s = int(slots_of(table, ctx, 16, b, [t])[0])
        cache.k[s // 16, :, s % 16, 3] = 0x7f if kind == E4 else value
    lse = torch.zeros((3, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, lse=lse)
    for b in range(3):
        n = int(nodes[b])
        assert not out[b, n:].any() and bool((lse[b, n:] == -math.inf).all())
    m = p.masks.cpu().numpy().view(np.uint32)
    ref, _, bound = NC.attention(q, cache, table, ctx, nodes, m, 1 / 8)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(out.double()), torch.isnan(ref))
    assert bool(((out.double() - ref).abs()[fin] <= bound[fin]).all())
