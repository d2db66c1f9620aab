"""The nodes' attention stays inside the workspace it asks for, and joins its
parts from there, at every width of a head and for few and many rows."""
import numpy as np
import pytest
import torch

from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding
from test_gpu_nodes import KINDS, attn_case, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("D", [16, 64, 72, 80, 96, 112, 128, 256])
@pytest.mark.parametrize("N,G", [(1, 3), (8, 4), (12, 7)])
def test_workspace(N, G, D, qdt, kind):
    if kind == torch.float8_e4m3fn and D % 16:
        pytest.skip("8-bit rows are multiples of 16 channels")
    ctx, nodes = np.array([9000, 40, 14001]), np.array([N, 1, N])
    case = attn_case(3, N, 2 * G, 2, D, 32, qdt, kind, ctx, nodes, N + D)
    q, cache, p = case[:3]
    n = int(binding.lib().spec_tree_attention_workspace_size(cache._ref, 2 * G))
    room = torch.full((n + (16 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
    out = binding.tree_attention(q, cache, p, workspace=room[:n])
    assert bool((room[n:] == 0xa5).all())
    room.fill_(0xff)  # NaN where a join reads what no part wrote
    assert torch.equal(out, binding.tree_attention(q, cache, p, workspace=room[:n]))
    assert torch.equal(out, check_attention(*case))
