"""The operators around the verification on several streams: one plan for all of
them, workspaces that hold anything, tensors of another stream."""
import numpy as np
import pytest
import torch

from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding
from test_gpu_nodes import BF, E4, HF, attn_case, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("qdt,kind", [(BF, BF), (HF, E4)])
@pytest.mark.parametrize("N,Hq", [(2, 8), (12, 24)])
def test_one_plan_on_several_streams(N, Hq, qdt, kind):
    """Calls that may overlap: every item of theirs is joined from parts."""
    q, cache, p, table, ctx, nodes = attn_case(2, N, Hq, 2, 64, 32, qdt, kind, [20000, 700], [N, N], 3)
    g = gen(4)
    qs = [randn(q.shape, qdt, g, 1.5) for _ in range(6)]
    want = [binding.tree_attention(x, cache, p) for x in qs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got += [binding.tree_attention(x, cache, p, stream=streams[i % 3]) for i, x in enumerate(qs)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 6]) for i, x in enumerate(got))


@pytest.mark.parametrize("N,Hq", [(1, 4), (12, 24)])
def test_workspace_of_any_content(N, Hq):
    q, cache, p, *_ = attn_case(3, N, Hq, 2, 64, 16, BF, BF, [9000, 40, 14001], [N, 1, N], 5)
    want = binding.tree_attention(q, cache, p)
    room = torch.empty(int(binding.lib().spec_tree_attention_workspace_size(cache._ref, Hq)), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    for fill in (0x00, 0xff, 0x01, 0x7f, None):
        if fill is None:
            room.copy_(torch.from_numpy(rng.integers(0, 256, room.numel(), dtype=np.uint8)))
        else:
            room.fill_(fill)
        for _ in range(3):
            assert torch.equal(binding.tree_attention(q, cache, p, workspace=room), want)
