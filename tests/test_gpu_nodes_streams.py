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


@pytest.mark.parametrize("kind", [BF, E4])
def test_tensors_of_another_stream_outlive_the_call(kind):
    """`stream=` behind a stream that is busy: what a call uses is dropped at once, and its
    memory is not given to anybody else before the call has run."""
    B, N, Hq, Hkv, D, page = 3, 4, 8, 2, 64, 16
    q, cache, p, table, ctx, nodes = attn_case(B, N, Hq, Hkv, D, page, BF, kind, [1000, 40, 300], [N] * 3, 9)
    side, g = torch.cuda.Stream(), gen(1)
    t = lambda *s: randn(s, BF, g)  # noqa: E731
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = p.slots.view(-1)
    par = i([[-1, 0, 0, 1]] * B)

    def check(call, make):
        """`make`: the call's tensors, dropped after it."""
        want = call(*[x.clone() for x in make], stream=None)
        want = [x.clone() for x in want]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)                  # some 50 ms
        args = [x.clone() for x in make]
        side.wait_stream(torch.cuda.current_stream())
        got = call(*args, stream=side)
        held = {x.data_ptr() for x in args}
        sizes = [(x.shape, x.dtype) for x in args]
        del args
        assert not side.query()                             # the call has not run yet
        other = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes for _ in range(3)]
        assert not held & {x.data_ptr() for x in other}
        for x in other:
            x.fill_(-1)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)

    def table_of(turns):
        return binding.RopeTable(turns, "half", 1.0)

    turns = binding.rope_table(64).turns
    check(lambda a, b, c, d, stream: binding.rope(a, b, c, table_of(d), stream=stream), [t(12, 8, 64), t(12, 2, 64), i([5] * 12), turns])
    check(lambda a, b, c, d, e, f, stream: (binding.kv_write(cache, a, b, c, positions=d, table=table_of(e), q=f, stream=stream),),
          [t(12, 2, 64), t(12, 2, 64), slots, i([5] * 12), turns, t(12, 8, 64)])
    check(lambda a, stream: binding.kv_read(cache, a, stream=stream), [slots])

    def plan(a, b, c, d, stream):
        x = binding.tree_plan(a, b, c, d, cache, stream=stream)
        return x.positions, x.slots, x.masks

    check(plan, [par, i(nodes.tolist()), i(ctx.tolist()), table])
    check(lambda a, b, stream: (binding.tree_attention(a, cache, p, masks=b, stream=stream),), [q, p.masks])
    check(lambda a, stream: (binding.kv_commit([cache], p, a, stream=stream),), [i([-1, -1, -1])])
