"""The prompt's pass and the log probabilities on another stream: what a call uses is dropped at once, and its memory is
not given to anybody else before the call has run."""
import pytest
import torch

from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def test_tensors_of_another_stream_outlive_the_call():
    g, side = torch.Generator(device="cuda").manual_seed(1), torch.cuda.Stream()
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = binding.new_kv_cache(8, 16, 2, 64)
    table = binding.rope_table(64)
    plan = binding.prompt_plan(i([0, 70, 100]), 100, 8, 2)

    def check(call, make):
        want = [x.clone() for x in call(*[x.clone() for x in make], stream=None)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)                  # some 50 ms
        args = [x.clone() for x in make]
        side.wait_stream(torch.cuda.current_stream())
        got = call(*args, stream=side)
        held, sizes = {x.data_ptr() for x in args}, [(x.shape, x.dtype) for x in args]
        del args
        assert not side.query()                             # the call has not run yet
        other = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes for _ in range(3)]
        assert not held & {x.data_ptr() for x in other}
        for x in other:
            x.fill_(-1)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)

    w = 1 + 0.1 * t(64)
    check(lambda a, b, c, d, stream: binding.rope(a, b, c, table, norm=binding.HeadNorm(d, d), stream=stream),
          [t(12, 8, 64), t(12, 2, 64), i([5] * 12), w])

    def write(a, b, c, d, e, f, stream):
        k = torch.empty_like(a)
        q = binding.kv_write(cache, a, b, c, positions=d, table=table, q=e, out_k=k, norm=binding.HeadNorm(f, f), stream=stream)
        return q, k
    check(write, [t(12, 2, 64), t(12, 2, 64), torch.arange(12, device="cuda"), i([5] * 12), t(12, 8, 64), w])
    check(lambda a, b, c, stream: (binding.prompt_attention(a, b, c, plan, stream=stream),), [t(100, 8, 64), t(100, 2, 64), t(100, 2, 64)])

    def make_plan(a, b, stream):
        p = binding.prompt_plan(a, 100, 8, 2, page_table=b, cache=cache, stream=stream)
        return p.positions, p.slots
    check(make_plan, [i([0, 70, 100]), i([[0, 1, 2, 3, 4], [5, 6, 7, 0, 0]])])

    def lp(a, b, c, stream):
        r = binding.token_logprobs(a, b, temperature=c, top=4, entropy=True, stream=stream)
        return r.logprobs, r.entropy, r.top_ids, r.top_logprobs
    check(lp, [t(30, 5001), i([7] * 30), torch.full((30,), 0.7, device="cuda")])
