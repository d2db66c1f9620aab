"""Plans and positions that are written anew in the same memory between calls that read them, with nothing waited for on the
host: kernels begin early behind one another, and each reads what the one before it wrote."""
import pytest
import torch

import prompt_common as P
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", [(40, 2, 1), (700, 8, 2)])
def test_one_plan_buffer_for_batches_one_behind_the_other(T, Hq, Hkv, graph):
    D, n = 64, 24
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    cuts = [sorted(torch.randint(0, T + 1, (3,), generator=torch.Generator().manual_seed(i)).tolist()) for i in range(n)]
    offs = [i32([0] + c + [T]) for c in cuts]
    want, want_pos = [], []
    for o in offs:
        p = binding.prompt_plan(o, T, Hq, Hkv)
        want.append(binding.prompt_attention(q, k, v, p))
        want_pos.append(p.positions)
        torch.cuda.synchronize()
    table = binding.rope_table(D)
    want_turned = [binding.rope(q, None, pos, table, norm=binding.HeadNorm()) for pos in want_pos]
    plan = binding.prompt_plan(offs[0], T, Hq, Hkv)
    out, turned = [torch.zeros_like(q) for _ in offs], [torch.zeros_like(q) for _ in offs]
    norm = binding.HeadNorm()
    lib = binding.lib()
    torch.cuda.synchronize()

    def run():
        stream = torch.cuda.current_stream().cuda_stream
        for o, y, z in zip(offs, out, turned):
            assert lib.spec_prompt_plan(o.data_ptr(), None, 4, T, T, Hq, Hkv, None, 0, 0, 0, plan.positions.data_ptr(), None,
                                        plan.buffer.data_ptr(), plan.buffer.numel(), None, stream) == 0
            binding.rope(q, None, plan.positions, table, out_q=z, norm=norm)
            binding.prompt_attention(q, k, v, plan, out=y)

    def check():
        torch.cuda.synchronize()
        for a, b in zip(out + turned, want + want_turned):
            assert torch.equal(a, b)
            a.zero_()
    if not graph:
        for _ in range(10):
            run()
            check()
        return
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    check()
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.graph(captured):
        run()
    for _ in range(20):
        captured.replay()
        captured.replay()
        check()


def test_workspace_of_log_probabilities_used_again():
    """One workspace for calls one behind the other, each on other logits that a kernel has just written."""
    E, V, n = 30, 5003, 20
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = [3.0 * torch.randn((E, V), generator=g, device="cuda").to(BF) for _ in range(n)]
    tokens = torch.randint(0, V, (E,), generator=g, device="cuda").to(torch.int32)
    want = [binding.token_logprobs(x, tokens, top=5, entropy=True) for x in logits]
    ws = torch.empty(int(binding.lib().spec_token_logprobs_workspace_size(E, V)), dtype=torch.uint8, device="cuda")
    here = torch.empty_like(logits[0])
    for _ in range(10):
        got = []
        for x in logits:
            here.copy_(x)
            got.append(binding.token_logprobs(here, tokens, top=5, entropy=True, workspace=ws))
        for a, b in zip(got, want):
            for name in ("logprobs", "entropy", "top_ids", "top_logprobs"):
                assert torch.equal(getattr(a, name), getattr(b, name)), name
    lp = P.logprobs(logits[0], tokens)[0]
    assert float((want[0].logprobs.double() - lp).abs().max()) < 1e-4
