"""Prompts and the decoding behind them, the operators in a run: what is decoded follows the target computed whole, and the
log probabilities are its own."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_common import ensure_built

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,nodes,width,head_norm", [("bf16", 16, 3, False), ("bf16", 1, 1, True), ("e4m3", 32, 4, True),
                                                         ("bf16", 5, 1, True)])
def test_prompts_then_steps(cache, nodes, width, head_norm):
    ensure_built()
    import tree_decode as T
    target = T.make_target(head_norm=head_norm)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (1, 2, 17, 130, 300)]
    lp = []
    _, tokens, kept = T.decode(nodes=nodes, width=width, steps=8, cache=cache, target=target, prompts=prompts, logprobs=lp)
    # bf16 operands and logits: a logit of size 8 is off by 2^-8 of it and by its operands' roundings, some 0.1 in all;
    # 8-bit keys and values (4 bits) more.  A log probability is off by two such logits.
    slack = 0.25 if cache == "bf16" else 1.0
    for p, t, l in zip(prompts, tokens, lp):
        assert t[:len(p)] == p and len(l) == len(t) - 1 and len(t) >= len(p) + 8
        ref = T.reference_logits(target, t)[:-1]
        got = ref.gather(1, torch.tensor(t[1:], device=ref.device)[:, None])[:, 0]
        assert len(p) > len(t) - 1 or float((ref.amax(1) - got)[len(p) - 1:].max()) <= slack
        want = torch.log_softmax(ref, -1).gather(1, torch.tensor(t[1:], device=ref.device)[:, None])[:, 0]
        assert float((want.cpu() - torch.tensor(l)).abs().max()) <= 2 * slack


def test_sampling_runs():
    ensure_built()
    import tree_decode as T
    lp = []
    _, tokens, kept = T.decode(nodes=8, width=2, steps=5, temperature=1.0, cache="e4m3", target=T.make_target(head_norm=True),
                               prompts=[[5, 6, 7]] * 3, logprobs=lp)
    assert all(len(t) >= 8 for t in tokens) and all(x <= 0 for l in lp for x in l)
