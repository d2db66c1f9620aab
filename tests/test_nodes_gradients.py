"""The operators around the verification have no backward: tensors whose history a
call would drop are refused (before anything else is looked at, so on the CPU
too)."""
import os
import shutil

import pytest
import torch
from torch.autograd import forward_ad

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verification_51_gb300 import binding, build
    build.build()
    return binding


@needs_nvcc
def test_gradients_are_refused(binding):
    x = torch.zeros(3, 2, 64)
    leaf = torch.zeros(3, 2, 64, requires_grad=True)
    i = torch.zeros(3, dtype=torch.int32)
    for y in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            binding.rope(y, None, i, None)
        with torch.no_grad(), pytest.raises(Exception) as e:      # refused for what comes next
            binding.rope(y, None, i, None)
        assert "gradient" not in str(e.value)
    with pytest.raises(ValueError, match="gradient"):
        binding._ops().rope(leaf.detach(), leaf, i, None, None, None, False, None)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="gradient"):
            binding.rope(dual, None, i, None)


@pytest.mark.gpu
def test_gradients_are_refused_by_every_call(binding):
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    g = lambda *s: t(*s).requires_grad_(True)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = binding.new_kv_cache(4, 16, 2, 64)
    table = binding.rope_table(64)
    slots = torch.arange(3, device="cuda")
    p = binding.tree_plan(i(1, 1), i(1) + 1, i(1), i(1, 1), cache)
    calls = [lambda f: binding.rope(f(3, 2, 64), None, i(3), table),
             lambda f: binding.rope(t(3, 2, 64), f(3, 2, 64), i(3), table),
             lambda f: binding.rope(t(3, 2, 64), None, i(3), table, out_q=f(3, 2, 64)),
             lambda f: binding.kv_write(cache, f(3, 2, 64), t(3, 2, 64), slots),
             lambda f: binding.kv_write(cache, t(3, 2, 64), f(3, 2, 64), slots),
             lambda f: binding.kv_write(cache, t(3, 2, 64), t(3, 2, 64), slots, positions=i(3), table=table, q=f(3, 4, 64)),
             lambda f: binding.kv_read(cache, slots, out_k=f(3, 2, 64)),
             lambda f: binding.tree_attention(f(1, 1, 4, 64), cache, p),
             lambda f: binding.tree_attention(t(1, 1, 4, 64), cache, p, out=f(1, 1, 4, 64))]
    for call in calls:
        call(t)
        with pytest.raises(ValueError, match="gradient"):
            call(g)
        with torch.no_grad():
            call(g)
        with torch.inference_mode():
            call(g)
