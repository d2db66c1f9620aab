"""Weights of a norm whose memory or type is another one since the norm was made: every call uses those that it checks."""
import pytest
import torch

from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def params(dt, n=64):
    g = gen(1)
    return [torch.nn.Parameter((1.0 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(dt), requires_grad=False) for _ in range(2)]


def calls(norm, q, k):
    """All that takes a norm: the rotation, and the write into a cache."""
    T = q.shape[0]
    pos, table = torch.arange(T, dtype=torch.int32, device="cuda"), binding.rope_table(64)
    cache = binding.new_kv_cache(2, 16, k.shape[1], 64, dtype=BF)
    out_k = torch.empty_like(k)
    oq = binding.kv_write(cache, k, k, torch.arange(T, device="cuda"), positions=pos, table=table, q=q, out_k=out_k, norm=norm)
    return *binding.rope(q, k, pos, table, norm=norm), oq, out_k, cache.k


@pytest.mark.parametrize("to", [BF, HF, F32])
def test_weights_given_other_memory_and_another_type(to):
    g = gen(2)
    q, k = (torch.randn((20, h, 64), generator=g, device="cuda").to(BF) for h in (4, 2))
    p = params(BF)
    norm = binding.HeadNorm(*p, eps=1e-5)
    before = calls(norm, q, k)
    kept = [x.data for x in p]  # (stays alive: its memory is nobody else's here)
    for x in p:
        x.data = (2.0 * x.data).to(to)
    got, want = calls(norm, q, k), calls(binding.HeadNorm(*p, eps=1e-5), q, k)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # (twice a bfloat16 is exact in all three types, and so is what is rounded in the end)
    for a, b in zip(got, before):
        assert torch.equal(a, 2 * b)
    assert all(x.data_ptr() != y.data_ptr() for x, y in zip(p, kept))


def test_attributes_set_anew():
    g = gen(3)
    q, k = (torch.randn((20, h, 64), generator=g, device="cuda").to(BF) for h in (4, 2))
    p = params(F32)
    norm = binding.HeadNorm(*p)
    norm.q_weight, norm.k_weight, norm.eps = p[1], None, 0.5
    for a, b in zip(calls(norm, q, k), calls(binding.HeadNorm(p[1], eps=0.5), q, k)):
        assert torch.equal(a, b)


def test_weights_that_no_longer_fit_are_refused():
    g = gen(4)
    q, k = (torch.randn((20, h, 64), generator=g, device="cuda").to(BF) for h in (4, 2))

    def refused(change, match):
        p = params(BF)
        norm = binding.HeadNorm(*p)
        change(norm, p)
        with pytest.raises(ValueError, match=match):
            binding.rope(q, k, None, None, norm=norm)
        with pytest.raises(ValueError, match=match):
            binding.kv_write(binding.new_kv_cache(2, 16, 2, 64, dtype=BF), k, k, torch.arange(20, device="cuda"), norm=norm)

    def data(to):
        def change(norm, p):
            p[0].data = to(p[0].data)
        return change
    refused(data(lambda x: x.float()), "one type")
    refused(data(lambda x: x.to(torch.int16)), "float32")
    refused(data(lambda x: torch.ones(128, dtype=BF, device="cuda")[::2]), "contiguous")
    refused(data(lambda x: x[:32]), "entries")
    refused(data(lambda x: x.cpu()), "CUDA")

    def eps(norm, p):
        norm.eps = float("nan")
    norm = binding.HeadNorm()
    eps(norm, None)
    with pytest.raises(binding.SpecVerifyError):
        binding.rope(q, k, None, None, norm=norm)
