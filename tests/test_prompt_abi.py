"""Host-side refusals of the prompt's pass and of the log probabilities (CPU only: no call here reaches CUDA)."""
import ctypes
import os
import shutil

import pytest
import torch
from torch.autograd import forward_ad

from test_nodes_abi import BAD_CACHES, cache

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verification_51_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


def norm(b, q=0x1000, k=0x2000, dtype=1, eps=1e-6):
    return b._CNorm(q, k, dtype, eps)


def test_norm_rope(binding):
    t, n = binding._CTable(0x1000, 64, 0, 1.0), norm(binding)
    tp, np_ = ctypes.addressof(t), ctypes.addressof(n)

    def call(D=64, T=3, dt=1, q=0x50000, table=tp, hq=2, nm=np_, pos=0x70000, out=0x60000):
        return binding.lib().spec_norm_rope(nm, q, hq, 128, 64, out, 128, 64, None, 0, 0, 0, None, 0, 0, dt, D, T, pos, table, None)
    assert call(nm=None) == INVALID and call(T=-1) == INVALID and call(dt=3) == INVALID and call(q=None) == INVALID
    assert call(pos=None) == INVALID and call(D=32) == INVALID and call(D=300) == UNSUPPORTED and call(D=65) == UNSUPPORTED
    assert call(q=0x50001) == UNSUPPORTED and call(out=None) == INVALID
    assert call(T=0) == OK and call(hq=0) == OK and call(T=0, table=None, pos=None) == OK
    for bad, status in ((norm(binding, eps=-1.0), INVALID), (norm(binding, eps=float("nan")), INVALID),
                        (norm(binding, eps=float("inf")), INVALID), (norm(binding, dtype=3), INVALID),
                        (norm(binding, q=0x1001), UNSUPPORTED), (norm(binding, k=0x2002, dtype=0), UNSUPPORTED)):
        assert call(nm=ctypes.addressof(bad)) == status


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(binding, change, status):
    c = cache(binding, **change)
    dt = 2 if change.get("dtype") == 2 else 1
    n = norm(binding)
    assert binding.lib().spec_norm_kv_write(ctypes.addressof(c), ctypes.addressof(n), 0x50000, 128, 64, None, 0, 0, 0x60000, 128, 64, dt,
                                            3, 0x70000, None, None, None, 0, 0, 0, None, 0, 0, None, None) == status


def test_norm_kv_write(binding):
    c, n = cache(binding), norm(binding)

    def call(dt=1, T=3, nm=ctypes.addressof(n), q=None, hq=0, oq=None, ok=None, slots=0x70000, k=0x50000):
        return binding.lib().spec_norm_kv_write(ctypes.addressof(c), nm, k, 128, 64, ok, 128, 64, 0x60000, 128, 64, dt, T, slots, None,
                                                None, q, hq, 128, 64, oq, 128, 64, None, None)
    assert call(dt=0) == INVALID and call(dt=2) == INVALID and call(T=-1) == INVALID and call(slots=None) == INVALID
    assert call(nm=None, q=0x80000, hq=2, oq=0x90000) == INVALID                # queries that nothing happens to
    assert call(q=0x80000, hq=2) == INVALID and call(ok=0x80001) == UNSUPPORTED and call(k=None) == INVALID
    assert call(slots=0x70004) == UNSUPPORTED and call(T=0) == OK


def test_prompt_plan(binding):
    L = binding.lib()
    big = 1 << 28

    def call(off=0x1000, koff=None, B=2, T=10, M=10, Hq=4, Hkv=2, table=None, mp=4, ps=16, npg=8, slots=None, plan=0x10000, n=big,
             st=None):
        return L.spec_prompt_plan(off, koff, B, T, M, Hq, Hkv, table, mp, ps, npg, 0x2000, slots, plan, n, st, None)
    assert call(off=None) == INVALID and call(plan=None) == INVALID and call(B=-1) == INVALID and call(T=-1) == INVALID
    assert call(M=11) == INVALID and call(Hq=3) == INVALID and call(Hkv=0) == INVALID and call(slots=0x3000) == INVALID
    assert call(Hq=258, Hkv=2) == UNSUPPORTED and call(T=1 << 31, M=1 << 31) == UNSUPPORTED
    assert call(table=0x4000, ps=24) == UNSUPPORTED and call(table=0x4000, mp=0) == INVALID and call(table=0x4000, npg=0) == INVALID
    assert call(off=0x1001) == UNSUPPORTED and call(st=0x1002) == UNSUPPORTED and call(table=0x4000, slots=0x3004) == UNSUPPORTED
    assert call(plan=0x10080) == WORKSPACE and call(n=64) == WORKSPACE
    assert L.spec_prompt_plan_size(2, 10, 3, 2) == 0 and L.spec_prompt_plan_size(-1, 10, 4, 2) == 0
    assert L.spec_prompt_plan_size(1000, 100000, 32, 8) >= 32 * (100000 // 64)


def test_prompt_attention(binding):
    def call(q=0x10000, k=0x20000, v=0x30000, st=(512, 64, 128, 64, 128, 64), dt=1, B=2, T=10, M=10, Hq=8, Hkv=2, D=64, plan=0x40000,
             scale=0.125, window=0, out=0x50000, lse=None):
        return binding.lib().spec_prompt_attention(q, st[0], st[1], k, st[2], st[3], v, st[4], st[5], dt, B, T, M, Hq, Hkv, D, plan, scale,
                                                   window, out, lse, None, None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(plan=None), dict(out=None), dict(dt=0), dict(dt=3), dict(B=-1), dict(D=0),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(Hq=3)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(D=264), dict(q=0x10008), dict(out=0x50008), dict(lse=0x2), dict(st=(512, 64, 128, 68, 128, 64)),
                dict(st=(-512, 64, 128, 64, 128, 64)), dict(Hq=258), dict(T=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(plan=0x40010) == WORKSPACE and call(T=0) == OK and call(B=0) == OK


def test_token_logprobs(binding):
    L = binding.lib()

    def call(logits=0x10000, dt=1, R=4, st=1000, V=1000, rows=None, tokens=0x20000, temp=None, E=4, top=5, lp=0x30000, ent=0x40000,
             ids=0x50000, lps=0x60000, ws=0x100000, n=1 << 30, status=None):
        return L.spec_token_logprobs(logits, dt, R, st, V, rows, tokens, temp, E, top, lp, ent, ids, lps, ws, n, status, None)
    for bad in (dict(R=-1), dict(E=-1), dict(V=0), dict(top=33), dict(top=-1), dict(E=5), dict(dt=3), dict(st=999), dict(logits=None),
                dict(tokens=None), dict(lp=None), dict(ids=None), dict(lps=None), dict(ws=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(V=(1 << 24) + 1, st=1 << 25), dict(logits=0x10001), dict(tokens=0x20002), dict(lp=0x30001), dict(temp=0x3)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(E=0) == OK and call(E=0, R=0, logits=None) == OK
    assert L.spec_token_logprobs_workspace_size(-1, 100) == 0 and L.spec_token_logprobs_workspace_size(4, 0) == 0
    assert L.spec_token_logprobs_workspace_size(4, 100) > 0


def test_head_norm(binding):
    with pytest.raises(ValueError, match="CUDA"):
        binding.HeadNorm(torch.ones(8))
    with pytest.raises(ValueError, match="eps"):
        binding.HeadNorm(eps=-1.0)
    with pytest.raises(ValueError, match="float32"):
        binding.HeadNorm(torch.ones(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="inverse"):
        binding.rope(torch.zeros(1, 1, 8), None, None, None, norm=binding.HeadNorm(), inverse=True)


def test_gradients_are_refused(binding):
    """As in the other calls: before anything else is looked at."""
    leaf, x = torch.zeros(3, 2, 64, requires_grad=True), torch.zeros(3, 2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    plan = binding.PromptPlan(i, None, 1, 3, 3, 2, 2, torch.zeros(1))
    calls = [lambda y: binding.rope(y, None, i, None, norm=binding.HeadNorm()), lambda y: binding.prompt_attention(y, x, x, plan),
             lambda y: binding.prompt_attention(x, y, x, plan), lambda y: binding.prompt_attention(x, x, y, plan),
             lambda y: binding.token_logprobs(y, i)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(leaf)
        with pytest.raises(ValueError, match="gradient"):
            call(leaf * 2)
        with forward_ad.dual_level(), pytest.raises(ValueError, match="gradient"):
            call(forward_ad.make_dual(x, torch.ones_like(x)))
        with torch.no_grad(), pytest.raises(Exception) as e:             # refused for what comes next
            call(leaf)
        assert "gradient" not in str(e.value)
