"""Host-side refusals of the operators around the verification (CPU only: no
call here reaches CUDA), and the rotary frequencies, which are host code."""
import ctypes
import math
import os
import shutil
from fractions import Fraction

import numpy as np
import pytest

from nodes_common import thetas

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verification_51_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


@pytest.mark.parametrize("rot,scaling,factor", [(2, "none", 1), (64, "none", 1), (128, "linear", 4), (96, "ntk", 8),
                                                (128, "by_parts", 32), (256, "by_parts", 1.5)])
def test_rope_turns(binding, rot, scaling, factor):
    out = (ctypes.c_uint64 * (rot // 2))()
    scale = ctypes.c_float()
    rc = binding.lib().spec_rope_turns(rot, 10000.0, binding.ROPE_SCALING[scaling], factor, 4096.0, 32.0, 1.0,
                                       ctypes.addressof(out), ctypes.addressof(scale))
    assert rc == OK
    th, s = thetas(rot, scaling=scaling, factor=factor, original_len=4096.0)
    # double precision of theta / (2 pi): 2^-50 of it
    for got, want in zip(out, th):
        w = Fraction(float(want)) / Fraction(2 * math.pi)
        assert abs(Fraction(got, 2 ** 64) - w) <= w / 2 ** 50 + Fraction(1, 2 ** 63)
    assert scale.value == np.float32(s)


@pytest.mark.parametrize("args", [(63, 1e4, 0, 1, 0, 32, 1), (0, 1e4, 0, 1, 0, 32, 1), (258, 1e4, 0, 1, 0, 32, 1),
                                  (64, 1.0, 0, 1, 0, 32, 1), (64, float("nan"), 0, 1, 0, 32, 1), (64, 1e4, 4, 1, 0, 32, 1),
                                  (64, 1e4, 1, 0.5, 0, 32, 1), (64, 1e4, 3, 2, 0, 32, 1), (64, 1e4, 3, 2, 4096, 1, 1)])
def test_rope_turns_refuses(binding, args):
    out = (ctypes.c_uint64 * 128)()
    scale = ctypes.c_float()
    assert binding.lib().spec_rope_turns(*args, ctypes.addressof(out), ctypes.addressof(scale)) == INVALID
    assert binding.lib().spec_rope_turns(64, 1e4, 0, 1, 0, 32, 1, None, ctypes.addressof(scale)) == INVALID


def cache(b, **kw):
    a = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, dtype=b.SPEC_BF16, num_pages=4, page_size=16,
             heads=2, head_dim=64, page_stride=2048, head_stride=1024, token_stride=64)
    a.update(kw)
    return b._CCache(*a.values())


BAD_CACHES = [
    (dict(k=0), INVALID), (dict(dtype=0), INVALID), (dict(dtype=7), INVALID), (dict(num_pages=0), INVALID),
    (dict(heads=0), INVALID), (dict(token_stride=32), INVALID), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=131072), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED), (dict(head_dim=264, token_stride=264), UNSUPPORTED),
    (dict(k=0x10008), UNSUPPORTED), (dict(token_stride=66), UNSUPPORTED), (dict(page_stride=-2048), UNSUPPORTED),
    (dict(dtype=3, k_scale=0), INVALID), (dict(dtype=3, head_dim=72, token_stride=80), UNSUPPORTED),
    (dict(dtype=3, v_scale=0x40004), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(binding, change, status):
    L = binding.lib()
    c = cache(binding, **change)
    p = ctypes.addressof(c)
    dt = 2 if change.get("dtype") == 2 else 1
    assert L.spec_kv_read(p, 3, 0x50000, dt, 0x60000, 0x70000, None) == status
    assert L.spec_kv_write(p, 0x50000, 128, 64, 0x60000, 128, 64, dt, 3, 0x70000, None, None, None, 0, 0, 0, None, 0, 0,
                           None, None) == status
    assert L.spec_tree_attention(0x50000, 512, 256, 64, dt, 1, 2, 4, p, 0x60000, 4, 0x70000, 0x80000, 1.0, 0x90000, None,
                                 0xA0000, 1 << 30, None, None) == status
    assert L.spec_kv_commit(p, 1, 0x50000, 0x60000, 0x70000, 0x80000, 1, 2, 0x90000, None, None) == status
    assert L.spec_tree_attention_workspace_size(p, 4) == 0


def test_other_refusals(binding):
    L = binding.lib()
    c = cache(binding)
    p = ctypes.addressof(c)
    # types that do not go together
    for dt in (0, 2, 3):
        assert L.spec_kv_write(p, 0x50000, 128, 64, 0x60000, 128, 64, dt, 3, 0x70000, None, None, None, 0, 0, 0, None, 0,
                               0, None, None) == INVALID
    assert L.spec_kv_read(p, 3, 0x50000, 3, 0x60000, 0x70000, None) == INVALID
    assert L.spec_kv_read(p, -1, 0x50000, 1, 0x60000, 0x70000, None) == INVALID
    assert L.spec_kv_read(p, 3, None, 1, 0x60000, 0x70000, None) == INVALID
    assert L.spec_kv_read(p, 3, 0x50000, 1, 0x60008, 0x70000, None) == UNSUPPORTED
    assert L.spec_kv_read(p, 0, None, 1, None, None, None) == OK              # nothing to do

    def attn(q=0x50000, st=(512, 256, 64), dt=1, B=1, N=2, Hq=4, ws=1 << 30, wsp=0xA0000, plan=0x80000):
        return L.spec_tree_attention(q, *st, dt, B, N, Hq, p, 0x60000, 4, 0x70000, plan, 1.0, 0x90000, None, wsp, ws, None,
                                     None)
    assert attn(N=33) == UNSUPPORTED and attn(N=0) == INVALID and attn(B=-1) == INVALID
    assert attn(Hq=3) == UNSUPPORTED and attn(dt=2) == INVALID and attn(dt=0) == INVALID
    assert attn(q=0x50004) == UNSUPPORTED and attn(st=(512, 256, 68)) == UNSUPPORTED
    assert attn(q=None) == INVALID and attn(wsp=0xA0010) == WORKSPACE and attn(plan=0x80010) == WORKSPACE
    assert attn(B=0) == OK

    def plan(B=1, N=2, mp=4, ps=16, npg=4, buf=0x80000, n=1 << 20, par=0x10000):
        return L.spec_tree_plan(par, 0x20000, 0x30000, 0x40000, B, N, mp, ps, npg, 0x50000, 0x60000, 0x70000, buf, n, None,
                                None)
    assert plan(N=33) == UNSUPPORTED and plan(N=0) == INVALID and plan(ps=8) == UNSUPPORTED and plan(mp=0) == INVALID
    assert plan(mp=1 << 28) == UNSUPPORTED and plan(par=None) == INVALID
    assert plan(buf=0x80080) == WORKSPACE and plan(n=16) == WORKSPACE and plan(B=0) == OK
    assert L.spec_tree_plan_size(-1) == 0 and L.spec_tree_plan_size(100) >= 4 * 301
    two = (binding._CCache * 2)(c, cache(binding, page_stride=4096))
    assert L.spec_kv_commit(ctypes.addressof(two), 2, 0x50000, 0x60000, 0x70000, 0x80000, 1, 2, 0x90000, None, None) == INVALID
    assert L.spec_kv_commit(p, 65, 0x50000, 0x60000, 0x70000, 0x80000, 1, 2, 0x90000, None, None) == INVALID
    assert L.spec_kv_commit(p, 1, None, 0x60000, 0x70000, 0x80000, 1, 2, 0x90000, None, None) == INVALID

    t = binding._CTable(0x1000, 64, 0, 1.0)
    tp = ctypes.addressof(t)

    def rope(D=64, T=3, dt=1, q=0x50000, table=tp, hq=2):
        return L.spec_rope(q, hq, 128, 64, 0x60000, 128, 64, None, 0, 0, 0, None, 0, 0, dt, D, T, 0x70000, table, 0, None)
    assert rope(D=32) == INVALID and rope(D=300) == UNSUPPORTED and rope(D=65) == UNSUPPORTED
    assert rope(dt=3) == INVALID and rope(q=None) == INVALID and rope(table=None) == INVALID and rope(T=-1) == INVALID
    assert rope(q=0x50001) == UNSUPPORTED and rope(T=0) == OK and rope(hq=0) == OK
    for bad in (binding._CTable(None, 64, 0, 1.0), binding._CTable(0x1000, 63, 0, 1.0), binding._CTable(0x1000, 0, 0, 1.0),
                binding._CTable(0x1000, 64, 2, 1.0)):
        assert rope(table=ctypes.addressof(bad)) == INVALID
