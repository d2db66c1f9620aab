"""The norm of each head with the rotation, alone and on the way into the cache, against its 64-bit form."""
import numpy as np
import pytest
import torch

import nodes_common as C
import prompt_common as P
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dt, g, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dt)


def weights(D, dt, g):
    return 1.0 + 0.3 * torch.randn(D, generator=g, device="cuda").to(dt)


def want_of(x, w, eps, pos, th, layout, dtype, scale=1.0):
    """(value, bound) of a normalised and turned tensor, before the last rounding and with it."""
    y = P.norm(x, w, eps)
    nb = P.norm_bound(y, x.shape[-1])
    if th is None:
        return y, nb + C.U[dtype] * (y.abs() + nb) + C.TINY[dtype]
    r = C.rotate(y, pos, th, layout, scale)
    n = 2 * len(th)
    # a pair's members carry each other's error
    mate = nb.clone()
    if layout == "half":
        a, b = nb[..., :n // 2], nb[..., n // 2:n]
        mate[..., :n // 2], mate[..., n // 2:n] = a + b, a + b
    else:
        a, b = nb[..., 0:n:2], nb[..., 1:n:2]
        mate[..., 0:n:2], mate[..., 1:n:2] = a + b, a + b
    bound = mate * scale * (1 + C.U[dtype]) + C.rotate_bound(y, th, layout, dtype, scale)
    bound[..., n:] += C.U[dtype] * y[..., n:].abs() + C.TINY[dtype]        # what does not turn is rounded here too
    return r, bound


def near(got, want, bound):
    got = got.detach().cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    far = ((got - want).abs() - bound)[~want.isnan()]
    assert float(far.max()) <= 0, float(far.max())


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (80, 40), (96, 96), (256, 128), (20, 6), (2, 2), (250, 10)])
def test_norm_rope(D, rot, layout, dt):
    g = gen(D + rot)
    T, Hq, Hkv = 19, 5, 3
    q, k = randn((T, Hq, D), dt, g, 3.0), randn((T, Hkv, D), dt, g, 0.2)
    q[3, 1] *= 1e-3
    wq, wk = weights(D, dt, g), weights(D, dt, g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 - 5
    table = binding.rope_table(rot, layout=layout)
    th, _ = C.thetas(rot)
    a, b = binding.rope(q, k, pos, table, norm=binding.HeadNorm(wq, wk, eps=1e-5))
    near(a, *want_of(q, wq, 1e-5, pos, th, layout, dt))
    near(b, *want_of(k, wk, 1e-5, pos, th, layout, dt))
    a2 = binding.rope(q, None, pos, table, norm=binding.HeadNorm(wq.float(), None, eps=1e-5))
    assert torch.equal(a2, a)


def test_norm_alone_and_without_weights():
    g = gen(1)
    q, k = randn((33, 4, 128), BF, g), randn((33, 2, 128), BF, g)
    a, b = binding.rope(q, k, None, None, norm=binding.HeadNorm(eps=1e-6))
    near(a, *want_of(q, None, 1e-6, None, None, None, BF))
    near(b, *want_of(k, None, 1e-6, None, None, None, BF))
    w = weights(128, BF, g)
    c = binding.rope(q, None, None, None, norm=binding.HeadNorm(w))
    near(c, *want_of(q, w, 1e-6, None, None, None, BF))


def test_scaled_table():
    g = gen(2)
    q = randn((9, 2, 128), BF, g)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") + 100000
    kw = dict(scaling="by_parts", factor=8.0, original_len=4096)
    table = binding.rope_table(128, **kw)
    th, sc = C.thetas(128, **kw)
    a = binding.rope(q, None, pos, table, norm=binding.HeadNorm())
    near(a, *want_of(q, None, 1e-6, pos, th, "half", BF, sc))


def test_strides_and_in_place():
    g = gen(3)
    T = 50
    qkv = randn((T, 8 + 2 + 2, 64), BF, g)
    q, k = qkv[:, :8], qkv[:, 8:10]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    table, n = binding.rope_table(64), binding.HeadNorm(weights(64, BF, g), weights(64, BF, g))
    want = binding.rope(q.contiguous(), k.contiguous(), pos, table, norm=n)
    a, b = binding.rope(q, k, pos, table, norm=n)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    keep = qkv[:, 10:].clone()
    binding.rope(q, k, pos, table, out_q=q, out_k=k, norm=n)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 10:], keep)
    odd = randn((T, 3, 67), BF, g)[:, :, 1:65]                        # nothing is aligned
    c = binding.rope(odd, None, pos, table, norm=n)
    near(c, *want_of(odd, n.q_weight, 1e-6, pos, C.thetas(64)[0], "half", BF))


def test_zeros_and_values_that_are_not_finite():
    q = torch.zeros((4, 1, 64), dtype=BF, device="cuda")
    q[1, 0, 5], q[2, 0, 6] = float("nan"), float("inf")
    q[3] = 1e18
    a = binding.rope(q, None, None, None, norm=binding.HeadNorm()).float()
    assert bool((a[0] == 0).all()) and bool(a[1].isnan().all())
    assert bool(a[2, 0, 6].isnan()) and bool((a[2, 0, :6] == 0).all())
    near(a[3], *want_of(q[3], None, 1e-6, None, None, None, BF))
    b = binding.rope(q, None, None, None, norm=binding.HeadNorm(eps=0.0)).float()
    assert bool(b[0].isnan().all())


@pytest.mark.parametrize("T", [1, 2, 700, 9000])
def test_few_and_many_tokens(T):
    """Every division of the heads over groups of lanes."""
    g = gen(T)
    q, k = randn((T, 16, 128), BF, g), randn((T, 4, 128), BF, g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    wq, wk = weights(128, BF, g), weights(128, BF, g)
    for layout in ("half", "interleaved"):
        table = binding.rope_table(128, layout=layout)
        a, b = binding.rope(q, k, pos, table, norm=binding.HeadNorm(wq, wk))
        i = torch.arange(0, T, max(1, T // 50))
        near(a[i], *want_of(q[i], wq, 1e-6, pos[i], C.thetas(128)[0], layout, BF))
        near(b[i], *want_of(k[i], wk, 1e-6, pos[i], C.thetas(128)[0], layout, BF))


@pytest.mark.parametrize("dt,kind", [(BF, BF), (HF, HF), (BF, E4), (HF, E4), (F32, E4)])
@pytest.mark.parametrize("D,rot,layout", [(128, 128, "half"), (64, 32, "interleaved"), (96, 96, "half"), (48, 0, "half"), (256, 64, "half"),
                                          (16, 6, "interleaved")])
def test_norm_kv_write(D, rot, layout, dt, kind):
    g = gen(D)
    T, Hq, Hkv, page = 37, 6, 2, 16
    cache = binding.new_kv_cache(5, page, Hkv, D, dtype=kind)
    q, k, v = randn((T, Hq, D), dt, g), randn((T, Hkv, D), dt, g, 2.0), randn((T, Hkv, D), dt, g)
    wq, wk = weights(D, dt, g), weights(D, dt, g)
    slots = torch.randperm(5 * page, generator=g, device="cuda")[:T]
    slots[5], slots[9] = -1, 5 * page + 3
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 50
    table = binding.rope_table(rot, layout=layout) if rot else None
    th = C.thetas(rot)[0] if rot else None
    n = binding.HeadNorm(wq, wk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out_k = torch.empty_like(k)
    oq = binding.kv_write(cache, k, v, slots, positions=pos if rot else None, table=table, q=q, out_k=out_k, norm=n, dev_status=status)
    assert int(status) == binding.BADBIT["page"]
    near(oq, *want_of(q, wq, 1e-6, pos, th, layout, dt))
    near(out_k, *want_of(k, wk, 1e-6, pos, th, layout, dt))
    gk, gv = binding.kv_read(cache, slots, dtype=F32)
    there = (slots >= 0) & (slots < 5 * page)
    assert bool((gk[~there] == 0).all())
    if kind == E4:
        # the cache holds the value before its rounding to 16 bits, in 4 significant bits of the row's power of two
        y, b = want_of(k, wk, 1e-6, pos, th, layout, F32)
        vals, e = C.e4m3_values(y.numpy())
        step = torch.from_numpy(np.exp2(e.astype(np.float64)))[..., None] * 2.0 ** -10
        near(gk[there], y[there.cpu()], ((y.abs() * 2.0 ** -4).maximum(step.expand_as(y)) * 1.01 + b)[there.cpu()])
        # away from a border between two values it is the nearest one
        off = (gk.cpu().double() - torch.from_numpy(vals)).abs()[there.cpu()]
        assert float((off > 0).double().mean()) < 1e-3
    else:
        assert torch.equal(gk[there], out_k[there].float())
    plain = binding.new_kv_cache(5, page, Hkv, D, dtype=kind)
    binding.kv_write(plain, k, v, slots)
    assert torch.equal(binding.kv_read(plain, slots, dtype=F32)[1], gv)


def test_out_k_without_a_norm_is_the_rotation():
    """Keys to a tensor besides their slots, the norm left out: what rope and kv_write give, bit for bit."""
    g = gen(5)
    T, Hq, Hkv, D = 100, 8, 2, 128
    q, k, v = randn((T, Hq, D), BF, g), randn((T, Hkv, D), BF, g), randn((T, Hkv, D), BF, g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(128, generator=g, device="cuda")[:T]
    slots[::7] = -1
    for kind in (BF, E4):
        table = binding.rope_table(D)
        a, b = (binding.new_kv_cache(8, 16, Hkv, D, dtype=kind) for _ in range(2))
        wq = binding.kv_write(a, k, v, slots, positions=pos, table=table, q=q)
        wk = binding.rope(k, None, pos, table)
        k2 = k.clone()
        oq = binding.kv_write(b, k2, v, slots, positions=pos, table=table, q=q, out_k=k2)      # in place
        assert torch.equal(oq, wq) and torch.equal(k2, wk)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
        if kind == E4:
            assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
        plain = torch.empty_like(k)
        c = binding.new_kv_cache(8, 16, Hkv, D, dtype=kind)
        binding.kv_write(c, k, v, slots, out_k=plain)
        assert torch.equal(plain, k)
