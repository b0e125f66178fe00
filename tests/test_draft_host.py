"""Host-side checks of a drafting step's entry points: exported, bound under their names,
declining bad arguments before the device is touched; the host's frequencies; and the GPU
tests' reference."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import draftref
import kv8ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10008      # never dereferenced: the checks come first
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 6, 10
NAMES = ["cq_attn_kv8_tree", "cq_kv8_write_rope", "cq_rope", "cq_rope_freqs", "cq_verify"]


@pytest.fixture(scope="module")
def L():
    from block_quantized_weight_02_gb300 import build
    build.build()
    return cq.lib()


def test_exported_and_bound(L):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cq_draft.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(cq_[a-z0-9_]+)\s*\(", src))) == NAMES
    for n in NAMES:
        assert hasattr(L, n) and hasattr(cq, n)


def spec(**k):
    d = dict(freq=FAKE, rot=64, layout=0, mag=1.0)
    d.update(k)
    return ctypes.byref(cq._rope_desc(*[d[n] for n, _ in cq._rope_desc._fields_]))


def cache(**k):
    d = dict(Kq=FAKE, Ks=FAKE, Vq=FAKE, Vs=FAKE, pages=10, Hkv=2, page=64, D=128, table=FAKE, ldt=4, B=3)
    d.update(k)
    return ctypes.byref(cq._kv8_desc(*[d[n] for n, _ in cq._kv8_desc._fields_]))


def rope(L, X=FAKE, xt=1, T=5, H=2, D=128, ldx=256, r=None, pos=FAKE, Y=0x100000, yt=1, ldy=256, **k):
    return L.cq_rope(X, xt, T, H, D, ldx, r or spec(**k), pos, Y, yt, ldy, None)


def write(L, c=None, K=FAKE, V=FAKE, xt=1, T=5, ldk=256, ldv=256, qs=FAKE, lens=FAKE, r=None, pos=None, **k):
    return L.cq_kv8_write_rope(c or cache(), K, V, xt, T, ldk, ldv, qs, lens, r or spec(**k), pos, None)


def tree(L, Q=FAKE, xt=1, T=5, Hq=4, ldq=512, c=None, qs=FAKE, lens=FAKE, max_q=5, scale=0.1, mask=FAKE, ldm=1, O=FAKE, yt=2, ldo=512,
         lse=None, ws=FAKE, wsb=1 << 40):
    return L.cq_attn_kv8_tree(Q, xt, T, Hq, ldq, c or cache(), qs, lens, max_q, scale, mask, ldm, O, yt, ldo, lse, ws, wsb, None)


def verify(L, P=FAKE, pt=2, T=5, V=100, ldp=100, Q=None, ldq=100, tokens=FAKE, mask=None, ldm=0, qs=FAKE, B=2, max_q=4, u=FAKE, ul=FAKE,
           out=FAKE, path=FAKE, ldo=4, count=FAKE):
    return L.cq_verify(P, pt, T, V, ldp, Q, ldq, tokens, mask, ldm, qs, B, max_q, u, ul, out, path, ldo, count, None)


@pytest.mark.parametrize("change,status", [
    (dict(freq=None), NULL), (dict(rot=0), SHAPE), (dict(rot=8), SHAPE), (dict(rot=72), SHAPE), (dict(rot=144), SHAPE), (dict(layout=2), ARG),
    (dict(layout=-1), ARG), (dict(mag=math.inf), ARG), (dict(mag=math.nan), ARG), (dict(freq=FAKE + 2), ALIGN)])
def test_positions_are_checked(L, change, status):
    for f, who in ((rope, "cq_rope"), (write, "cq_kv8_write_rope")):
        assert f(L, **change) == status
        assert cq.cq_last_error().startswith("decline: " + who + ":")
        assert L.cq_last_launches() == 0


@pytest.mark.parametrize("change,status", [
    (dict(X=None), NULL), (dict(Y=None), NULL), (dict(pos=None), NULL), (dict(xt=3), DTYPE), (dict(yt=-1), DTYPE), (dict(T=0), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(D=120), SHAPE), (dict(D=0), SHAPE), (dict(D=1040, ldx=4096, ldy=4096), SHAPE), (dict(ldx=255), SHAPE),
    (dict(ldx=260), SHAPE), (dict(ldy=248), SHAPE), (dict(X=ODD), ALIGN), (dict(Y=ODD), ALIGN), (dict(pos=FAKE + 1), ALIGN),
    (dict(Y=FAKE, yt=2), ARG), (dict(Y=FAKE, ldy=264), ARG), (dict(Y=FAKE + 16), ARG), (dict(Y=FAKE + 512), ARG), (dict(Y=FAKE - 512), ARG),
    (dict(T=1, Y=FAKE + 256), ARG), (dict(ldx=512, ldy=512, Y=FAKE + 256), ARG), (dict(ldx=512, ldy=512, Y=FAKE + 1024 - 256), ARG)])
def test_rope_refusals(L, change, status):
    assert rope(L, **change) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="the call would run")
def test_rope_takes_columns_side_by_side(L):
    """Queries and keys of one product's rows, and a tensor in place: the checks of the arguments pass."""
    for y in (FAKE, FAKE + 512, FAKE - 512):
        assert rope(L, ldx=512, ldy=512, Y=y) in (7, 9)


@pytest.mark.parametrize("change,status", [
    (dict(K=None), NULL), (dict(V=None), NULL), (dict(qs=None), NULL), (dict(lens=None), NULL), (dict(xt=3), DTYPE), (dict(T=0), SHAPE),
    (dict(ldk=255), SHAPE), (dict(ldv=128), SHAPE), (dict(K=ODD), ALIGN), (dict(qs=FAKE + 1), ALIGN), (dict(pos=FAKE + 2), ALIGN)])
def test_write_refusals(L, change, status):
    assert write(L, **change) == status


def test_write_cache_refusals(L):
    for change, status in ((dict(Kq=None), NULL), (dict(D=96), SHAPE), (dict(page=48), SHAPE), (dict(B=0), SHAPE), (dict(Ks=ODD), ALIGN)):
        assert write(L, c=cache(**change)) == status
        assert tree(L, c=cache(**change)) == status
    assert L.cq_kv8_write_rope(None, FAKE, FAKE, 1, 5, 256, 256, FAKE, FAKE, spec(), None, None) == NULL
    assert L.cq_kv8_write_rope(cache(), FAKE, FAKE, 1, 5, 256, 256, FAKE, FAKE, None, None, None) == NULL
    assert L.cq_attn_kv8_tree(FAKE, 1, 5, 4, 512, None, FAKE, FAKE, 5, 0.1, FAKE, 1, FAKE, 2, 512, None, FAKE, 1 << 40, None) == NULL


@pytest.mark.parametrize("change,status", [
    (dict(Q=None), NULL), (dict(O=None), NULL), (dict(mask=None), NULL), (dict(ws=None), NULL), (dict(xt=2), DTYPE), (dict(Hq=5), SHAPE),
    (dict(ldq=511), SHAPE), (dict(ldm=0), SHAPE), (dict(T=50, max_q=33), SHAPE), (dict(T=50, max_q=1000, ldm=1), SHAPE), (dict(mask=FAKE + 2), ALIGN),
    (dict(max_q=0), SHAPE), (dict(scale=0.0), ARG), (dict(ws=FAKE + 16), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(lse=FAKE + 2), ALIGN)])
def test_tree_refusals(L, change, status):
    assert tree(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(P=None), NULL), (dict(tokens=None), NULL), (dict(qs=None), NULL), (dict(u=None), NULL), (dict(ul=None), NULL), (dict(out=None), NULL),
    (dict(path=None), NULL), (dict(count=None), NULL), (dict(pt=3), DTYPE), (dict(V=0), SHAPE), (dict(V=1 << 30, ldp=1 << 30), SHAPE), (dict(T=0), SHAPE),
    (dict(ldp=99), SHAPE), (dict(ldp=102), SHAPE), (dict(Q=FAKE, ldq=96), SHAPE), (dict(P=ODD), ALIGN), (dict(Q=ODD), ALIGN), (dict(B=0), SHAPE),
    (dict(B=65537), SHAPE), (dict(max_q=0), SHAPE), (dict(max_q=1025, ldo=1025), SHAPE), (dict(ldo=3), SHAPE), (dict(mask=FAKE, ldm=0), SHAPE),
    (dict(mask=FAKE, ldm=1, max_q=40, ldo=40), SHAPE), (dict(mask=FAKE + 1, ldm=1), ALIGN), (dict(tokens=FAKE + 2), ALIGN), (dict(u=FAKE + 1), ALIGN),
    (dict(out=FAKE + 3), ALIGN)])
def test_verify_refusals(L, change, status):
    assert verify(L, **change) == status
    assert L.cq_last_launches() == 0


def test_binding_refuses_wrong_tensors():
    f = torch.zeros(32)
    r = cq.cq_rope_spec(f)
    for bad in (f.double(), f.view(2, 16), torch.zeros(64)[::2]):
        with pytest.raises(ValueError):
            cq.cq_rope_spec(bad)
    x, pos = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int32)
    for args in ((x.view(3, 256), pos), (x.transpose(0, 1), pos), (torch.zeros(3, 2, 256)[..., ::2], pos)):
        with pytest.raises(ValueError):
            cq.cq_rope(args[0], r, args[1])
    with pytest.raises(ValueError):
        cq.cq_rope(x, r, pos, torch.zeros(3, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        cq.cq_rope(x, r, pos)
    q = lambda *s: torch.zeros(*s, dtype=torch.int8)
    c = cq.cq_kv8_cache(q(4, 2, 64, 128), torch.zeros(4, 2, 2), q(4, 2, 64, 128), torch.zeros(4, 2, 2), torch.zeros(1, 2, dtype=torch.int32))
    qs, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        cq.cq_kv8_write_rope(c, x, x.half(), qs, lens, r)
    with pytest.raises(ValueError, match="GPU"):
        cq.cq_kv8_write_rope(c, x, x, qs, lens, r)
    h, m = x.half(), torch.zeros(3, 1, dtype=torch.int32)
    for bad in (m[:2], m.long(), m[:, 0]):
        with pytest.raises(ValueError):
            cq.cq_attn_kv8_tree(h, c, qs, lens, 3, bad, x, None)
    with pytest.raises(ValueError):
        cq.cq_attn_kv8_tree(torch.zeros(40, 2, 128).half(), c, qs, lens, 40, torch.zeros(40, 1, dtype=torch.int32), torch.zeros(40, 2, 128), None)
    with pytest.raises(ValueError, match="GPU"):
        cq.cq_attn_kv8_tree(h, c, qs, lens, 3, m, x, None)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    p, one = torch.zeros(3, 8), torch.zeros(1)
    good = dict(P=p, tokens=i(3), q_start=i(2), max_q=3, u=torch.zeros(3), u_last=one, out=i(1, 3), path=i(1, 3), count=i(1))
    for change in (dict(P=p[0]), dict(P=p.t()), dict(Q=p.half()), dict(Q=p[:2]), dict(out=i(1, 2)), dict(path=i(2, 3)), dict(out=torch.zeros(1, 3)),
                   dict(mask=i(2, 1)), dict(mask=i(3, 1), max_q=40, out=i(1, 40), path=i(1, 40))):
        with pytest.raises(ValueError):
            cq.cq_verify(**{**good, **change})
    with pytest.raises(ValueError, match="GPU"):
        cq.cq_verify(**good)


def test_what_is_assigned_to_positions_reaches_the_descriptor():
    """The descriptor holds addresses: it must follow the tensor, whose old one is given up."""
    a, b = torch.zeros(32), torch.ones(16)
    r = cq.cq_rope_spec(a, cq.CQ_ROPE_PAIRS, 1.25)
    assert (r.freq is a, r.layout, r.mag) == (True, cq.CQ_ROPE_PAIRS, 1.25)
    r.freq = b
    assert r.freq is b and (r.desc.freq, r.desc.rot, r.desc.layout, r.desc.mag) == (b.data_ptr(), 32, cq.CQ_ROPE_PAIRS, 1.25)
    assert r._device == b.get_device()
    r.mag, r.layout = 2.0, cq.CQ_ROPE_HALF
    assert (r.desc.freq, r.desc.layout, r.desc.mag) == (b.data_ptr(), cq.CQ_ROPE_HALF, 2.0)
    assert ctypes.cast(r._ref, ctypes.POINTER(cq._rope_desc)).contents.mag == 2.0     # what calls hand over
    for bad in (b.double(), b.view(2, 8), torch.zeros(32)[::2]):
        with pytest.raises(ValueError):
            r.freq = bad
    for name, bad in (("layout", "half"), ("mag", "large")):
        with pytest.raises(TypeError):
            setattr(r, name, bad)
    assert r.freq is b and (r.desc.freq, r.desc.layout, r.desc.mag) == (b.data_ptr(), cq.CQ_ROPE_HALF, 2.0) and (r.layout, r.mag) == (0, 2.0)


# ---- frequencies ----------------------------------------------------------------------------------------------------

def test_frequencies():
    i = np.arange(32)
    f = 10000.0 ** (-2 * i / 64)
    near = lambda a, b: np.testing.assert_allclose(a.numpy(), b, rtol=2.0 ** -23)     # one rounding to f32, and 64-bit powers
    got, mag = cq.cq_rope_freqs(64)
    near(got, f)
    assert mag == 1.0
    got, mag = cq.cq_rope_freqs(64, kind=cq.CQ_ROPE_LINEAR, factor=8.0)
    near(got, f / 8)
    assert mag == 1.0
    got, mag = cq.cq_rope_freqs(64, kind=cq.CQ_ROPE_BASE, factor=8.0)
    near(got, (10000.0 * 8.0 ** (64 / 62)) ** (-2 * i / 64))
    np.testing.assert_allclose(float(got[-1]), f[-1] / 8, rtol=1e-6)                   # the slowest one by the factor
    got, mag = cq.cq_rope_freqs(64, kind=cq.CQ_ROPE_RAMP, factor=16.0, low=1.0, high=32.0, trained=8192.0)
    lo, hi = (64 * math.log(8192 / (2 * math.pi * n)) / (2 * math.log(10000.0)) for n in (32, 1))
    ramp = np.clip((i - math.floor(lo)) / (math.ceil(hi) - math.floor(lo)), 0, 1)
    near(got, f / 16 * ramp + f * (1 - ramp))
    assert abs(mag - (0.1 * math.log(16) + 1)) < 1e-6
    got, mag = cq.cq_rope_freqs(64, kind=cq.CQ_ROPE_BANDS, factor=8.0, low=1.0, high=4.0, trained=8192.0)
    turn = 2 * math.pi / f
    s = (8192 / turn - 1) / 3
    near(got, np.where(turn < 8192 / 4, f, np.where(turn > 8192, f / 8, (1 - s) * f / 8 + s * f)))
    assert mag == 1.0


@pytest.mark.parametrize("change", [dict(rot=0), dict(rot=24), dict(rot=1040), dict(base=1.0), dict(base=math.nan), dict(kind=5), dict(kind=1, factor=0.5),
                                    dict(kind=2, factor=math.inf), dict(kind=3, low=0.0), dict(kind=4, low=4.0, high=4.0), dict(kind=3, trained=0.0)])
def test_frequency_refusals(change):
    with pytest.raises(cq.CQError):
        cq.cq_rope_freqs(**{**dict(rot=64), **change})


# ---- the reference of the GPU tests ---------------------------------------------------------------------------------

def test_reference_rotation_keeps_lengths_and_differences():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 1, 32))
    f = 100.0 ** (-np.arange(8) / 8)
    for layout in ("half", "pairs"):
        a, b = draftref.rotate(x, [5, 9], f, layout), draftref.rotate(x, [105, 109], f, layout)
        np.testing.assert_allclose((a ** 2).sum(-1), (x ** 2).sum(-1))
        np.testing.assert_allclose(a[0, 0] @ a[1, 0], b[0, 0] @ b[1, 0])              # scores know differences of positions only
        np.testing.assert_array_equal(a[..., 16:], x[..., 16:])


def test_reference_tree_attention_is_the_chain_where_the_tree_is_one():
    rng = np.random.default_rng(2)
    c = kv8ref.Cache(1, 1, 64)
    c.write(0, rng.standard_normal((40, 1, 64)), rng.standard_normal((40, 1, 64)))
    q = rng.standard_normal((5, 2, 64))
    o, lse, *_ = draftref.attend(c, 0, q, 0.125, [(2 << i) - 1 for i in range(5)], "f32")
    o2, lse2, *_ = kv8ref.attend(c, 0, q, 0.125, True, 0)
    np.testing.assert_allclose(o, o2, atol=1e-14)
    np.testing.assert_allclose(lse, lse2)


@pytest.mark.parametrize("drawn", [True, False])
def test_reference_check_gives_the_targets_distribution(drawn):
    """Over many draws the token after the root is distributed as P of the root, whatever the drafts are."""
    rng = np.random.default_rng(3)
    V, N = 5, 40000
    P = rng.dirichlet(np.ones(V), size=4)
    Q = rng.dirichlet(np.ones(V), size=4)
    parents = [-1, 0, 0, 1]
    seen = np.zeros(V)
    for _ in range(N):
        t = [0, *(rng.choice(V, p=Q[0], size=2) if drawn else (2, 4)), rng.choice(V, p=Q[1])]
        out, path = draftref.verify(P, Q if drawn else None, t, parents, rng.random(4), rng.random())
        assert len(out) == len(path)
        seen[out[0]] += 1
    # five standard deviations of a count
    assert np.all(np.abs(seen - N * P[0]) < 5 * np.sqrt(N * P[0] * (1 - P[0])))
