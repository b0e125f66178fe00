"""Host-side checks of the 8-bit cache's entry points: exported, bound under
their names, and declining bad arguments before the device is touched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import kv8ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10008      # never dereferenced: the checks come first
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 6, 10


@pytest.fixture(scope="module")
def L():
    from block_quantized_weight_02_gb300 import build
    build.build()
    return cq.lib()


def test_exported_and_bound(L):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cq_kv8.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(cq_[a-z0-9_]+)\s*\(", src)))
    assert names == ["cq_attn_kv8", "cq_attn_kv8_workspace_bytes", "cq_kv8_read", "cq_kv8_write"]
    for n in names:
        assert hasattr(L, n) and hasattr(cq, n)


def desc(**k):
    d = dict(Kq=FAKE, Ks=FAKE, Vq=FAKE, Vs=FAKE, pages=10, Hkv=2, page=64, D=128, table=FAKE, ldt=4, B=3)
    d.update(k)
    return cq._kv8_desc(*[d[n] for n, _ in cq._kv8_desc._fields_])


def write(L, c=None, K=FAKE, V=FAKE, xt=1, T=5, ldk=256, ldv=256, qs=FAKE, lens=FAKE):
    return L.cq_kv8_write(ctypes.byref(c or desc()), K, V, xt, T, ldk, ldv, qs, lens, None)


def read(L, c=None, K=FAKE, V=FAKE, yt=1, T=5, ldk=256, ldv=256, first=None, start=FAKE):
    return L.cq_kv8_read(ctypes.byref(c or desc()), first, start, K, V, yt, T, ldk, ldv, None)


def attn(L, c=None, Q=FAKE, xt=1, T=5, Hq=4, ldq=512, qs=FAKE, lens=FAKE, max_q=5, scale=0.1, causal=1, window=0, O=FAKE,
         yt=2, ldo=512, lse=None, ws=FAKE, wsb=1 << 40):
    return L.cq_attn_kv8(Q, xt, T, Hq, ldq, ctypes.byref(c or desc()), qs, lens, max_q, scale, causal, window, O, yt, ldo, lse,
                         ws, wsb, None)


BAD_CACHE = [(dict(Kq=None), NULL), (dict(Vs=None), NULL), (dict(table=None), NULL), (dict(D=96), SHAPE), (dict(D=0), SHAPE),
             (dict(page=48), SHAPE), (dict(page=0), SHAPE), (dict(pages=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=1025), SHAPE),
             (dict(pages=1 << 24), SHAPE), (dict(B=0), SHAPE), (dict(B=65537), SHAPE), (dict(ldt=0), SHAPE), (dict(Kq=ODD), ALIGN),
             (dict(Ks=ODD), ALIGN), (dict(table=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_cache_is_checked(L, change, status):
    for f in (write, read, attn):
        assert f(L, desc(**change)) == status
        assert cq.cq_last_error().startswith("decline: " + {write: "cq_kv8_write", read: "cq_kv8_read", attn: "cq_attn_kv8"}[f])
        assert L.cq_last_launches() == 0


@pytest.mark.parametrize("change,status", [
    (dict(K=None), NULL), (dict(V=None), NULL), (dict(T=0), SHAPE), (dict(T=1 << 31), SHAPE), (dict(ldk=255), SHAPE),
    (dict(ldv=260), SHAPE), (dict(ldk=128), SHAPE), (dict(K=ODD), ALIGN), (dict(V=ODD), ALIGN)])
def test_rows_are_checked(L, change, status):
    for f in (write, read):
        assert f(L, **change) == status


def test_store_refusals(L):
    assert write(L, xt=3) == DTYPE and read(L, yt=-1) == DTYPE
    assert write(L, lens=None) == NULL and write(L, qs=None) == NULL and read(L, start=None) == NULL
    assert write(L, qs=FAKE + 1) == ALIGN and read(L, first=FAKE + 2) == ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(Q=None), NULL), (dict(O=None), NULL), (dict(qs=None), NULL), (dict(lens=None), NULL), (dict(ws=None), NULL),
    (dict(xt=2), DTYPE), (dict(yt=3), DTYPE), (dict(Hq=5), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=130, ldq=130 * 128), SHAPE),
    (dict(T=0), SHAPE), (dict(T=1 << 30), SHAPE), (dict(ldq=511), SHAPE), (dict(ldq=516), SHAPE), (dict(ldo=510), SHAPE),
    (dict(Q=ODD), ALIGN), (dict(O=ODD), ALIGN), (dict(lse=FAKE + 2), ALIGN), (dict(max_q=0), SHAPE), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(window=-1), ARG),
    (dict(causal=2), ARG), (dict(causal=0, window=5), ARG), (dict(ws=FAKE + 16), WORKSPACE), (dict(wsb=0), WORKSPACE)])
def test_attention_refusals(L, change, status):
    assert attn(L, **change) == status


def test_workspace_sizes(L):
    f = cq.cq_attn_kv8_workspace_bytes
    assert f(0, 4, 2, 128, 1, 1) == 0 and f(1, 5, 2, 128, 1, 1) == 0
    assert f(1, 4, 2, 128, 1, 1) > 0
    assert f(100000, 64, 8, 128, 4, 50000) >= f(1, 8, 8, 64, 1, 1)


def test_binding_refuses_wrong_tensors():
    q = lambda *s: torch.zeros(*s, dtype=torch.int8)
    s = lambda *x: torch.zeros(*x)
    t = torch.zeros(1, 2, dtype=torch.int32)
    cache = cq.cq_kv8_cache(q(4, 2, 64, 128), s(4, 2, 2), q(4, 2, 64, 128), s(4, 2, 2), t)
    for bad in [(q(4, 2, 64, 128), s(4, 2, 1)), (s(4, 2, 64, 128), s(4, 2, 2)), (q(4, 64, 2, 128).transpose(1, 2), s(4, 2, 2))]:
        with pytest.raises(ValueError):
            cq.cq_kv8_cache(bad[0], bad[1], q(4, 2, 64, 128), s(4, 2, 2), t)
    with pytest.raises(ValueError):
        cq.cq_kv8_cache(cache.Kq, cache.Ks, cache.Vq, cache.Vs, t.long())
    x = torch.zeros(3, 2, 128)
    qs, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for k in (torch.zeros(3, 2, 64), torch.zeros(2, 3, 128).transpose(0, 1), torch.zeros(3, 256)):
        with pytest.raises(ValueError):
            cq.cq_kv8_write(cache, k, k, qs, lens)
        with pytest.raises(ValueError):
            cq.cq_kv8_read(cache, None, qs, k, k)
    with pytest.raises(ValueError):
        cq.cq_kv8_write(cache, x, x.half(), qs, lens)
    with pytest.raises(ValueError):
        cq.cq_kv8_write(cache, x, x, qs.long(), lens)
    with pytest.raises(ValueError):
        cq.cq_attn_kv8(x.half(), cache, qs, lens, 1, torch.zeros(3, 4, 128), None)
    with pytest.raises(ValueError):
        cq.cq_attn_kv8(x.half(), cache, qs, lens, 1, x, None, lse=torch.zeros(3, 1))


# ---- the reference of the GPU tests is itself checked ---------------------------------------------------------------

def test_reference_scale():
    for e in (-64, -20, 0, 5):
        s = 2.0 ** e
        assert kv8ref.least_scale(127 * s) == s
        assert kv8ref.least_scale(np.nextafter(127 * s, np.inf)) == 2 * s
    assert kv8ref.least_scale(0.0) == 2.0 ** -64 and kv8ref.least_scale(1e-40) == 2.0 ** -64
    assert math.isnan(kv8ref.least_scale(math.inf)) and math.isnan(kv8ref.least_scale(math.nan))


def test_reference_cache_is_near_its_input():
    rng = np.random.default_rng(1)
    c = kv8ref.Cache(1, 2, 64)
    x, y = rng.standard_normal((100, 2, 64)), rng.standard_normal((100, 2, 64))
    for i, j in ((0, 40), (40, 41), (41, 100)):
        c.write(0, x[i:j], y[i:j])
    for i, z in enumerate((x, y)):
        s = c.s[i][0][np.arange(100) // 32][:, :, None]
        assert np.all(np.abs(c.q[i][0]) <= 127)
        assert np.all(np.abs(c.values(i, 0) - z) <= 1.5 * s)      # one rounding, and one more for a block that grew


def test_reference_attention_by_differences():
    """The gradient of lse in the scores is the weights: the reference's output follows from differences of its lse."""
    rng = np.random.default_rng(2)
    c = kv8ref.Cache(1, 1, 64)
    c.write(0, rng.standard_normal((9, 1, 64)), rng.standard_normal((9, 1, 64)))
    q = rng.standard_normal((3, 2, 64))
    o, lse, *_ = kv8ref.attend(c, 0, q, 0.125, True, 0)
    k, v = c.values(0, 0)[:, 0], c.values(1, 0)[:, 0]
    s = 0.125 * np.einsum("nhd,kd->nhk", q, k)
    for i in range(3):
        hi = 9 - 3 + i + 1
        for h in range(2):
            def f(x):
                return math.log(sum(math.exp(t) for t in x[:hi]))
            w = [(f(s[i, h] + 1e-6 * np.eye(9)[j]) - f(s[i, h] - 1e-6 * np.eye(9)[j])) / 2e-6 for j in range(hi)]
            assert abs(f(s[i, h]) - lse[i, h]) < 1e-12
            assert np.allclose(np.array(w) @ v[:hi], o[i, h], atol=1e-8)
