"""Host-side properties of the 8-bit cache's entry points that a program relies
on between calls."""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import kv8ref
import kv8tight


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_quantized_weight_02_gb300 import build
    build.build()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (40, 8), (32, 4), (16, 1), (64, 1)])
def test_workspace_grows_with_every_size(Hq, Hkv, D):
    """A buffer for the largest call serves the smaller ones: 25 rows of a head must not take less than one."""
    f = cq.cq_attn_kv8_workspace_bytes
    size = 0
    for q in range(1, 201):
        size, last = f(4000, Hq, Hkv, D, 64, q), size
        assert size >= last > -1
    for q in (1, 5, 33, 200):
        for a, b in ((q, 4000), (4000, 4001), (4000, 500000)):
            assert f(a, Hq, Hkv, D, 64, q) <= f(b, Hq, Hkv, D, 64, q)
        assert f(4000, Hq, Hkv, D, 1, q) <= f(4000, Hq, Hkv, D, 64, q) <= f(4000, Hq, Hkv, D, 4000, q)
    assert f(3, Hq, Hkv, D, 3, 1) <= f(15, Hq, Hkv, D, 3, 5)


def cache(pages=4, Hkv=2, page=64, D=128, table=None):
    return cq.cq_kv8_cache.empty(pages, Hkv, page, D, torch.zeros(3, 2, dtype=torch.int32) if table is None else table, "cpu")


def test_descriptor_follows_the_tensors():
    """A table or pool that is put in place of another is the one that calls get."""
    c, new = cache(), cache(9)
    c.table = torch.ones(5, 7, dtype=torch.int32)
    assert (c.desc.table, c.desc.ldt, c.desc.B, c.B) == (c.table.data_ptr(), 7, 5, 5) and c.table.shape == (5, 7)
    for name in ("Kq", "Vq", "Ks", "Vs"):
        t = getattr(c, name).clone()
        setattr(c, name, t)
        assert getattr(c, name) is t and getattr(c.desc, name) == t.data_ptr()
        assert c._ref._obj is c.desc
    before = {n: getattr(c, n) for n in ("Kq", "Ks", "Vq", "Vs", "table")}
    for name, t in (("Kq", new.Kq), ("Vs", new.Vs), ("Vq", c.Vq.float()), ("table", c.table.long()), ("table", c.table.t())):
        with pytest.raises(ValueError):
            setattr(c, name, t)
        for n, x in before.items():
            assert getattr(c, n) is x and getattr(c.desc, n) == x.data_ptr()


def test_table_rows_are_readable_to_their_pitch():
    """A length is checked against the pitch, so a wrong one may read up to it: not past the table's memory."""
    wide = torch.zeros(4, 8, dtype=torch.int32)
    for ok in (wide, wide[:, :3], wide[:3, 5:], wide[3:, 5:], wide[1:2, 2:4]):
        c = cache(table=ok)
        assert c.desc.table == ok.data_ptr()
    for bad in (wide[:, 5:], wide[2:, 1:4]):
        with pytest.raises(ValueError, match="pitch"):
            cache(table=bad)


# ---- the bounds of the GPU tests are themselves checked ----------------------------------------------------------

def one_term(cache, q, scale):
    """kv8tight.attend's causal output with every weight rounded to one fp16 term."""
    k, v = cache.values(0, 0)[:, 0], cache.values(1, 0)[:, 0]
    n, Hq, _ = q.shape
    o = np.zeros_like(q)
    for i in range(n):
        hi = len(k) - n + i + 1
        for h in range(Hq):
            s = scale * (k[:hi] @ q[i, h])
            w = np.exp(s - s.max())
            o[i, h] = (w * 2.0 ** 12).astype(np.float16).astype(float) / 2.0 ** 12 @ v[:hi] / w.sum()
    return o


@pytest.mark.parametrize("D", [64, 128])
def test_f32_bound_notices_a_missing_term(D):
    rng = np.random.default_rng(3)
    c = kv8ref.Cache(1, 1, D)
    c.write(0, rng.standard_normal((300, 1, D)), rng.standard_normal((300, 1, D)))
    q = rng.standard_normal((4, 4, D))
    for out, ok in (("bf16", True), ("f16", True), ("f32", False)):
        o, _, lim, _ = kv8tight.attend(c, 0, q, D ** -0.5, True, 0, out)
        assert np.all(np.abs(one_term(c, q, D ** -0.5) - o) <= lim) == ok
