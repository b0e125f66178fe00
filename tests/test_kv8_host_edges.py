"""Host-side properties of the 8-bit cache's entry points that a program relies
on between calls."""
import pytest
import torch

import block_quantized_weight_02_gb300 as cq


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
