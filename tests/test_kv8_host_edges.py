"""Host-side properties of the 8-bit cache's entry points that a program relies
on between calls."""
import pytest

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
