"""The 8-bit cache and its attention at the edges of what their header allows,
against the plain 64-bit reference of kv8ref."""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import kv8ref
from cqtest import DEV
from test_gpu_kv8 import Setup, f64, i32, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_dev):
    import __graft_entry__
    __graft_entry__.build()


# one size for each attention kernel, by the query rows of a KV head: few, narrow, one row tile, two row tiles
FORMS = [(1, 4), (5, 4), (20, 4), (70, 4)]


# ---- windows and lengths -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 62, 2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("n,group", FORMS + [(16, 1)])
def test_windows_without_end(n, group, window):
    """A window past every length is no window, in sequences with more rows than tokens too."""
    held = [2, 0, 40]
    s = Setup(51, [100] * 3, 1, 64, 32)
    s.write(held)
    counts = [n, 1, n]
    q, o, z = s.check_attend(counts, group, window=window)
    _, o0, z0 = s.attend(counts, group, q=q)
    assert torch.equal(o, o0) and torch.equal(z, z0)


@pytest.mark.parametrize("n,group", FORMS)
def test_lengths_up_to_31_bits(n, group):
    """A table of one page over and over holds 2^31 tokens; attention declines lengths whose tokens' numbers would overflow."""
    s = Setup(52, [1024], 1, 64, 1024)
    table = torch.full((1, 2 ** 21 + 1), int(s.table[0, 0]), dtype=torch.int32, device=DEV)
    s.cache = cq.cq_kv8_cache(s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs, table)
    s.write([1024])
    q, o = s.rows(n, group, "bf16"), torch.zeros(n, group, 64, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(n, group, 1, 64, 1, n), dtype=torch.uint8, device=DEV)
    for L, status in ((2 ** 31 - 1, 5), (2 ** 31 - 2047, 5), (2 ** 31 - 2048, 0), (1024, 0)):
        cq.cq_attn_kv8(q, s.cache, starts([n]), i32([L]), n, o, ws, window=900)
        assert cq.cq_get_device_error() == status, L
    # the last window of the longest length is the page's: rows end at token 1023 of it
    cq.cq_attn_kv8(q, s.cache, starts([n]), i32([2 ** 31 - 2048]), n, o, ws, window=900)
    _, want, _ = s.attend([n], group, q=q, window=900)
    assert torch.equal(o, want)


# ---- waits that run out ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,group", FORMS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_wait_timeout_reports_status_and_the_next_call_is_right(n, group, out):
    """Copies that never come: the kernel ends by its limit and reports it, and what follows is as if it had not been."""
    s = Setup(53, [3000, 500], 2, 128, 64)
    s.write([3000, 500])
    q, want, z = s.attend([n, n], group, out=out)
    o = torch.empty_like(want)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(2 * n, 2 * group, 2, 128, 2, n), dtype=torch.uint8, device=DEV)
    old = cq.cq_get_option(cq.CQ_OPT_WAIT_NS)
    try:
        cq.cq_set_option(cq.CQ_OPT_WAIT_NS, 20_000_000)       # 20 ms
        cq.cq_set_option(cq.CQ_OPT_TEST_STALL, 1)
        cq.cq_attn_kv8(q, s.cache, starts([n, n]), i32(s.len), n, o, ws)
        assert cq.cq_get_option(cq.CQ_OPT_TEST_STALL) == 0     # of one call only
        assert cq.cq_get_device_error() == 8                   # CQ_ERR_TIMEOUT
        assert cq.cq_get_device_error() == 0
    finally:
        cq.cq_set_option(cq.CQ_OPT_WAIT_NS, old)
        cq.cq_set_option(cq.CQ_OPT_TEST_STALL, 0)
    _, o, z2 = s.attend([n, n], group, out=out, q=q)
    assert torch.equal(o, want) and torch.equal(z, z2)
