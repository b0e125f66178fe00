"""The 8-bit cache and its attention at the edges of what their header allows,
against the plain 64-bit reference of kv8ref."""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import kv8ref
from cqtest import DEV
from kv8tight import attend
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


# ---- values far apart --------------------------------------------------------------------------------------------

def check(s, counts, group, out, causal=True, window=0, **kw):
    q, o, z = s.attend(counts, group, out=out, causal=causal, window=window, **kw)
    at = 0
    for b, n in enumerate(counts):
        if n:
            ro, rz, eo, ez = attend(s.ref, b, f64(q[at:at + n]), s.D ** -0.5, causal, window, out)
            err = np.abs(f64(o[at:at + n]) - ro)
            assert np.all(err <= eo), (b, float(np.nanmax(err / np.maximum(eo, 1e-300))), int((~(err <= eo)).sum()), err.size)
            gz = f64(z[at:at + n])
            seen = np.isfinite(rz)
            assert np.array_equal(np.isneginf(gz), ~seen) and np.all(np.abs(gz[seen] - rz[seen]) <= ez[seen])
        at += n


FAR = [(2, 4), (5, 4), (2, 16), (20, 4), (12, 2), (70, 4), (64, 1), (200, 1)]


@pytest.mark.parametrize("n,group", FAR)
@pytest.mark.parametrize("bits", [20, 40, 70, 110])
@pytest.mark.parametrize("D,out", [(64, "bf16"), (128, "f32")])
def test_values_that_a_row_does_not_see(n, group, bits, D, out):
    """Large values in a block behind a row's position, or ahead of its window, are nothing to it."""
    s = Setup(54, [400], 1, D, 32)
    edge = 96
    v = s.rows(edge + n // 2, 1, "f32", 0.3)
    v[edge:] *= 2.0 ** bits                         # rows from n / 2 on see this block, those before it do not
    s.write([len(v)], "f32", k=s.rows(len(v), 1, "f32", 0.3), v=v)
    check(s, [n], group, out)
    s = Setup(55, [400], 1, D, 32)
    v = s.rows(edge + n, 1, "f32", 0.3)
    v[:32] *= 2.0 ** bits                           # rows before n / 2 see this block, later ones' windows begin behind it
    s.write([len(v)], "f32", k=s.rows(len(v), 1, "f32", 0.3), v=v)
    check(s, [n], group, out, window=65 + n // 2)


@pytest.mark.parametrize("n,group", [(1, 4)] + FAR)
@pytest.mark.parametrize("bits", [20, 40, 60])
@pytest.mark.parametrize("D,out", [(64, "bf16"), (128, "f32")])
def test_values_without_weight(n, group, bits, D, out):
    """Large values under scores far below the row's largest count as their weights do: here not at all."""
    for block in (0, 3, 7):
        s = Setup(56, [300], 1, D, 64)
        k, v = s.rows(300, 1, "f32", 0.3), s.rows(300, 1, "f32", 0.3)
        v[32 * block:32 * block + 32] *= 2.0 ** bits
        k[:, 0, 7] = 0
        k[32 * block:32 * block + 32, 0, 7] = -30
        s.write([300], "f32", k=k, v=v)
        q = s.rows(n, group, "bf16", 0.3)
        q[:, :, 7] = 100
        check(s, [n], group, out, q=q)


@pytest.mark.parametrize("n,group", [(1, 1)] + FAR)
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("D,out", [(64, "f32"), (128, "bf16")])
def test_values_and_scores_far_apart(n, group, seed, D, out):
    """Every block of a size of its own, from 2^-60 to 2^60, some zero, and scores of a level of its own."""
    s = Setup(100 + seed, [700], 1, D, 64)
    L = 330 + n + 50 * seed
    k, v = s.rows(L, 1, "f32", 0.3), s.rows(L, 1, "f32", 0.3)
    blocks = -(-L // 32)
    size = s.rng.uniform(-60, 60, blocks)
    level = -s.rng.uniform(0, 90, blocks)           # in units of 2: up to 2^90
    f = np.where(s.rng.random(blocks) < 0.2, 0.0, 2.0 ** size)
    at = np.arange(L) // 32
    v *= torch.from_numpy(f[at]).to(DEV).float()[:, None, None]
    k[:, 0, 7] = torch.from_numpy(level[at] * np.log(2) * D ** 0.5 / 100).to(DEV).float()
    s.write([L], "f32", k=k, v=v)
    q = s.rows(n, group, "bf16", 0.3)
    q[:, :, 7] = 100
    for causal, window in ((True, 0), (False, 0), (True, 100)):
        check(s, [n], group, out, causal, window, q=q)


# ---- scores that are not finite ----------------------------------------------------------------------------------

@pytest.mark.parametrize("n,group", [(1, 1)] + FAR)
@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_infinite_queries(n, group, dtype, out):
    """An infinity in a query makes every score of its row -inf, or +inf: NaN either way, not a row that sees nothing, in
    its own row only.  Short and long contexts, whole and in shares."""
    for L in (n, 150 + n, 3000 + n):
        s = Setup(57, [L], 1, 64, 64)
        k = s.rows(L, 1, "f32", 0.1)
        k[:, 0, 5] = 3.0
        s.write([L], "f32", k=k)
        for causal, window in ((True, 0), (False, 0), (True, 60)):
            q, o, z = s.attend([n], group, dtype, out, causal, window)
            assert torch.isfinite(o).all() and torch.isfinite(z).all()
            for inf in (float("-inf"), float("inf")):
                bad = q.clone()
                bad[n // 2, group - 1, 5] = inf
                _, o2, z2 = s.attend([n], group, dtype, out, causal, window, q=bad)
                assert torch.isnan(o2[n // 2, group - 1]).all() and torch.isnan(z2[n // 2, group - 1])
                keep = torch.ones(n, group, dtype=torch.bool, device=DEV)
                keep[n // 2, group - 1] = False
                assert torch.equal(o2[keep], o[keep]) and torch.equal(z2[keep], z[keep])


@pytest.mark.parametrize("n,group", [(1, 1)] + FAR)
@pytest.mark.parametrize("block", [0, 2, 40])
def test_some_scores_overflow(n, group, block):
    """Scores below f32's range in one block weigh nothing; the row is the mean of what it sees besides."""
    L = 1400
    s = Setup(58, [L + n], 1, 64, 64)
    k, v = torch.zeros(L + n, 1, 64, device=DEV), s.rows(L + n, 1, "f32", 0.3)
    k[32 * block:32 * block + 32, 0, 5] = 1e30
    s.write([L + n], "f32", k=k, v=v)
    q = torch.zeros(n, group, 64, device=DEV, dtype=torch.bfloat16)
    q[:, :, 5] = -1e38
    _, o, z = s.attend([n], group, q=q)
    values = s.ref.values(1, 0)[:, 0]
    for i in range(n):
        seen = np.arange(L + i + 1)
        seen = seen[seen // 32 != block]
        want, mass = values[seen].mean(0), np.abs(values[seen]).mean(0)
        assert np.all(np.abs(f64(o[i]) - want) <= 2.0 ** -15 * mass)
        assert np.all(np.abs(f64(z[i]) - np.log(len(seen))) <= 2.0 ** -14)


# ---- buffers and descriptors -------------------------------------------------------------------------------------

@pytest.mark.parametrize("most", [5, 20, 200])
def test_one_workspace_for_every_step(most):
    """A buffer for the longest guesses or prompts serves single tokens as well."""
    s = Setup(59, [700] * 3, 2, 128, 64)
    s.write([500, 300, 700])
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(3 * most, 10, 2, 128, 3, most), dtype=torch.uint8, device=DEV)
    for n in (1, 3, 5, 7, 20, 25, 200):
        if n <= most:
            q, want, _ = s.attend([n] * 3, 5)
            o = torch.empty_like(want)
            cq.cq_attn_kv8(q, s.cache, starts([n] * 3), i32(s.len), n, o, ws)
            assert torch.equal(o, want)


# ---- f32 outputs, element by element -----------------------------------------------------------------------------

@pytest.mark.parametrize("Hkv,group,counts,held", [
    (2, 4, [1, 1, 1, 1], [0, 40, 700, 1990]),             # single tokens
    (1, 3, [4, 1, 0, 5], [3, 300, 9, 1500]),              # up to 16 rows of a head
    (2, 5, [5, 1, 6, 3], [0, 64, 900, 1500]),             # up to 32
    (1, 8, [16, 7, 1, 12], [40, 0, 2000, 333]),           # up to 128
    (2, 2, [130, 1, 200, 40], [0, 700, 500, 1200]),       # more
])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 77), (False, 0)])
def test_f32_outputs(Hkv, group, counts, held, D, causal, window):
    s = Setup(60, [a + b for a, b in zip(held, counts)], Hkv, D, 64)
    s.write(held, spread=0.4)
    s.write(counts, spread=0.4)
    check(s, counts, group, "f32", causal, window)


@pytest.mark.parametrize("n,group", [(1, 4), (5, 5), (20, 4), (60, 4)])
def test_f32_outputs_joined(n, group):
    """One long sequence: its work is cut into a share for every SM, and partials are joined."""
    s = Setup(61, [12000], 1, 64, 128)
    s.write([12000 - n], spread=0.4)
    s.write([n], spread=0.4)
    check(s, [n], group, "f32")
    check(s, [n], group, "f32", window=5000)


# ---- rejected tokens ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rejected_tokens(dtype):
    """Lengths that go back and are written over: a block that keeps tokens keeps its scale (and its NaN) too, one that
    is begun again does not."""
    s = Setup(62, [200, 200, 200], 2, 64, 32)
    s.write([70, 33, 64], dtype)
    for keep, new, big in (([66, 31, 64], [5, 5, 1], 8.0), ([64, 33, 40], [7, 1, 30], 1.0), ([65, 32, 0], [1, 40, 3], 0.01),
                           ([60, 70, 2], [100, 1, 31], 1.0)):
        k, v = s.rows(sum(new), 2, "f32", 0.5) * big, s.rows(sum(new), 2, "f32", 0.5) * big
        k, v = k.to(kv8ref.TORCH[dtype]), v.to(kv8ref.TORCH[dtype])
        if big == 1.0:
            v[3, 1, 9] = float("inf")
        s.len = [a + b for a, b in zip(keep, new)]
        cq.cq_kv8_write(s.cache, k, v, starts(new), i32(s.len))
        assert cq.cq_get_device_error() == 0
        at = 0
        for b, n in enumerate(new):
            s.ref.write(b, f64(k[at:at + n]), f64(v[at:at + n]), at=keep[b])
            at += n
        s.check_values()


# ---- calls in a chain --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,group", FORMS)
def test_calls_in_a_chain(n, group):
    """Writes and attention that follow each other without a pause see each other's results: queries and tokens from the
    kernel before, blocks whose scale grows from step to step, one workspace."""
    s = Setup(63, [400, 400], 2, 64, 32)
    s.write([50, 200])
    steps = [(s.rows(2 * n, 2, "bf16", 0.5) * 1.3 ** i, s.rows(2 * n, 2, "bf16", 0.5) * 1.3 ** i, s.rows(2 * n, 2 * group, "bf16", 0.3))
             for i in range(30)]
    counts, first = [n, n], [50, 200]
    last = [[min(400, a + n * (i % 3 + 1)) for a in first] for i in range(30)]
    lens = [i32(x) for x in last]
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(2 * n, 2 * group, 2, 64, 2, n), dtype=torch.uint8, device=DEV)
    before = [t.clone() for t in (s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs)]
    k, v, q = (torch.empty_like(t) for t in steps[0])
    qs = starts(counts)

    def run(pause):
        for t, b in zip((s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs), before):
            t.copy_(b)
        out = []
        for i, x in enumerate(steps):
            for t, y in zip((k, v, q), x):
                t.copy_(y)
                pause()
            o, z = torch.empty(2 * n, 2 * group, 64, device=DEV), torch.empty(2 * n, 2 * group, device=DEV)
            for f in (lambda: cq.cq_kv8_write(s.cache, k.bfloat16(), v.bfloat16(), qs, lens[i]),
                      lambda: cq.cq_attn_kv8(q.bfloat16(), s.cache, qs, lens[i], n, o, ws, lse=z)):
                f()
                pause()
            out += [o, z]
        torch.cuda.synchronize()
        return out

    want, got = run(torch.cuda.synchronize), run(lambda: None)
    assert cq.cq_get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# ---- sums that the tensor cores truncate -------------------------------------------------------------------------

@pytest.mark.parametrize("n,group", [(1, 4), (1, 16), (5, 5), (16, 4), (150, 1)])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_long_sums_of_one_sign(n, group, out, D):
    """Values of one sign over 40960 tokens that one SM (few rows: one warp) takes in turn.  Truncation shrinks such sums
    the most, all alike: the results' projection on the exact ones may be off by 5e-6 for f32 outputs (a window of 128
    products, at most 4.3e-8 each) and 7e-5 for 16-bit ones (1024 products, measured at most 6.6e-8 each)."""
    B, Hkv, L, page = 64, 16, 40960, 1024
    s = Setup(64, [L], Hkv, D, page, spare=0)
    s.len = [L]
    k, v = s.rows(L, Hkv, "bf16", 0.3), s.rows(L, Hkv, "bf16", 0.3).abs()
    cq.cq_kv8_write(s.cache, k, v, starts([L]), i32([L]))
    k, v = (x.double().transpose(0, 1) for x in s.read("f32"))
    s.cache = cq.cq_kv8_cache(s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs, s.table.repeat(B, 1))   # all over the same pages
    s.B, s.len = B, [L] * B
    q, o, _ = s.attend([n] * B, group, "f16", out, causal=False, lse=False)
    for b in (0, 30, 63):
        x = q[b * n:b * n + n].double().view(n, Hkv, group, D).permute(1, 0, 2, 3).reshape(Hkv, n * group, D)
        w = torch.softmax(x @ k.transpose(1, 2) * D ** -0.5, 2)
        ref = (w @ v).view(Hkv, n, group, D).transpose(0, 1).reshape(n, Hkv * group, D)
        err = o[b * n:b * n + n].double() - ref
        along = float((err * ref).sum() / (ref * ref).sum())
        assert abs(along) <= (5e-6 if out == "f32" else 7e-5), along
