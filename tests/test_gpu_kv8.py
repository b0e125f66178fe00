"""GPU parity of the 8-bit key/value cache and its attention against the plain
64-bit reference of kv8ref: the codes and scales exactly, the attention
within bounds that follow from its roundings."""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import kv8ref
from kv8ref import BLOCK, TORCH

from cqtest import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_dev):
    import __graft_entry__
    __graft_entry__.build()


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device=DEV)


def starts(counts):
    return i32(np.concatenate([[0], np.cumsum(counts)]))


def f64(t):
    return t.double().cpu().numpy()


class Setup:
    """A cache whose pages lie in random order, everything not written to left as garbage, beside its reference."""

    def __init__(self, seed, caps, Hkv, D, page, spare=2):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(DEV).manual_seed(seed)
        per = [max(1, -(-c // page)) for c in caps]
        pages = sum(per) + spare
        order = self.rng.permutation(pages)
        table = np.full((len(caps), max(per) + 1), -7, np.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).to(DEV)
        pool = lambda: torch.randint(-127, 128, (pages, Hkv, page, D), generator=self.gen, device=DEV, dtype=torch.int8)
        scale = lambda: torch.full((pages, Hkv, page // BLOCK), float("nan"), device=DEV)
        self.cache = cq.cq_kv8_cache(pool(), scale(), pool(), scale(), self.table)
        self.ref = kv8ref.Cache(len(caps), Hkv, D)
        self.B, self.Hkv, self.D = len(caps), Hkv, D
        self.len = [0] * len(caps)

    def rows(self, n, heads, dtype, spread=1.0):
        x = torch.randn(n, heads, self.D, generator=self.gen, device=DEV)
        return (x * torch.exp(spread * torch.randn(n, heads, 1, generator=self.gen, device=DEV))).to(TORCH[dtype])

    def write(self, counts, dtype="bf16", k=None, v=None, spread=1.0):
        T = sum(counts)
        k = self.rows(max(T, 1), self.Hkv, dtype, spread) if k is None else k
        v = self.rows(max(T, 1), self.Hkv, dtype, spread) if v is None else v
        self.len = [a + c for a, c in zip(self.len, counts)]
        cq.cq_kv8_write(self.cache, k, v, starts(counts), i32(self.len))
        assert cq.cq_get_device_error() == 0
        at = 0
        for b, c in enumerate(counts):
            if c:
                self.ref.write(b, f64(k[at:at + c]), f64(v[at:at + c]))
            at += c

    def read(self, dtype="f32", first=None, counts=None):
        first = [0] * self.B if first is None else first
        counts = [n - f for n, f in zip(self.len, first)] if counts is None else counts
        k = torch.full((max(sum(counts), 1), self.Hkv, self.D), 77.0, dtype=TORCH[dtype], device=DEV)
        v = torch.full_like(k, 78.0)
        cq.cq_kv8_read(self.cache, i32(first), starts(counts), k, v)
        assert cq.cq_get_device_error() == 0
        return k, v

    def check_values(self):
        k, v = self.read("f32")
        for i, t in enumerate((k, v)):
            want = [self.ref.values(i, b) for b in range(self.B)]
            got = f64(t)[:sum(self.len)]
            assert np.array_equal(got, np.concatenate(want), equal_nan=True)

    def attend(self, counts, group, dtype="bf16", out="f32", causal=True, window=0, scale=None, lse=True, q=None, max_q=None):
        Hq, T = self.Hkv * group, sum(counts)
        q = self.rows(T, Hq, dtype, 0.3) if q is None else q
        o = torch.full((T, Hq, self.D), float("nan"), dtype=TORCH[out], device=DEV)
        z = torch.full((T, Hq), float("nan"), device=DEV) if lse else None
        max_q = max(counts) if max_q is None else max_q
        size = cq.cq_attn_kv8_workspace_bytes(T, Hq, self.Hkv, self.D, self.B, max_q)
        ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device=DEV)   # NaN wherever it is read as f32
        cq.cq_attn_kv8(q, self.cache, starts(counts), i32(self.len), max_q, o, ws, scale=scale, causal=causal,
                       window=window, lse=z)
        assert cq.cq_get_device_error() == 0
        return q, o, z

    def check_attend(self, counts, group, dtype="bf16", out="f32", causal=True, window=0, scale=None, **kw):
        q, o, z = self.attend(counts, group, dtype, out, causal, window, scale, **kw)
        s = self.D ** -0.5 if scale is None else float(np.float32(scale))
        at = 0
        for b, n in enumerate(counts):
            if not n:
                continue
            ro, rz, mass, top, reach = kv8ref.attend(self.ref, b, f64(q[at:at + n]), s, causal, window)
            go = f64(o[at:at + n])
            lim = kv8ref.bound(ro, mass, top, reach, out)
            err = np.abs(go - ro)
            assert np.all(err <= lim), (b, float(np.nanmax(err / np.maximum(lim, 1e-300))), np.isnan(go).sum())
            if z is not None:
                gz = f64(z[at:at + n])
                seen = np.isfinite(rz)
                assert np.array_equal(np.isneginf(gz), ~seen)
                assert np.all(np.abs(gz[seen] - rz[seen]) <= kv8ref.lse_bound(rz, reach)[seen])
            at += n
        return q, o, z


# ---- writing and reading back ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 32), (3, 128, 96), (8, 128, 64), (2, 64, 256)])
def test_write_then_read(dtype, Hkv, D, page):
    """Ragged prompts (none, one token, block edges), then more tokens behind them."""
    s = Setup(11, [200, 200, 200, 300, 40], Hkv, D, page)
    s.write([0, 1, 31, 33, 32], dtype)
    s.check_values()
    s.write([5, 31, 66, 0, 1], dtype, spread=2.0)
    s.check_values()
    s.write([100, 1, 1, 200, 0], dtype)
    s.check_values()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_write_token_by_token(dtype):
    """The block's scale grows as larger tokens arrive; the kept codes are rounded again each time."""
    s = Setup(12, [70, 70], 2, 64, 32)
    for t in range(70):
        k = s.rows(2, 2, dtype, 0.1) * (1.07 ** t)
        s.write([1, 1], dtype, k=k.to(TORCH[dtype]))
    s.check_values()


def test_write_scale_edges():
    """127 * 2^e is the largest value of its scale, the next f32 takes the next one; zeros; tiny and huge values."""
    s = Setup(13, [400], 1, 64, 64)
    edge = [127.0 * 2.0 ** -9, float(np.nextafter(np.float32(127.0 * 2.0 ** -9), np.float32(1))), 0.0, 1e-30, 2.0 ** -58,
            127.0 * 2.0 ** -64, 3.0e38, 63.5, 1.0, 2.0 ** -66, 1e-44]
    k = torch.zeros(32 * len(edge), 1, 64, device=DEV)
    for i, e in enumerate(edge):
        k[32 * i:32 * i + 32, 0] = torch.linspace(-1, 1, 32 * 64, device=DEV).view(32, 64) * e
        k[32 * i + 3, 0, 5] = e
    s.write([len(k)], "f32", k=k, v=-k)
    s.check_values()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_write_not_finite(dtype):
    """An infinity or NaN makes its block of its head read as NaN, until the block is written again from its start."""
    s = Setup(14, [128], 2, 128, 32)
    k = s.rows(70, 2, dtype)
    k[10, 0, 3] = float("inf")
    k[40, 1, 100] = float("nan")
    s.write([70], dtype, k=k)
    s.check_values()
    s.write([3], dtype)
    s.check_values()
    kk, _ = s.read("f32")
    assert torch.isnan(kk[:32, 0]).all() and not torch.isnan(kk[:32, 1]).any()
    assert torch.isnan(kk[32:64, 1]).all() and not torch.isnan(kk[32:, 0]).any()
    s.ref = kv8ref.Cache(1, 2, 128)
    s.len = [0]
    s.write([60], dtype)
    s.check_values()


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_read_ranges(out):
    """Any token range of each sequence, every output type; rows outside stay as they were."""
    s = Setup(15, [100, 100, 10], 3, 64, 32)
    s.write([97, 64, 5], "bf16")
    first, counts = [33, 0, 4], [40, 64, 1]
    k, v = s.read(out, first, counts)
    for i, t in enumerate((k, v)):
        want = np.concatenate([s.ref.values(i, b, f, f + n) for b, (f, n) in enumerate(zip(first, counts))])
        want = torch.from_numpy(want).to(TORCH[out])
        assert torch.equal(t.cpu(), want)
    k, v = s.read(out, [5, 5, 5], [0, 7, 0])
    assert torch.equal(k.cpu(), torch.from_numpy(s.ref.values(0, 1, 5, 12)).to(TORCH[out]))


def test_pitched_rows():
    """q, k and v as slices of one projection's rows, the output inside a wider tensor."""
    s = Setup(16, [150, 90], 2, 128, 64)
    T, group = 100, 3
    qkv = torch.randn(T, (group + 1) * 2 + 2, 128, generator=s.gen, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:10]
    s.write([60, 40], "bf16", k=k, v=v)
    s.check_values()
    wide = torch.full((T, 9, 128), 5.0, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, 6, 2, 128, 2, 60), dtype=torch.uint8, device=DEV)
    cq.cq_attn_kv8(q, s.cache, starts([60, 40]), i32(s.len), 60, wide[:, 1:7], ws)
    _, o, _ = s.check_attend([60, 40], group, q=q)
    assert torch.equal(wide[:, 1:7], o)
    assert (wide[:, 0] == 5).all() and (wide[:, 7:] == 5).all()
    kw = torch.full((T, 5, 128), 5.0, device=DEV)
    cq.cq_kv8_read(s.cache, None, starts(s.len), kw[:, :2], kw[:, 2:4])
    assert torch.equal(kw[:, :2].double().cpu(), torch.from_numpy(np.concatenate([s.ref.values(0, b) for b in (0, 1)])))
    assert (kw[:, 4] == 5).all()


# ---- attention ---------------------------------------------------------------------------------------------------

LENS = [1, 2, 31, 32, 33, 64, 100, 257, 700]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("Hkv,group,D,page", [(2, 1, 64, 32), (1, 8, 128, 64), (3, 3, 128, 96), (2, 16, 64, 128),
                                              (1, 64, 128, 32), (4, 5, 128, 256), (1, 24, 64, 32)])
def test_single_tokens(dtype, out, Hkv, group, D, page):
    s = Setup(21, LENS, Hkv, D, page)
    s.write(LENS, dtype)
    s.check_attend([1] * len(LENS), group, dtype, out)


@pytest.mark.parametrize("window", [0, 1, 7, 32, 100, 5000])
def test_single_tokens_window(window):
    s = Setup(22, LENS, 2, 64, 32)
    s.write(LENS, "f16")
    s.check_attend([1] * len(LENS), 4, "f16", "f32", window=window)


@pytest.mark.parametrize("Hkv,group,D,page", [(2, 1, 64, 32), (2, 4, 128, 64), (1, 8, 128, 96), (1, 5, 64, 32), (1, 16, 128, 128)])
@pytest.mark.parametrize("counts", [[2, 3, 1, 0, 4], [5, 5, 5, 5, 5], [8, 1, 7, 6, 2]])
def test_few_tokens(Hkv, group, D, page, counts):
    held = [0, 40, 300, 9, 95]
    s = Setup(23, [a + b for a, b in zip(held, counts)], Hkv, D, page)
    s.write(held)
    s.write(counts)
    s.check_attend(counts, group)
    s.check_attend(counts, group, window=20)
    s.check_attend(counts, group, causal=False)


@pytest.mark.parametrize("Hkv,group,D,page", [(1, 1, 128, 32), (2, 4, 64, 64), (1, 7, 128, 96), (1, 32, 64, 32)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (True, 200)])
def test_prompts(Hkv, group, D, page, causal, window):
    """Prompts and chunks behind kept context: one row, tile edges, ragged."""
    held, counts = [0, 0, 200, 3, 130, 0], [1, 129, 70, 200, 16, 0]
    s = Setup(24, [a + b for a, b in zip(held, counts)], Hkv, D, page)
    s.write(held)
    s.write(counts)
    s.check_attend(counts, group, causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_prompt_types(dtype, out):
    s = Setup(25, [333], 2, 128, 64)
    s.write([333], dtype)
    s.check_attend([333], 2, dtype, out)


@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 1, 2], [40, 1, 60]])
def test_empty_rows(counts):
    """Empty sequences, and more rows than tokens: rows that see nothing give 0 and -inf."""
    held = [0, 5, min(2, counts[2])]
    s = Setup(26, [8, 8, 8], 2, 128, 32)
    s.write(held)
    for causal in (True, False):
        _, o, z = s.check_attend(counts, 4, causal=causal)
        assert (o[:counts[0]] == 0).all() and torch.isneginf(z[:counts[0]]).all()


@pytest.mark.parametrize("n", [1, 60])
def test_scales_far_apart(n):
    """Values whose blocks differ by 2^40 and zero blocks, peaked and flat scores."""
    s = Setup(27, [320], 1, 64, 32)
    k, v = s.rows(320, 1, "f32", 0.1), s.rows(320, 1, "f32", 0.1)
    for i, f in enumerate([1.0, 2.0 ** -20, 0.0, 2.0 ** 20, 1e-3, 0.0, 2.0 ** -19, 30.0, 2.0 ** 18, 1.0]):
        v[32 * i:32 * i + 32] *= f
    k[100:140] *= 6
    s.write([320], "f32", k=k, v=v)
    s.check_attend([n], 4)
    s.check_attend([n], 4, scale=2.0)
    s.check_attend([n], 4, scale=1e-4)


@pytest.mark.parametrize("n", [1, 60])
def test_large_and_growing_scores(n):
    """Scores in the hundreds that rise along the sequence, so the running maximum moves in every block; and their mirror."""
    for sign in (1.0, -1.0):
        s = Setup(28, [500], 1, 128, 64)
        k = s.rows(500, 1, "f32", 0.1) * 0.05
        k[:, 0, 7] = sign * torch.linspace(-30, 30, 500, device=DEV)
        s.write([500], "f32", k=k)
        q = s.rows(n, 4, "bf16", 0.1)
        q[:, :, 7] = 100.0
        s.check_attend([n], 4, q=q)


@pytest.mark.parametrize("n,group", [(1, 4), (3, 5), (5, 5), (8, 4), (25, 4), (100, 4)])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e9])
def test_huge_scores(n, group, size):
    """Scores whose own rounding is far above 1: the largest one's value is the result, to the last weight."""
    s = Setup(39, [300], 2, 128, 64)
    k = s.rows(300, 2, "f32", 0.1) * size
    s.write([300], "f32", k=k)
    q = (s.rows(n, 2 * group, "f32", 0.1) * size).bfloat16()
    for out in ("f32", "bf16"):
        _, o, z = s.attend([n], group, out=out, q=q)
        assert torch.isfinite(o).all() and torch.isfinite(z).all()
        kc, vc, go = s.ref.values(0, 0), s.ref.values(1, 0), f64(o)
        near = 0
        for i in range(n):
            L = 300 - n + i + 1
            for h in range(2 * group):
                x = f64(q[i, h]) * 128 ** -0.5
                sc = kc[:L, h // group] @ x
                reach = (np.abs(kc[:L, h // group]) @ np.abs(x)).max()
                a, b = np.argsort(sc)[::-1][:2]
                if sc[a] - sc[b] < 100 + 2.0 ** -14 * reach:      # apart by more than the scores' error, e^-100 of the rest
                    near += 1
                    continue
                v = vc[a, h // group]
                u = 2.0 ** -20 if out == "f32" else 2.0 ** -8
                assert np.all(np.abs(go[i, h] - v) <= u * np.abs(v) + 1e-30), (i, h)
        assert near < n * 2 * group / 2


@pytest.mark.parametrize("n", [1, 60])
def test_query_range(n):
    """bf16 queries beyond fp16's range, tiny ones, and a row of zeros."""
    s = Setup(29, [200], 2, 64, 32)
    s.write([200], "bf16", spread=0.1)
    q = s.rows(n, 8, "bf16", 0.1)
    q[0, 0] *= 1e6
    q[0, 1] *= 1e-9
    q[0, 2] = 0
    q[-1, 3] *= 3e30
    s.check_attend([n], 4, q=q, scale=1e-6)


@pytest.mark.parametrize("n", [1, 20, 60])
def test_not_finite_stays_in_its_rows(n):
    """NaN queries spoil their own row; a spoilt block spoils the rows that see it and no others."""
    s = Setup(30, [200], 1, 64, 32)
    s.write([199 - 32])
    k = s.rows(33, 1, "bf16")
    s.write([33], k=k)
    q, o, _ = s.attend([n], 4)
    q2 = q.clone()
    q2[0, 1] = float("nan")
    _, o2, _ = s.attend([n], 4, q=q2)
    assert torch.isnan(o2[0, 1]).all()
    keep = torch.ones(n, 4, dtype=torch.bool, device=DEV)
    keep[0, 1] = False
    assert torch.equal(o2[keep], o[keep])
    # token 0's block becomes NaN: a window keeps the last rows clear of it
    page, row = int(s.table[0, 0]), 0
    for pool in (s.cache.Ks, s.cache.Vs):
        old = pool[page, 0, row].item()
        pool[page, 0, row] = float("nan")
        _, bad, _ = s.attend([n], 4, q=q)
        assert torch.isnan(bad).all()
        _, fine, _ = s.attend([n], 4, q=q, window=100)
        pool[page, 0, row] = old
        _, want, _ = s.attend([n], 4, q=q, window=100)
        assert torch.equal(fine, want) and not torch.isnan(fine).any()


@pytest.mark.parametrize("n", [40, 130])
def test_spoilt_block_ahead_of_rows(n):
    """A block with scale NaN inside the rows' own tile spoils only rows at or past its first token."""
    s = Setup(31, [160], 1, 64, 32)
    s.write([n])
    q, o, _ = s.attend([n], 2)
    for pool in (s.cache.Ks, s.cache.Vs):
        page = int(s.table[0, 1])
        old = pool[page, 0, 0].item()
        pool[page, 0, 0] = float("nan")
        _, bad, _ = s.attend([n], 2, q=q)
        pool[page, 0, 0] = old
        assert torch.equal(bad[:32], o[:32]) and torch.isnan(bad[32:]).all()


@pytest.mark.parametrize("B,Hkv,group,L,n", [(1, 1, 4, 20000, 1), (2, 2, 8, 9000, 1), (1, 1, 1, 5000, 6), (1, 1, 4, 6000, 50)])
def test_long_contexts(B, Hkv, group, L, n):
    """Few rows over many tokens: the work is split along the tokens and joined."""
    lens = [L - 37 * b for b in range(B)]
    s = Setup(32, lens, Hkv, 128, 128)
    for b in range(B):
        k, v = s.rows(lens[b], Hkv, "bf16", 0.5), s.rows(lens[b], Hkv, "bf16", 0.5)
        s.write([lens[b] if i == b else 0 for i in range(B)], k=k, v=v)
    s.check_attend([n] * B, group)


def test_mixed_batch():
    """One long prompt among single tokens, in one call."""
    held = [0, 700, 33, 0, 1500, 64]
    counts = [300, 1, 1, 1, 1, 2]
    s = Setup(33, [a + b for a, b in zip(held, counts)], 2, 128, 64)
    s.write(held)
    s.write(counts)
    s.check_attend(counts, 4, "bf16", "bf16")


def test_many_sequences():
    lens = [(7 * i) % 90 for i in range(300)]
    s = Setup(34, [n + 1 for n in lens], 1, 64, 32)
    s.write(lens)
    s.write([1] * 300)
    s.check_values()
    s.check_attend([1] * 300, 2)


def exact(s, q, counts, causal, window):
    """kv8ref.attend for a batch, in 64 bits on the device, from the cache as cq_kv8_read gives it (exact in f32)."""
    kc, vc = (x.double() for x in s.read("f32"))
    cols = [[], [], [], [], []]
    at = tok = 0
    for n, L in zip(counts, s.len):
        k, v = kc[tok:tok + L].transpose(0, 1), vc[tok:tok + L].transpose(0, 1)            # [Hkv][L][D]
        x = q[at:at + n].double().view(n, s.Hkv, -1, s.D).permute(1, 2, 0, 3).flatten(1, 2)  # [Hkv][group n][D]
        p = torch.arange(L - n, L, device=DEV).repeat(x.shape[1] // max(n, 1))[:, None]
        j = torch.arange(L, device=DEV)[None]
        see = (j <= p) & (j > p - (window or L + 1)) if causal else torch.ones_like(j <= p)
        z = (x @ k.transpose(1, 2) * s.D ** -0.5).masked_fill(~see, float("-inf"))
        lse = torch.logsumexp(z, 2)
        w = torch.exp(z - lse[..., None])
        reach = ((x.abs() @ k.abs().transpose(1, 2)) * s.D ** -0.5).masked_fill(~see, 0).amax(2)
        top = torch.where(see, v.abs().amax(2)[:, None], 0.0).amax(2)
        for c, t in zip(cols, (w @ v, lse[..., None], w @ v.abs(), top[..., None], reach[..., None])):
            c.append(t.view(s.Hkv, -1, n, t.shape[2]).permute(2, 0, 1, 3).flatten(1, 2).cpu().numpy())
        at, tok = at + n, tok + L
    o, lse, mass, top, reach = (np.concatenate(c) for c in cols)
    return o, lse[..., 0], mass, top[..., 0], reach[..., 0]


@pytest.mark.parametrize("Hkv,group,B,rows,held", [
    (16, 1, 1, [1], [3, 200, 40, 900]),               # single tokens
    (16, 4, 48, [1, 2, 4], [1, 300, 70, 900]),        # up to 16 rows of a head
    (16, 5, 48, [5, 1, 4, 5], [1, 300, 70, 900]),     # up to 25
    (16, 8, 48, [4, 3], [1, 300, 70, 900]),           # 32
    (16, 11, 32, [3, 1], [5, 700, 100]),              # 33
    (16, 2, 48, [64, 1, 33], [0, 300, 70, 900]),      # 128
    (16, 1, 32, [256, 100, 30, 600], [1500, 2000, 1100]),   # items whose second half has rows and ones where it has none
    (8, 3, 24, [43, 200, 86, 1], [1300, 10, 700]),
])
@pytest.mark.parametrize("D,out", [(128, "bf16"), (128, "f32"), (64, "f32")])
def test_several_items_a_block(Hkv, group, B, rows, held, D, out):
    """More items than the GPU has room for at once, each unlike the one before it: rows, lengths, and values whose size
    differs by 2^16 from sequence to sequence."""
    counts = [rows[b % len(rows)] for b in range(B)]
    lens = [held[b % len(held)] + counts[b] for b in range(B)]
    s = Setup(38, lens, Hkv, D, 64)
    v = s.rows(sum(lens), Hkv, "f32", 0.5)
    at = 0
    for b, n in enumerate(lens):
        v[at:at + n] *= 2.0 ** (16 * (b % 2))
        at += n
    s.len = lens
    cq.cq_kv8_write(s.cache, s.rows(sum(lens), Hkv, "f32", 0.5), v, starts(lens), i32(lens))
    q = s.rows(sum(counts), Hkv * group, "bf16", 0.3)
    for causal, window in ((True, 0), (True, 150), (False, 0)):
        ro, rz, mass, top, reach = exact(s, q, counts, causal, window)
        lim = kv8ref.bound(ro, mass, top, reach, out)
        first = None
        for _ in range(3):
            _, o, z = s.attend(counts, group, "bf16", out, causal, window, q=q)
            assert first is None or torch.equal(o, first)
            first = o
        assert np.all(np.abs(f64(o) - ro) <= lim)
        assert np.all(np.abs(f64(z) - rz) <= kv8ref.lse_bound(rz, reach))


@pytest.mark.parametrize("n,group", [(1, 2), (3, 4), (5, 5), (60, 1), (200, 1), (1000, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_long_shares(n, group, D):
    """f32 outputs where one SM adds up thousands of tokens.  An accumulator takes at most 256 truncated sums (16 steps of
    16 products), on average a quarter of 2^-24 of it each: 4e-6; scores and weights add 2e-6 and less."""
    B, Hkv = 20, 16
    lens = [6000 - 31 * b for b in range(B)]
    s = Setup(40, lens, Hkv, D, 128)
    s.len = lens
    cq.cq_kv8_write(s.cache, s.rows(sum(lens), Hkv, "f32", 0.3), s.rows(sum(lens), Hkv, "f32", 0.3), starts(lens), i32(lens))
    counts = [n if b < 3 or n < 100 else 1 for b in range(B)]
    q, o, z = s.attend(counts, group, "f16", "f32")
    ro, rz, _, _, reach = exact(s, q, counts, True, 0)
    assert np.linalg.norm(f64(o) - ro) <= 1e-5 * np.linalg.norm(ro)
    assert np.all(np.abs(f64(z) - rz) <= kv8ref.lse_bound(rz, reach))


def test_max_q_larger_than_the_batch():
    """max_q only has to bound the rows: the result stays within the same bounds."""
    s = Setup(35, [100, 50], 2, 64, 32)
    s.write([100, 50])
    for mq in (1, 3, 17, 1000):
        s.check_attend([1, 1], 4, max_q=mq)


@pytest.mark.parametrize("counts", [[1, 1, 1], [90, 3, 200]])
def test_same_bits_every_time(counts):
    s = Setup(36, [400, 300, 2000], 2, 128, 64)
    s.write([400, 300, 2000])
    q, o, z = s.attend(counts, 4)
    for _ in range(5):
        _, o2, z2 = s.attend(counts, 4, q=q)
        assert torch.equal(o, o2) and torch.equal(z, z2)


def test_other_stream_and_graph():
    """On a side stream and replayed from a captured graph, with new lengths in the same buffers."""
    s = Setup(37, [300, 300], 2, 128, 64)
    s.write([100, 200])
    k, v, q = s.rows(2, 2, "bf16"), s.rows(2, 2, "bf16"), s.rows(2, 8, "bf16")
    o = torch.empty(2, 8, 128, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(2, 8, 2, 128, 2, 1), dtype=torch.uint8, device=DEV)
    lens, qs = i32([101, 201]), starts([1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = [t.clone() for t in (s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs)]

    def step():
        cq.cq_kv8_write(s.cache, k, v, qs, lens)
        cq.cq_attn_kv8(q, s.cache, qs, lens, 1, o, ws)

    with torch.cuda.stream(side):
        step()
        assert cq.cq_get_device_error() == 0
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    for t, b in zip((s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs), before):
        t.copy_(b)
    for _ in range(40):
        k.copy_(s.rows(2, 2, "bf16"))
        g.replay()
        s.len = [n + 1 for n in s.len]
        lens += 1
        torch.cuda.synchronize()
        for b in range(2):
            s.ref.write(b, f64(k[b:b + 1]), f64(v[b:b + 1]))
    s.check_values()
    _, want, _ = s.check_attend([1, 1], 4, q=q)
    assert torch.equal(o, want)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 codes, its last pages in use, and rows of more than 2^31 elements in all."""
    pages, Hkv, page, D = 40000, 8, 128, 128
    n = 300
    pools = [torch.zeros(pages, Hkv, page, D, dtype=torch.int8, device=DEV) for _ in range(2)]
    scales = [torch.full((pages, Hkv, page // 32), float("nan"), device=DEV) for _ in range(2)]
    table = i32([pages - 1, pages - 3, pages - 2]).view(1, 3)
    s = Setup(38, [n], Hkv, D, page)
    s.cache = cq.cq_kv8_cache(pools[0], scales[0], pools[1], scales[1], table)
    s.write([n])
    s.check_values()
    s.check_attend([1], 2)
    s.check_attend([n], 2)
    wide = torch.zeros(n, 8 * 1024 * 1024, dtype=torch.bfloat16, device=DEV)   # 2.5e9 elements
    q = wide.as_strided((n, 16, D), (8 * 1024 * 1024, D, 1))
    q.copy_(s.rows(n, 16, "bf16", 0.3))
    _, o, _ = s.check_attend([n], 2, q=q)
    wide.zero_()
    out = wide.as_strided((n, 16, D), (8 * 1024 * 1024, D, 1))
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(n, 16, Hkv, D, 1, n), dtype=torch.uint8, device=DEV)
    q2 = s.rows(n, 16, "bf16", 0.3)
    cq.cq_attn_kv8(q2, s.cache, starts([n]), i32([n]), n, out, ws)
    _, o, _ = s.attend([n], 2, q=q2, out="bf16")
    assert torch.equal(out, o)


# ---- what the device refuses -------------------------------------------------------------------------------------

def _bad(call):
    call()
    assert cq.STATUS[cq.cq_get_device_error()] == "CQ_ERR_INDEX"
    assert cq.cq_get_device_error() == 0


@pytest.mark.parametrize("n", [1, 100])
def test_device_errors(n):
    s = Setup(41, [128, 128], 2, 64, 32)
    s.write([128, 100])
    k = s.rows(2 * n, 2, "bf16")
    q, o = s.rows(2 * n, 4, "bf16"), torch.zeros(2 * n, 4, 64, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(2 * n, 4, 2, 64, 2, 2 * n), dtype=torch.uint8, device=DEV)
    att = lambda qs, lens, mq=2 * n, cache=s.cache: cq.cq_attn_kv8(q, cache, i32(qs), i32(lens), mq, o, ws)
    wr = lambda qs, lens, cache=s.cache: cq.cq_kv8_write(cache, k, k, i32(qs), i32(lens))
    rd = lambda qs, first: cq.cq_kv8_read(s.cache, i32(first), i32(qs), k.clone(), k.clone())
    ok = [0, n, 2 * n]
    for f in (att, wr):
        _bad(lambda: f([0, n, 2 * n + 1], [128, 128]))
        _bad(lambda: f([0, n, n - 1], [128, 128]))
        _bad(lambda: f([-1, n, 2 * n], [128, 128]))
        _bad(lambda: f(ok, [128, 10 ** 6]))
        _bad(lambda: f(ok, [-1, 128]))
    _bad(lambda: wr(ok, [n - 1, 128]))
    _bad(lambda: rd(ok, [0, -1]))
    _bad(lambda: rd(ok, [0, 10 ** 6]))
    if n > 1:
        _bad(lambda: att(ok, [128, 128], n - 1))
    for pid in (-1, s.cache.Kq.shape[0]):
        t = s.table.clone()
        t[1, 0] = pid
        broken = cq.cq_kv8_cache(s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs, t)
        _bad(lambda: att(ok, [128, 128], cache=broken))
        _bad(lambda: wr(ok, [128, min(n, 128)], cache=broken))
    # and the stream goes on as if nothing had been
    s = Setup(42, [128, 128], 2, 64, 32)
    s.write([128, 100])
    s.check_attend([1, 1], 2)
