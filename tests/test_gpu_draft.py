"""GPU parity of a drafting step against the 64-bit references of draftref: rotary positions
and masked attention within bounds that follow from their roundings, the cache's codes as
those of rotated keys, the check of drafted tokens exactly."""
import bisect
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_quantized_weight_02_gb300 as cq
import draftref
import kv8ref
from kv8ref import BLOCK, TORCH
from test_gpu_kv8 import Setup, f64, i32, starts

from cqtest import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_dev):
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def freqs(rot, base=10000.0):
    return torch.tensor(base ** (-np.arange(rot // 2) * 2.0 / rot), dtype=torch.float32, device=DEV)


LAYOUT = {"half": cq.CQ_ROPE_HALF, "pairs": cq.CQ_ROPE_PAIRS}


# ---- rotary positions -----------------------------------------------------------------------------------------------

def check_rope(x, y, pos, freq, layout, out, mag=1.0):
    a = f64(x)
    want = draftref.rotate(a, pos, f64(freq), layout, mag)
    e = draftref.rotate_bound(a, pos, f64(freq), layout, mag)
    rot = 2 * len(freq)
    e[:, :, rot:] = 0.0
    e += draftref.rounding(np.abs(want) + e, out)
    d = np.abs(f64(y) - want)
    assert np.all(d <= e), float((d / e).max())
    if out == {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[x.dtype]:
        assert torch.equal(y[:, :, rot:], x[:, :, rot:])


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 16, 16), (1, 32, 128, 128), (7, 3, 96, 48), (33, 5, 80, 80), (130, 2, 256, 64), (3, 1, 1024, 1024)])
def test_rope(layout, dtype, out, T, H, D, rot):
    g = gen(T * 7 + H)
    x = torch.randn(T, H, D, generator=g, device=DEV).to(TORCH[dtype])
    pos = torch.randint(0, 200000, (T,), generator=g, device=DEV).int()
    f = freqs(rot)
    y = torch.full((T, H, D), 55.0, dtype=TORCH[out], device=DEV)
    cq.cq_rope(x, cq.cq_rope_spec(f, LAYOUT[layout], 1.25), pos, y)
    check_rope(x, y, pos.tolist(), f, layout, out, 1.25)


def test_rope_any_position():
    """Positions of all 31 bits and below zero, frequencies from 0 to just under the limit and of both signs."""
    f = torch.tensor([0.0, 1.0, -1.0, 1e-3, 3.14159274, 300.5, 1e-6, 2.0 ** -70], device=DEV)
    pos = i32([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 2 ** 24 + 1])
    x = torch.randn(8, 2, 16, generator=gen(5), device=DEV)
    y = torch.empty_like(x)
    cq.cq_rope(x, cq.cq_rope_spec(f), pos, y)
    # (the reference's own angles, from 64-bit products, are what limits this one: the bound holds them)
    check_rope(x, y, pos.tolist(), f, "half", "f32")
    # against integers: frequency 1 at position 355 * k and so on is known from exact reductions
    from fractions import Fraction
    import math
    two_pi = Fraction(math.pi) * 2 + Fraction(2.4492935982947064e-16)        # pi to 2^-106
    big = f.cpu().double().numpy()
    for t, p in enumerate(pos.tolist()):
        for i, fr in enumerate(big):
            a = Fraction(float(fr)) * p
            r = float(a - round(a / two_pi) * two_pi)
            u, v = f64(x)[t, :, i], f64(x)[t, :, i + 8]
            assert np.all(np.abs(f64(y)[t, :, i] - (u * math.cos(r) - v * math.sin(r))) <= 2.0 ** -22 * (np.abs(u) + np.abs(v)))


def test_rope_not_finite():
    x = torch.randn(2, 1, 32, generator=gen(6), device=DEV)
    x[0, 0, 3], x[1, 0, 20] = float("inf"), float("nan")
    f = torch.tensor([1.0] * 4 + [float("inf"), float("nan"), 65536.0, 65535.0], device=DEV)
    y = torch.empty_like(x)
    cq.cq_rope(x, cq.cq_rope_spec(f), i32([3, 0]), y)
    bad = torch.isnan(y) | torch.isinf(y)
    want = torch.zeros_like(bad)
    want[0, 0, 3] = want[0, 0, 11] = True                       # an infinite channel spoils its pair
    want[:, :, 4:7] = want[:, :, 12:15] = True                  # frequencies that are no number, or too large
    want[1, 0, 20] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_in_place_and_pitched(layout, dtype):
    """Queries and keys are columns of one product's rows; each is turned in place, nothing else moves."""
    T, HQ, HKV, D = 45, 6, 2, 64
    y = torch.randn(T, HQ + 2 * HKV + 1, D, generator=gen(8), device=DEV).to(TORCH[dtype])
    before = y.clone()
    r = cq.cq_rope_spec(freqs(32), LAYOUT[layout])
    pos = torch.arange(100, 100 + T, device=DEV).int()
    cq.cq_rope(y[:, :HQ], r, pos)
    cq.cq_rope(y[:, HQ:HQ + HKV], r, pos)
    check_rope(before[:, :HQ + HKV], y[:, :HQ + HKV], pos.tolist(), r.freq, layout, dtype)
    assert torch.equal(y[:, HQ + HKV:], before[:, HQ + HKV:])
    # and from some columns to others of the same rows
    z = before.clone()
    cq.cq_rope(z[:, :HKV], r, pos, z[:, HQ:HQ + HKV])
    assert torch.equal(z[:, :HQ], before[:, :HQ]) and torch.equal(z[:, HQ + HKV:], before[:, HQ + HKV:])
    check_rope(before[:, :HKV], z[:, HQ:HQ + HKV], pos.tolist(), r.freq, layout, dtype)
    with pytest.raises(cq.CQError):
        cq.cq_rope(y[:, :HQ], r, pos, y[:, 1:HQ + 1])


def test_rope_offsets_past_32_bits():
    """Rows whose last elements lie past 2^31: a pitch of 2^20 elements and 2100 rows."""
    if torch.cuda.mem_get_info()[0] < 10 << 30:
        pytest.skip("needs 10 GB")
    T, ld = 2100, 1 << 20
    buf = torch.zeros(T * ld, dtype=torch.float16, device=DEV)
    x = buf.as_strided((T, 1, 64), (ld, 64, 1), 128)
    x.copy_(torch.randn(T, 1, 64, generator=gen(9), device=DEV))
    before = x.clone()
    r = cq.cq_rope_spec(freqs(64))
    pos = torch.arange(T, device=DEV).int()
    cq.cq_rope(x, r, pos)
    check_rope(before[-3:], x[-3:], pos.tolist()[-3:], r.freq, "half", "f16")
    assert not buf[:128].any() and not buf[-ld + 192:].any()


# ---- appending rotated keys -----------------------------------------------------------------------------------------

def rotated(s, k, v, counts, r, layout, pos=None):
    """Writes to the cache and to its reference (keys rotated as cq_rope does it, in f32: kv8ref rounds the same numbers)."""
    s.len = [a + c for a, c in zip(s.len, counts)]
    place = [p for n, c in zip(s.len, counts) for p in range(n - c, n)]
    kr = torch.empty(k.shape, dtype=torch.float32, device=DEV)
    cq.cq_rope(k, r, i32(place) if pos is None else pos, kr)
    cq.cq_kv8_write_rope(s.cache, k, v, starts(counts), i32(s.len), r, pos)
    assert cq.cq_get_device_error() == 0
    at = 0
    for b, c in enumerate(counts):
        if c:
            s.ref.write(b, f64(kr[at:at + c]), f64(v[at:at + c]))
        at += c


def same(s):
    """Codes and scales are the reference's, bit for bit."""
    k, v = s.read("f32")
    at = 0
    for b, n in enumerate(s.len):
        for i, x in enumerate((k, v)):
            np.testing.assert_array_equal(f64(x[at:at + n]), s.ref.values(i, b))
        at += n


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv,D,page,rot", [(1, 128, 32, 128), (2, 64, 96, 64), (3, 128, 64, 48), (5, 64, 32, 16), (8, 128, 128, 112)])
def test_append(layout, dtype, Hkv, D, page, rot):
    """Prompts, then single tokens (some sequences without), keys at their places."""
    s = Setup(rot + Hkv, [200, 40, 70, 33], Hkv, D, page)
    r = cq.cq_rope_spec(freqs(rot), LAYOUT[layout])
    for counts in ([150, 0, 64, 1], [1, 1, 1, 1], [33, 31, 0, 30], [1, 0, 1, 1]):
        T = max(sum(counts), 1)
        rotated(s, s.rows(T, Hkv, dtype), s.rows(T, Hkv, dtype), counts, r, layout)
    same(s)


def test_append_is_the_rotation():
    """Not only as cq_rope: what is read back is within a code's rounding (two for tokens that a growing block moved) of the 64-bit rotation."""
    s = Setup(3, [90, 300], 2, 128, 64)
    r = cq.cq_rope_spec.make(96, kind=cq.CQ_ROPE_RAMP, factor=16.0, low=1.0, high=32.0, trained=8192.0, layout=cq.CQ_ROPE_PAIRS)
    counts = [90, 300]
    k, v = s.rows(390, 2, "bf16", 0.3), s.rows(390, 2, "bf16", 0.3)
    pos = torch.randint(0, 1 << 20, (390,), generator=gen(4), device=DEV).int()
    rotated(s, k, v, counts, r, "pairs", pos)
    same(s)
    want = draftref.rotate(f64(k), pos.tolist(), f64(r.freq), "pairs", r.desc.mag)
    got = f64(s.read("f32")[0])
    step = np.concatenate([s.ref.s[0][b][np.arange(n) // BLOCK] for b, n in enumerate(counts)])[:, :, None]
    assert np.all(np.abs(got - want) <= step * (0.5 + 2.0 ** -12))


def test_append_siblings_and_pitch():
    """Drafted siblings share a position; rows are columns of a product."""
    s = Setup(11, [64, 64], 2, 64, 32)
    r = cq.cq_rope_spec(freqs(64))
    for counts, pos in (([20, 33], None), ([6, 5], i32([20, 21, 21, 22, 22, 22, 33, 34, 34, 34, 35]))):
        T = sum(counts)
        y = s.rows(T, 7, "bf16")
        rotated(s, y[:, 1:3], y[:, 4:6], counts, r, "half", pos)
    same(s)


def test_append_not_finite():
    """A channel that is not finite spoils its block's keys, and no other's."""
    s = Setup(12, [96], 2, 64, 32)
    r = cq.cq_rope_spec(freqs(32))
    k, v = s.rows(96, 2, "bf16"), s.rows(96, 2, "bf16")
    k[40, 1, 5] = float("inf")
    rotated(s, k, v, [96], r, "half")
    back = s.read("f32")[0]
    assert torch.isnan(back[32:64, 1]).all()
    assert torch.isfinite(back[:, 0]).all() and torch.isfinite(back[:32, 1]).all() and torch.isfinite(back[64:, 1]).all()
    same_v = s.read("f32")[1]
    np.testing.assert_array_equal(f64(same_v), s.ref.values(1, 0))


def test_append_device_errors():
    s = Setup(13, [64, 64], 2, 64, 32)
    r = cq.cq_rope_spec(freqs(64))
    k, v = s.rows(8, 2, "bf16"), s.rows(8, 2, "bf16")
    pools = [t.clone() for t in (s.cache.Kq, s.cache.Vq)]
    used = set(s.table.flatten().tolist())
    for qs, lens in (([0, 4, 3], [4, 4]), ([0, 4, 9], [4, 5]), ([0, 4, 8], [3, 4]), ([0, 4, 8], [4, 1 << 20]), ([-1, 4, 8], [5, 4])):
        cq.cq_kv8_write_rope(s.cache, k, v, i32(qs), i32(lens), r)
        assert cq.cq_get_device_error() == 5
    s.cache.table[1, 0] = 1 << 20
    cq.cq_kv8_write_rope(s.cache, k, v, i32([0, 4, 8]), i32([4, 4]), r)
    assert cq.cq_get_device_error() == 5
    for t, old in zip((s.cache.Kq, s.cache.Vq), pools):
        rest = [p for p in range(t.shape[0]) if p not in used]
        assert torch.equal(t[rest], old[rest])


# ---- attention for trees --------------------------------------------------------------------------------------------

def run_tree(s, counts, bits, dtype, out, group, lse=True, max_q=None, width=None, q=None):
    """The last counts[b] tokens of each sequence as rows with their bits; checked against the reference."""
    T, Hq = sum(counts), s.Hkv * group
    most = max(counts) if max_q is None else max_q
    width = (most + 31) // 32 if width is None else width
    q = s.rows(T, Hq, dtype, 0.3) if q is None else q
    o = torch.full((T, Hq, s.D), 99.0, dtype=TORCH[out], device=DEV)
    l = torch.full((T, Hq), 99.0, device=DEV) if lse else None
    mask = torch.from_numpy(draftref.words([x for b in bits for x in b], width)).to(DEV)
    size = cq.cq_attn_kv8_workspace_bytes(T, Hq, s.Hkv, s.D, s.B, most)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)               # NaN wherever it is read as f32
    cq.cq_attn_kv8_tree(q, s.cache, starts(counts), i32(s.len), most, mask, o, ws, lse=l)
    assert cq.cq_get_device_error() == 0
    at = 0
    for b, n in enumerate(counts):
        if n:
            want, z, e, ez = draftref.attend(s.ref, b, f64(q[at:at + n]), s.D ** -0.5, bits[b], out)
            d = np.abs(f64(o[at:at + n]) - want)
            assert np.all(d <= e), (b, float((d / e).max()))
            if lse:
                y = f64(l[at:at + n])
                assert np.array_equal(np.isinf(y), np.isinf(z))
                ok = np.isfinite(z)
                assert np.all(np.abs(y[ok] - z[ok]) <= ez[ok])
        at += n
    return o, l


def trees_of(rng, counts):
    return [draftref.bits_of(draftref.tree(rng, n)) if n else [] for n in counts]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("Hkv,group,D,page,counts,held", [
    (2, 1, 128, 32, [1, 5, 8], [0, 31, 100]),                   # few rows: one tile of eight
    (1, 4, 64, 64, [4, 1, 3, 2], [300, 0, 64, 7]),              # two tiles
    (2, 5, 128, 64, [6, 2, 5], [33, 700, 127]),                 # the narrow kernel
    (1, 1, 64, 96, [32, 17, 31], [5, 250, 96]),
    (2, 4, 128, 32, [26, 9, 0, 32], [130, 1, 40, 512]),         # one row tile, masks across a step's border
    (1, 1, 64, 64, [100, 128], [125, 260]),                     # masks of several words
    (1, 8, 128, 128, [40, 64], [1000, 90]),                     # two row tiles
    (2, 3, 64, 32, [150, 90], [77, 0])])
def test_trees(dtype, out, Hkv, group, D, page, counts, held):
    rng = np.random.default_rng(sum(counts))
    s = Setup(D + group, [n + h for n, h in zip(counts, held)], Hkv, D, page)
    s.write(held, "bf16", spread=0.5)
    s.write(counts, "bf16", spread=0.5)
    run_tree(s, counts, trees_of(rng, counts), dtype, out, group)


@pytest.mark.parametrize("group,n", [(1, 5), (2, 8), (4, 8), (4, 30), (8, 40)])
def test_any_mask(group, n):
    """Bits need not be a tree's: rows that see nothing of the last tokens, later tokens, all of them; bits past the last row
    count for nothing."""
    rng = np.random.default_rng(n)
    held = [0, 60, 200]
    s = Setup(n, [h + n for h in held], 2, 64, 32)
    s.write(held, "bf16")
    s.write([n] * 3, "bf16")
    bits = [[int.from_bytes(rng.bytes(8), "little") for _ in range(n)] for _ in held]
    for b in bits:
        b[0], b[1], b[2], b[3] = 0, (1 << 64) - 1, 1 << (n - 1), (1 << 64) - (1 << n)
    o, l = run_tree(s, [n] * 3, bits, "f16", "f32", group, width=2)
    for row in (0, 3):                                          # of the sequence without context
        assert not o[row].any() and torch.isinf(l[row]).all() and (l[row] < 0).all()


@pytest.mark.parametrize("group,n", [(1, 6), (3, 8), (4, 20), (8, 40)])
def test_more_rows_than_tokens(group, n):
    """Rows whose own tokens were taken back: bits of tokens that are not there count for nothing."""
    s = Setup(n + 1, [n + 4, n], 1, 64, 32)
    s.write([n - 3, n], "bf16")
    bits = [[(1 << n) - 1] * n, trees_of(np.random.default_rng(1), [n])[0]]
    bits[0][0], bits[0][1] = 7, 15                              # tokens -3 to -1; and token 0
    o, l = run_tree(s, [n, n], bits, "bf16", "f32", group)
    assert not o[0].any() and torch.isinf(l[0]).all()


@pytest.mark.parametrize("n,group", [(4, 2), (4, 4), (8, 4), (16, 4), (40, 8)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_hidden_values_that_are_not_finite(n, group, out):
    """The last drafted tokens' block is spoilt: rows that see no token of it stay right."""
    held, D = 64, 64
    s = Setup(n, [held + n], 1, D, 32)
    s.write([held], "bf16")
    s.write([n], "bf16")
    last = (n - 1) // 32 * 32                                   # the spoilt block's first row
    page = s.table[0, (held + last) // 32].item()
    s.cache.Ks[page, 0, 0] = s.cache.Vs[page, 0, 0] = float("nan")
    bits = [x & (1 << last) - 1 for x in trees_of(np.random.default_rng(n), [n])[0]]
    run_tree(s, [n], [bits], "bf16", out, group)


@pytest.mark.parametrize("counts,held,Hkv,group", [([5, 5, 5], [4000, 30, 9000], 2, 3), ([8], [20000], 1, 4), ([26, 30], [5000, 11000], 2, 4), ([64], [30000], 1, 8)])
def test_long_trees(counts, held, Hkv, group):
    """Contexts that are split over many SMs: the joins meet the mask too."""
    rng = np.random.default_rng(7)
    s = Setup(21, [n + h for n, h in zip(counts, held)], Hkv, 128, 64)
    s.write(held, "bf16", spread=0.3)
    s.write(counts, "bf16", spread=0.3)
    run_tree(s, counts, trees_of(rng, counts), "bf16", "bf16", group)


@pytest.mark.parametrize("counts,group", [([3, 4], 2), ([6, 4], 5), ([20, 26], 4), ([40, 64], 8)])
def test_chain_is_the_causal_call(counts, group):
    """A chain's mask gives what cq_attn_kv8 gives: each is within 2^-15 of its weighted values."""
    held = [300, 1000]
    s = Setup(31, [n + h for n, h in zip(counts, held)], 2, 128, 64)
    s.write(held, "bf16")
    s.write(counts, "bf16")
    T, Hq, most = sum(counts), 2 * group, max(counts)
    q = s.rows(T, Hq, "bf16")
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, Hq, 2, 128, 2, most), dtype=torch.uint8, device=DEV)
    a, b = torch.empty(T, Hq, 128, device=DEV), torch.empty(T, Hq, 128, device=DEV)
    mask = torch.from_numpy(draftref.words([(2 << i) - 1 for n in counts for i in range(n)], (most + 31) // 32)).to(DEV)
    cq.cq_attn_kv8(q, s.cache, starts(counts), i32(s.len), most, a, ws)
    cq.cq_attn_kv8_tree(q, s.cache, starts(counts), i32(s.len), most, mask, b, ws)
    assert cq.cq_get_device_error() == 0
    assert float((a - b).abs().max()) <= 2.0 ** -14 * max(np.abs(s.ref.values(1, b)).max() for b in range(2))


def test_tree_mask_pitch_and_spare_words():
    """A mask that is a slice of wider rows, with more words than the batch needs; max_q above the batch's."""
    counts, held = [7, 3], [50, 90]
    s = Setup(41, [70, 100], 1, 64, 32)
    s.write(held, "bf16")
    s.write(counts, "bf16")
    bits = trees_of(np.random.default_rng(3), counts)
    T, Hq = 10, 2
    wide = torch.full((T, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 4:7] = torch.from_numpy(draftref.words([x for b in bits for x in b], 3)).to(DEV)
    q = s.rows(T, Hq, "f16")
    for max_q in (7, 10):
        o = torch.empty(T, Hq, 64, device=DEV)
        ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, Hq, 1, 64, 2, max_q), dtype=torch.uint8, device=DEV)
        cq.cq_attn_kv8_tree(q, s.cache, starts(counts), i32(s.len), max_q, wide[:, 4:7], o, ws)
        at = 0
        for b, n in enumerate(counts):
            want, _, e, _ = draftref.attend(s.ref, b, f64(q[at:at + n]), 0.125, bits[b], "f32")
            assert np.all(np.abs(f64(o[at:at + n]) - want) <= e)
            at += n


@pytest.mark.parametrize("n", [2, 8, 30, 64])
def test_tree_device_errors(n):
    s = Setup(51, [100, 100], 1, 64, 32)
    s.write([n, n], "bf16")
    T = 2 * n
    q, o = s.rows(T, 2, "bf16"), torch.full((T + 1, 2, 64), 7.0, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, 2, 1, 64, 2, n), dtype=torch.uint8, device=DEV)
    mask = torch.full((T, 2), -1, dtype=torch.int32, device=DEV)
    for qs, lens in (([0, n, n - 1], s.len), ([0, n, T + 1], s.len), ([0, n, T], [n, 1 << 20]), ([0, n - 1, T], s.len)):
        cq.cq_attn_kv8_tree(q, s.cache, i32(qs), i32(lens), n, mask, o[:T], ws)
        assert cq.cq_get_device_error() == 5
        assert (o[T] == 7.0).all()


# ---- check of drafted tokens ----------------------------------------------------------------------------------------

def probabilities(g, rows, V, dtype, sharp):
    """Rows [rows][V] of a wider tensor whose other columns are NaN."""
    n = 16 // (4 if dtype == "f32" else 2)
    x = torch.full((rows, (V + n - 1) // n * n + n), float("nan"), dtype=TORCH[dtype], device=DEV)
    x[:, :V] = torch.softmax(sharp * torch.randn(rows, V, generator=g, device=DEV), 1).to(TORCH[dtype])
    return x[:, :V]


def check_verify(P, Q, tokens, parents, counts, u, u_last, width=None, tree=True, pad=0):
    T, B, most = sum(counts), len(counts), max(max(counts), 1) if width is None else width
    mask = None
    if tree:
        w = draftref.words([x for p in parents for x in draftref.bits_of(p)], (most + 31) // 32)
        mask = torch.from_numpy(w).to(DEV)
    out = torch.full((B, most + pad), 777, dtype=torch.int32, device=DEV)
    path, count = out.clone(), torch.full((B,), 777, dtype=torch.int32, device=DEV)
    cq.cq_verify(P, tokens, starts(counts), most, u, u_last, out, path, count, Q=Q, mask=mask)
    assert cq.cq_get_device_error() == 0
    p, q, at = f64(P), None if Q is None else f64(Q), 0
    tk, uu, ul = tokens.tolist(), f64(u), f64(u_last)
    for b, n in enumerate(counts):
        if n == 0:
            want, rows = [], []
        else:
            want, rows = draftref.verify(p[at:at + n], None if q is None else q[at:at + n], tk[at:at + n], parents[b], uu[at:at + n], ul[b])
        assert count[b].item() == max(len(rows) - 1, 0), b
        assert out[b].tolist() == want + [-1] * (most - len(want)) + [777] * pad, b
        assert path[b].tolist() == [at + r for r in rows] + [-1] * (most - len(rows)) + [777] * pad, b
        at += n


def drafted(g, Q, parents, counts, V):
    """Tokens drawn from Q at their parents."""
    at = np.concatenate([[0], np.cumsum(counts)])
    up = torch.tensor([max(p, 0) + at[b] for b, ps in enumerate(parents) for p in ps], device=DEV)
    return torch.multinomial(torch.nan_to_num(Q[up].float()) + 1e-20, 1, generator=g)[:, 0].int()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,counts", [(1, [1, 2]), (2, [3, 1, 4]), (7, [5, 0, 6, 1]), (100, [8] * 20), (1003, [12, 3, 30]), (40001, [6, 5, 9]), (150001, [4, 7])])
def test_verify(tree, drawn, dtype, V, counts):
    g, rng = gen(V + tree), np.random.default_rng(V)
    T = sum(counts)
    P, Q = probabilities(g, T, V, dtype, 2.0), probabilities(g, T, V, dtype, 1.5)
    parents = [(draftref.tree(rng, n) if tree else list(range(-1, n - 1))) if n else [] for n in counts]
    for _ in range(4):
        u, ul = torch.rand(T, generator=g, device=DEV), torch.rand(len(counts), generator=g, device=DEV)
        check_verify(P, Q if drawn else None, drafted(g, Q, parents, counts, V), parents, counts, u, ul, tree=tree, pad=3)


@pytest.mark.parametrize("B", [1, 3, 8, 40, 200])
def test_verify_batches(B):
    """As many clusters as there are sequences, of each size."""
    g, rng = gen(B), np.random.default_rng(B)
    counts = [int(c) for c in rng.integers(1, 6, B)]
    T, V = sum(counts), 30000
    P = probabilities(g, T, V, "f32", 3.0)
    Q = probabilities(g, T, V, "f32", 3.0)
    parents = [list(range(-1, n - 1)) for n in counts]
    u, ul = 0.3 * torch.rand(T, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
    check_verify(P, Q, drafted(g, Q, parents, counts, V), parents, counts, u, ul, tree=False)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_siblings(drawn):
    """Many children of one row, the same token several times: each rejection lessens what is left."""
    g, V, n = gen(5), 50, 40
    P, Q = probabilities(g, n, V, "f32", 1.0), probabilities(g, n, V, "f32", 1.0)
    parents = [[-1] + [0] * (n - 1)]
    for i in range(30):
        tokens = torch.randint(0, 6 if i % 2 else V, (n,), generator=g, device=DEV).int()
        u = 0.5 + 0.5 * torch.rand(n, generator=g, device=DEV) if i % 3 else torch.rand(n, generator=g, device=DEV)
        check_verify(P, Q if drawn else None, tokens, parents, [n], u, torch.rand(1, generator=g, device=DEV))


def test_verify_1024_rows():
    g, rng, n, V = gen(6), np.random.default_rng(6), 1024, 300
    P, Q = probabilities(g, n, V, "f32", 1.0), probabilities(g, n, V, "f32", 1.0)
    for parents in (list(range(-1, n - 1)), draftref.tree(rng, n, 0.9)):
        u = 0.05 * torch.rand(n, generator=g, device=DEV)
        check_verify(P, Q, drafted(g, Q, [parents], [n], V), [parents], [n], u, torch.rand(1, generator=g, device=DEV))


def test_verify_edges():
    """Draws of 0, of 1 and beyond; certain tokens; nothing left; nothing at all; entries that are no probabilities."""
    V = 70
    z = lambda n: torch.zeros(n, 72, device=DEV)[:, :V]         # (rows start on 16 bytes)
    f = lambda *v: torch.tensor(v, dtype=torch.float32, device=DEV)
    one = z(2)
    one[:, 9] = 1.0
    chain = [[-1, 0]]
    for u in (0.0, 0.5, 1.0):
        for ul in (0.0, 0.999, 1.0, 2.0):
            check_verify(one, one, i32([0, 9]), chain, [2], f(0.0, u), f(ul), tree=False)       # u = 1: rejected, nothing left: P again
            check_verify(one, None, i32([0, 9]), chain, [2], f(0.0, u), f(ul), tree=False)
            check_verify(one, one, i32([0, 3]), chain, [2], f(0.0, u), f(ul), tree=False)
            check_verify(z(2), one, i32([0, 9]), chain, [2], f(0.0, u), f(ul), tree=False)      # -1
            check_verify(z(2), None, i32([0, 9]), chain, [2], f(0.0, u), f(ul), tree=False)
    odd = z(2)
    odd[:, 9] = 1.0
    odd[:, 0], odd[:, 2], odd[:, 3], odd[:, 60] = float("nan"), -1.0, -float("inf"), 0.25
    for ul in (0.0, 0.79, 0.81, 1.0):
        check_verify(odd, odd, i32([0, 60]), chain, [2], f(0.0, 0.9), f(ul), tree=False)
        check_verify(odd, None, i32([0, 0]), chain, [2], f(0.0, 0.0), f(ul), tree=False)
    out, path, count = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((1, 2), (1, 2), (1,)))
    for k in (0, 35, 69):                                                                       # an infinite entry: some token, no more
        x = z(2)
        x.copy_(odd)
        x[:, k] = float("inf")
        for Q in (x, odd, None):
            cq.cq_verify(x, i32([0, 60]), i32([0, 2]), 2, f(0.0, 0.9), f(0.5), out, path, count, Q=Q)
            assert cq.cq_get_device_error() == 0 and -1 <= out[0, count.item()].item() < V
    flat = z(1) + 1.0 / 64
    for k in range(V):                                                                          # borders met exactly
        check_verify(flat, None, i32([0]), [[-1]], [1], f(0.0), f(k / V), tree=False)
    tiny = z(1) + 1e-44
    check_verify(tiny, None, i32([0]), [[-1]], [1], f(0.0), f(0.5), tree=False)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_numbers_out_of_range(drawn):
    """Random numbers of 1 and more, negative ones and NaN: nothing without a probability stands or is drawn."""
    g, V, n = gen(14), 40, 12
    P, Q = probabilities(g, n, V, "f32", 1.0), probabilities(g, n, V, "f32", 1.0)
    P[:, ::3] = 0.0
    nan = float("nan")
    for i, u in enumerate(([1.0] * n, [1.5] * n, [3.0] * n, [-1.0] * n, [nan] * n, [nan, 2.0, 0.5] * 4)):
        for ul in (1.0, 7.0, -2.0, nan):
            for parents in ([-1] + [0] * (n - 1), list(range(-1, n - 1))):
                tokens = torch.randint(0, V, (n,), generator=g, device=DEV).int()
                check_verify(P, Q if drawn else None, tokens, [parents], [n], torch.tensor(u, device=DEV), torch.tensor([ul], device=DEV))


def test_verify_next_to_borders():
    """Draws as near to a border as f32 numbers come, over a vocabulary whose running sums 32 bits cannot hold."""
    g, V = gen(8), 120000
    P = probabilities(g, 1, V, "f32", 2.0)
    cum = np.cumsum(f64(P)[0])
    ks = np.random.default_rng(8).integers(0, V, 40)
    for k in ks:
        at = np.float32(cum[k] / cum[-1])
        for ul in (np.nextafter(at, np.float32(0)), at, np.nextafter(at, np.float32(2))):
            # 64-bit sums in two orders differ by 2^-53 a term: draws that lie nearer to a border than 2^-40 say nothing
            if np.abs(float(ul) * cum[-1] - cum[max(k - 9, 0):k + 9]).min() > 2.0 ** -40:
                check_verify(P, None, i32([0]), [[-1]], [1], torch.zeros(1, device=DEV), torch.tensor([ul], device=DEV), tree=False)


def test_verify_unreachable_rows_and_masks():
    """Rows without a parent are left out; bits of a row itself and after it do not count."""
    g, V, n = gen(9), 30, 6
    P = probabilities(g, n, V, "f32", 1.0)
    tokens = i32([0, 1, 2, 3, 4, 5])
    u = torch.zeros(n, device=DEV)                                     # whatever has a parent stands
    out, path = torch.empty(1, n, dtype=torch.int32, device=DEV), torch.empty(1, n, dtype=torch.int32, device=DEV)
    count = torch.empty(1, dtype=torch.int32, device=DEV)
    mask = i32([0, -2, 0b000101 | 0b111000, 0, 0b000111, 0b010000]).view(n, 1)
    cq.cq_verify(P, tokens, i32([0, n]), n, u, torch.zeros(1, device=DEV), out, path, count, mask=mask)
    # 1: bits 1 up: no parent; 2: parent 0; 3: none; 4: parent 2; 5: parent 4
    assert path[0, :4].tolist() == [0, 2, 4, 5] and count.item() == 3 and out[0, :3].tolist() == [2, 4, 5]


def test_verify_device_errors():
    g, V = gen(10), 40
    P = probabilities(g, 6, V, "f32", 1.0)
    u, ul = torch.rand(6, generator=g, device=DEV), torch.rand(2, generator=g, device=DEV)
    out, path, count = (torch.full(s, 5, dtype=torch.int32, device=DEV) for s in ((2, 4), (2, 4), (2,)))
    good = i32([0, 1, 2, 0, 1, 2])
    for qs, tokens, max_q in (([0, 4, 3], good, 4), ([0, 3, 7], good, 4), ([0, 3, 6], good, 2), ([0, 3, 6], i32([0, V, 0, 0, 0, 0]), 4),
                              ([0, 3, 6], i32([0, 0, 0, 0, -1, 0]), 4), ([-1, 3, 6], good, 4)):
        cq.cq_verify(P, tokens, i32(qs), max_q, u, ul, out, path, count, Q=P)
        assert cq.cq_get_device_error() == 5
    cq.cq_verify(P, i32([-5, 1, 2, V + 9, 1, 2]), i32([0, 3, 6]), 4, u, ul, out, path, count, Q=P)   # a first row's token is not read
    assert cq.cq_get_device_error() == 0


def test_verify_offsets_past_32_bits():
    """Rows past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    rows, V = 70000, 32768
    P = torch.zeros(rows, V, dtype=torch.float16, device=DEV)
    counts = [2] * 35000
    P[:, 77] = 0.5
    P[-1, 77], P[-1, 31000] = 0.0, 1.0
    parents = [[-1, 0]] * 35000
    out, path = torch.empty(35000, 2, dtype=torch.int32, device=DEV), torch.empty(35000, 2, dtype=torch.int32, device=DEV)
    count = torch.empty(35000, dtype=torch.int32, device=DEV)
    tokens = torch.full((rows,), 77, dtype=torch.int32, device=DEV)
    cq.cq_verify(P, tokens, starts(counts), 2, torch.full((rows,), 0.25, device=DEV), torch.full((35000,), 0.5, device=DEV), out, path, count)
    assert cq.cq_get_device_error() == 0
    assert (count == 1).all() and (out[:-1] == 77).all() and out[-1].tolist() == [77, 31000]
    assert path[-1].tolist() == [rows - 2, rows - 1]


# ---- the step as it is used -----------------------------------------------------------------------------------------

def test_a_step_on_another_stream_and_in_graphs():
    """Rotate, append, attend a tree, check the drafts, append what stands: eagerly on another stream, then twice out of two captured
    graphs that share the workspace; the same bits."""
    B, Hkv, G, D, V, n = 3, 2, 4, 64, 500, 6
    rng = np.random.default_rng(5)
    held = [40, 100, 0]
    s = Setup(61, [h + 2 * n for h in held], Hkv, D, 32)
    s.write(held, "bf16")
    pools = [t.clone() for t in (s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs)]
    parents = [draftref.tree(rng, n) for _ in range(B)]
    depth = [[0] * n for _ in range(B)]
    for d, p in zip(depth, parents):
        for i in range(1, n):
            d[i] = d[p[i]] + 1
    T = B * n
    r = cq.cq_rope_spec(freqs(D))
    qkv = s.rows(T, Hkv * (G + 2), "bf16", 0.2)
    g = gen(62)
    P, Q = probabilities(g, T, V, "bf16", 2.0), probabilities(g, T, V, "bf16", 2.0)
    tokens = drafted(g, Q, parents, [n] * B, V)
    u, ul = torch.rand(T, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
    mask = torch.from_numpy(draftref.words([x for p in parents for x in draftref.bits_of(p)], 1)).to(DEV)
    pos = i32([h + d for h, ds in zip(held, depth) for d in ds])
    qs, lens = starts([n] * B), i32([h + n for h in held])
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, Hkv * G, Hkv, D, B, n), dtype=torch.uint8, device=DEV)

    def buffers():
        e = lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device=DEV)
        return {"q": e(T, Hkv * G, D, dtype=torch.bfloat16), "o": e(T, Hkv * G, D, dtype=torch.bfloat16), "out": e(B, n), "path": e(B, n),
                "count": e(B), "k": e(B * n, Hkv, D, dtype=torch.bfloat16), "v": e(B * n, Hkv, D, dtype=torch.bfloat16)}

    def step(x):
        q, k, v = qkv[:, :Hkv * G], qkv[:, Hkv * G:Hkv * (G + 1)], qkv[:, Hkv * (G + 1):]
        cq.cq_rope(q, r, pos, x["q"])
        cq.cq_kv8_write_rope(s.cache, k, v, qs, lens, r, pos)
        cq.cq_attn_kv8_tree(x["q"], s.cache, qs, lens, n, mask, x["o"], ws)
        cq.cq_verify(P, tokens, qs, n, u, ul, x["out"], x["path"], x["count"], Q=Q, mask=mask)
        # the rows that stand become their sequences' last tokens (their places are their positions)
        stands = x["path"].flatten() >= 0
        rows = x["path"].flatten().clamp(min=0).long()
        keep = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), (x["count"] + 1).cumsum(0).int()])
        order = torch.argsort(~stands, stable=True)
        x["k"].copy_(k[rows[order]])
        x["v"].copy_(v[rows[order]])
        x["lens"] = i32h + x["count"] + 1
        cq.cq_kv8_write_rope(s.cache, x["k"], x["v"], keep, x["lens"], r)

    i32h = i32(held)

    def reset():
        for t, p in zip((s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs), pools):
            t.copy_(p)

    side = torch.cuda.Stream()
    first = buffers()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(first)
        assert cq.cq_get_device_error() == 0
    torch.cuda.synchronize()
    seen = [t.clone() for t in (s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs)]
    graphs = []
    for _ in range(2):
        x = buffers()
        reset()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(x)
        graphs.append((graph, x))
    for _ in range(2):
        for graph, x in graphs:
            reset()
            for t in x.values():
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for name in ("q", "o", "out", "path", "count"):
                assert torch.equal(x[name], first[name]), name
            for t, w in zip((s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs), seen):
                assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    # and against the reference: keys at the positions of what stands, then the drafted step before them rolled back
    at = 0
    for b in range(B):
        want, rows = draftref.verify(f64(P)[b * n:b * n + n], f64(Q)[b * n:b * n + n], tokens.tolist()[b * n:b * n + n], parents[b],
                                     f64(u)[b * n:b * n + n], f64(ul)[b])
        assert first["out"][b, :len(want)].tolist() == want and first["path"][b, :len(rows)].tolist() == [b * n + i for i in rows]
        kr = draftref.rotate(f64(qkv[:, Hkv * G:Hkv * (G + 1)])[[b * n + i for i in rows]], [held[b] + d for d in range(len(rows))], f64(r.freq), "half")
        s.len[b] = held[b] + len(rows)
        back = f64(s.read("f32", [0 if c != b else held[b] for c in range(B)], [0 if c != b else len(rows) for c in range(B)])[0][:len(rows)])
        blocks = [(s.table[b, (held[b] + i) // 32].item()) for i in range(len(rows))]
        scale = np.stack([f64(s.cache.Ks[p, :, 0]) for p in blocks])[:, :, None]
        assert np.all(np.abs(back - kr) <= scale * (0.5 + 2.0 ** -12))


def test_one_workspace_for_trees_and_chains():
    """The workspace of the largest call serves smaller trees, whichever kernel they go to."""
    s = Setup(71, [200], 2, 64, 32)
    s.write([100], "bf16")
    s.write([40], "bf16")
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(40, 8, 2, 64, 1, 40), dtype=torch.uint8, device=DEV)
    for n in (1, 2, 4, 5, 8, 9, 33, 40):
        bits = trees_of(np.random.default_rng(n), [n])
        q = s.rows(n, 8, "bf16", 0.2)
        o = torch.empty(n, 8, 64, device=DEV)
        mask = torch.from_numpy(draftref.words(bits[0], 2)).to(DEV)
        cq.cq_attn_kv8_tree(q, s.cache, starts([n]), i32(s.len), n, mask, o, ws)
        assert cq.cq_get_device_error() == 0
        want, _, e, _ = draftref.attend(s.ref, 0, f64(q), 0.125, bits[0], "f32")
        assert np.all(np.abs(f64(o) - want) <= e)


@pytest.mark.parametrize("n,group", [(2, 2), (6, 4), (20, 4), (40, 8)])
def test_tree_wait_timeout_reports_status_and_the_next_call_is_right(n, group):
    s = Setup(81, [600], 1, 64, 32)
    s.write([500], "bf16")
    s.write([n], "bf16")
    bits = trees_of(np.random.default_rng(n), [n])
    q, o = s.rows(n, group, "bf16", 0.2), torch.empty(n, group, 64, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(n, group, 1, 64, 1, n), dtype=torch.uint8, device=DEV)
    mask = torch.from_numpy(draftref.words(bits[0], 2)).to(DEV)
    old = cq.cq_get_option(cq.CQ_OPT_WAIT_NS)
    cq.cq_set_option(cq.CQ_OPT_WAIT_NS, 20_000_000)
    try:
        cq.cq_set_option(cq.CQ_OPT_TEST_STALL, 1)
        cq.cq_attn_kv8_tree(q, s.cache, starts([n]), i32(s.len), n, mask, o, ws)
        assert cq.cq_get_device_error() == 8
    finally:
        cq.cq_set_option(cq.CQ_OPT_WAIT_NS, old)
        cq.cq_set_option(cq.CQ_OPT_TEST_STALL, 0)
    cq.cq_attn_kv8_tree(q, s.cache, starts([n]), i32(s.len), n, mask, o, ws)
    assert cq.cq_get_device_error() == 0
    want, _, e, _ = draftref.attend(s.ref, 0, f64(q), 0.125, bits[0], "f32")
    assert np.all(np.abs(f64(o) - want) <= e)


# ---- calls that no list of sizes makes ------------------------------------------------------------------------------

@pytest.mark.parametrize("n,group", [(3, 2), (6, 4), (20, 4), (40, 8)])
def test_rows_behind_the_last_sequence(n, group):
    """Rows past q_start[B] belong to nobody: outputs, lse and the cache's other pages stay as they were."""
    held = [50, 10]
    s = Setup(91, [120, 80], 2, 64, 32)
    s.write(held, "bf16")
    r = cq.cq_rope_spec(freqs(64))
    T, real = 2 * n + 5, 2 * n
    k, v = s.rows(T, 2, "bf16"), s.rows(T, 2, "bf16")
    pools = [t.clone() for t in (s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs)]
    s.len = [h + n for h in held]
    kr = torch.empty(k.shape, device=DEV)
    place = i32([p for h in held for p in range(h, h + n)] + [0] * 5)
    cq.cq_rope(k, r, place, kr)
    cq.cq_kv8_write_rope(s.cache, k, v, starts([n, n]), i32(s.len), r, place)
    for b in range(2):
        s.ref.write(b, f64(kr[b * n:b * n + n]), f64(v[b * n:b * n + n]))
    same(s)
    used = set(s.table.flatten().tolist())
    for t, old in zip((s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs), pools):
        rest = [p for p in range(t.shape[0]) if p not in used]
        assert rest and torch.equal(t[rest].view(torch.uint8), old[rest].view(torch.uint8))
    bits = trees_of(np.random.default_rng(n), [n, n])
    q = s.rows(T, 2 * group, "bf16", 0.2)
    o, l = torch.full((T, 2 * group, 64), 7.0, device=DEV), torch.full((T, 2 * group), 8.0, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, 2 * group, 2, 64, 2, n), dtype=torch.uint8, device=DEV)
    mask = torch.from_numpy(draftref.words([x for b in bits for x in b] + [(1 << n) - 1] * 5, 2)).to(DEV)
    cq.cq_attn_kv8_tree(q, s.cache, starts([n, n]), i32(s.len), n, mask, o, ws, lse=l)
    assert cq.cq_get_device_error() == 0
    assert (o[real:] == 7.0).all() and (l[real:] == 8.0).all()
    for b in range(2):
        want, _, e, _ = draftref.attend(s.ref, b, f64(q[b * n:b * n + n]), 0.125, bits[b], "f32")
        assert np.all(np.abs(f64(o[b * n:b * n + n]) - want) <= e)


def test_mask_and_keys_past_32_bits():
    """Masks and keys whose last rows lie past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n, B, pitch = 7, 300, 1 << 20
    T = n * B
    s = Setup(92, [n + 3] * B, 1, 64, 32)
    s.write([3] * B, "bf16")
    wide = torch.zeros(T * pitch, dtype=torch.float16, device=DEV)
    k = wide.as_strided((T, 1, 64), (pitch, 64, 1))
    k.copy_(s.rows(T, 1, "f16", 0.3))
    v = s.rows(T, 1, "f16", 0.3)
    r = cq.cq_rope_spec(freqs(32))
    rotated(s, k, v, [n] * B, r, "half")
    back = s.read("f32", [0] * (B - 1) + [0], [0] * (B - 1) + [n + 3])[0]
    np.testing.assert_array_equal(f64(back), s.ref.values(0, B - 1))
    del wide, k
    bits = trees_of(np.random.default_rng(2), [n] * B)
    words = torch.zeros(T * pitch, dtype=torch.int32, device=DEV)
    mask = words.as_strided((T, 1), (pitch, 1))
    mask.copy_(torch.from_numpy(draftref.words([x for b in bits for x in b], 1)).to(DEV))
    q, o = s.rows(T, 2, "f16", 0.3), torch.empty(T, 2, 64, device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, 2, 1, 64, B, n), dtype=torch.uint8, device=DEV)
    cq.cq_attn_kv8_tree(q, s.cache, starts([n] * B), i32(s.len), n, mask, o, ws)
    assert cq.cq_get_device_error() == 0
    for b in (0, B // 2, B - 1):
        want, _, e, _ = draftref.attend(s.ref, b, f64(q[b * n:b * n + n]), 0.125, bits[b], "f32")
        assert np.all(np.abs(f64(o[b * n:b * n + n]) - want) <= e)


def test_verify_many_sequences():
    """As many sequences as the call takes, most of them without rows."""
    g, B, V = gen(93), 65536, 24
    counts = [0] * B
    for b in range(0, B, 997):
        counts[b] = 1 + b % 3
    T = sum(counts)
    P = probabilities(g, T, V, "f32", 1.0)
    Q = probabilities(g, T, V, "f32", 1.0)
    parents = [list(range(-1, c - 1)) for c in counts]
    u, ul = torch.rand(T, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
    out, path = torch.empty(B, 3, dtype=torch.int32, device=DEV), torch.empty(B, 3, dtype=torch.int32, device=DEV)
    count = torch.empty(B, dtype=torch.int32, device=DEV)
    tokens = drafted(g, Q, [p for p in parents if p], [c for c in counts if c], V)
    cq.cq_verify(P, tokens, starts(counts), 3, u, ul, out, path, count, Q=Q)
    assert cq.cq_get_device_error() == 0
    out, path, count = out.tolist(), path.tolist(), count.tolist()
    at = 0
    for b, n in enumerate(counts):
        if n == 0:
            assert out[b] == path[b] == [-1] * 3 and count[b] == 0
            continue
        want, rows = draftref.verify(f64(P[at:at + n]), f64(Q[at:at + n]), tokens.tolist()[at:at + n], parents[b], f64(u[at:at + n]), f64(ul)[b])
        assert out[b] == want + [-1] * (3 - len(want)) and path[b] == [at + i for i in rows] + [-1] * (3 - len(rows)) and count[b] == len(rows) - 1
        at += n


def test_calls_on_two_streams_at_once():
    """The same calls with their own buffers on two streams, many times over: the bits of a call alone."""
    rng, n, B = np.random.default_rng(94), 20, 3
    sets = []
    for seed in (94, 95):
        s = Setup(seed, [400] * B, 2, 64, 32)
        s.write([300, 100, 7], "bf16")
        s.write([n] * B, "bf16")
        q = s.rows(n * B, 8, "bf16", 0.2)
        g = gen(seed)
        P = probabilities(g, n * B, 9000, "bf16", 2.0)
        parents = [draftref.tree(rng, n) for _ in range(B)]
        sets.append({"s": s, "q": q, "r": cq.cq_rope_spec(freqs(64)), "pos": torch.arange(n * B, device=DEV).int(), "y": torch.empty_like(q),
                     "mask": torch.from_numpy(draftref.words([x for p in parents for x in draftref.bits_of(p)], 1)).to(DEV),
                     "o": torch.empty(n * B, 8, 64, device=DEV), "P": P, "tokens": drafted(g, P, parents, [n] * B, 9000),
                     "ws": torch.empty(cq.cq_attn_kv8_workspace_bytes(n * B, 8, 2, 64, B, n), dtype=torch.uint8, device=DEV),
                     "u": torch.rand(n * B, generator=g, device=DEV), "ul": torch.rand(B, generator=g, device=DEV), "qs": starts([n] * B), "lens": i32(s.len),
                     "out": torch.empty(B, n, dtype=torch.int32, device=DEV), "path": torch.empty(B, n, dtype=torch.int32, device=DEV),
                     "count": torch.empty(B, dtype=torch.int32, device=DEV)})

    def call(x):
        cq.cq_rope(x["q"], x["r"], x["pos"], x["y"])
        cq.cq_attn_kv8_tree(x["y"], x["s"].cache, x["qs"], x["lens"], n, x["mask"], x["o"], x["ws"])
        cq.cq_verify(x["P"], x["tokens"], x["qs"], n, x["u"], x["ul"], x["out"], x["path"], x["count"], Q=x["P"], mask=x["mask"])

    names = ("y", "o", "out", "path", "count")
    alone = []
    for x in sets:
        call(x)
        alone.append([x[k].clone() for k in names])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for x, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                call(x)
    torch.cuda.synchronize()
    for x, want, stream in zip(sets, alone, streams):
        assert cq.cq_get_device_error(stream) == 0
        for k, w in zip(names, want):
            assert torch.equal(x[k], w), k


@pytest.mark.parametrize("n,group", [(1, 4), (5, 5), (16, 4), (150, 1)])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [False, True])
def test_long_sums_of_trees(n, group, out, D, sign):
    """Sums over 40960 tokens that one SM takes in turn, of one sign (truncation shrinks them all alike) and of both: the
    results' projection on the exact ones.  f32 outputs put back 1.6e-8 a product of a window of 128 (64 channels: 64),
    which loses 0.4e-8 to 4.3e-8: 3.5e-6 at most; 16-bit ones lose up to 6.6e-8 of each of 1024: 7e-5."""
    B, Hkv, L, page = 32, 16, 40960, 1024
    s = Setup(65, [L], Hkv, D, page, spare=0)
    s.len = [L]
    k, v = s.rows(L, Hkv, "bf16", 0.3), s.rows(L, Hkv, "bf16", 0.3)
    v = v.abs() if sign else v
    cq.cq_kv8_write(s.cache, k, v, starts([L]), i32([L]))
    k, v = (x.double().transpose(0, 1) for x in s.read("f32"))
    s.cache = cq.cq_kv8_cache(s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs, s.table.repeat(B, 1))   # all over the same pages
    q = s.rows(B * n, Hkv * group, "f16", 0.3)
    o = torch.empty(B * n, Hkv * group, D, dtype=TORCH[out], device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(B * n, Hkv * group, Hkv, D, B, n), dtype=torch.uint8, device=DEV)
    mask = torch.full((B * n, (n + 31) // 32), -1, dtype=torch.int32, device=DEV)
    cq.cq_attn_kv8_tree(q, s.cache, starts([n] * B), i32([L] * B), n, mask, o, ws)
    assert cq.cq_get_device_error() == 0
    for b in (0, B - 1):
        x = q[b * n:b * n + n].double().view(n, Hkv, group, D).permute(1, 0, 2, 3).reshape(Hkv, n * group, D)
        w = torch.softmax(x @ k.transpose(1, 2) * D ** -0.5, 2)
        ref = (w @ v).view(Hkv, n, group, D).transpose(0, 1).reshape(n, Hkv * group, D)
        err = o[b * n:b * n + n].double() - ref
        along = float((err * ref).sum() / (ref * ref).sum())
        assert abs(along) <= (3.5e-6 if out == "f32" else 7e-5), along


# ---- what is left after several rejected siblings -------------------------------------------------------------------

class Left:
    """max(P - A q, 0) after `fell` rejected children drawn from q, in rational arithmetic."""

    def __init__(self, p, q, fell):
        P, Q = ([int(x) for x in np.ldexp(np.where(r > 0, r, 0.0), 149)] for r in (f64(p), f64(q)))
        a, bits, m = 0, 0, 1                                    # A and the mass in 2^-bits
        for _ in range(fell):
            a += m
            w = [max((x << bits) - a * y, 0) for x, y in zip(P, Q)]
            bits, a, m = bits + 149, a << 149, sum(w)           # entries are whole numbers of 2^-149
        self.sums, self.at = list(itertools.accumulate(w)), [x for x, y in enumerate(w) if y]
        self.whole, self.mass = m, float(Fraction(m, 1 << bits))

    def drawn(self, ul):
        """The token that a number draws, and how far from it the nearest border of another one lies."""
        u = Fraction(float(ul))
        x = bisect.bisect_right(self.sums, u.numerator * self.whole // u.denominator)
        if x >= len(self.sums):
            return self.at[-1], self.mass                       # (nothing after the last one can be drawn)
        below, aim = self.sums[x - 1] if x else 0, u * self.whole
        near = [self.sums[x] - aim] if x < self.at[-1] else [self.whole]
        near += [aim - below] if x > self.at[0] else []
        return x, float(min(near) / self.whole) * self.mass

    def border(self, x):
        return np.float32(float(Fraction(self.sums[x], self.whole)))


def siblings_fall(P, Q, fell, ul):
    """The token that cq_verify draws for a row whose `fell` children all fall (their numbers are NaN)."""
    n = fell + 1
    tokens, u = torch.zeros(n, dtype=torch.int32, device=DEV), torch.full((n,), float("nan"), device=DEV)
    mask = torch.from_numpy(draftref.words(draftref.bits_of([-1] + [0] * fell), 1)).to(DEV)
    out, path, count = (torch.full(s, 777, dtype=torch.int32, device=DEV) for s in ((1, n), (1, n), (1,)))
    cq.cq_verify(P, tokens, i32([0, n]), n, u, torch.tensor([float(ul)], device=DEV), out, path, count, Q=Q, mask=mask)
    assert cq.cq_get_device_error() == 0 and count.item() == 0 and path[0].tolist() == [0] + [-1] * fell
    return out[0, 0].item()


def first_row(row, n, dtype="f32"):
    """[n][V] with this first row, rows on 16 bytes."""
    x = torch.zeros(n, (len(row) + 7) // 8 * 8, dtype=TORCH[dtype], device=DEV)[:, :len(row)]
    x[0] = torch.as_tensor(row)
    return x


@pytest.mark.parametrize("fell", [1, 2, 3, 6])
@pytest.mark.parametrize("V,dtype", [(300, "f32"), (32000, "f32"), (32000, "bf16"), (150001, "f32"), (150001, "f16")])
def test_verify_siblings_next_to_borders(fell, V, dtype):
    """Draws as near to the borders of max(P - A q, 0) as f32 numbers come.  Entries are within 2^-45 of the larger of P and A q and
    sums within 2^-40; A is a sum of up to 6 of them, whose errors do not grow (a larger A leaves less): with rows that sum to 1,
    borders lie within 7 2^-45 + 7 2^-40 < 2^-37 of where they belong."""
    g = gen(V + fell)
    logits = 2.0 * torch.randn(V, generator=g, device=DEV)
    P = first_row(torch.softmax(logits, 0), fell + 1, dtype)
    Q = first_row(torch.softmax(logits + 0.5 * torch.randn(V, generator=g, device=DEV), 0), fell + 1, dtype)
    left, tried = Left(P[0], Q[0], fell), 0
    for x in np.random.default_rng(V + fell).choice(left.at, 12):
        u = left.border(x)
        for ul in (np.nextafter(u, np.float32(0)), u, np.nextafter(u, np.float32(1))):
            want, margin = left.drawn(ul)
            if margin > 2.0 ** -37:
                tried += 1
                assert siblings_fall(P, Q, fell, ul) == want, (x, ul, margin)
    assert tried > 12


@pytest.mark.parametrize("fell", [1, 2, 3, 5])
@pytest.mark.parametrize("V,dtype", [(32000, "f32"), (100000, "bf16")])
def test_verify_siblings_leave_few_tokens(fell, V, dtype):
    """Whatever is left lies in the first tokens, though every other one has a probability: none of those is drawn, and there is
    always a token."""
    g = gen(fell)
    q = torch.softmax(0.5 * torch.randn(V, generator=g, device=DEV), 0)
    p = 0.98 * q
    p[:200] = 4.0 * fell * q[:200]
    P, Q = first_row(p, fell + 1, dtype), first_row(q, fell + 1, dtype)
    left = Left(P[0], Q[0], fell)
    assert 0 < left.mass and left.at[-1] < 200
    for ul in (0.0, 0.3, 0.7, 0.99, 1.0 - 2.0 ** -24, 1.0, 2.0):
        want, margin = left.drawn(np.float32(ul))
        assert margin > 2.0 ** -37
        assert siblings_fall(P, Q, fell, ul) == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_siblings_leave_roundings(dtype):
    """P is A q as the type rounds it, so that what is left are those roundings, 2^-9 or 2^-25 of an entry (bf16, f32) in half of
    them, and no other entry is drawn.  A is 5/4 and a little, of which sums lose 2^-42, and entries are within 2^-45 of
    5/4 q: as Q sums to 1, borders lie within 2^-41 of where they belong."""
    V, fell = 1000, 2
    r = np.random.default_rng(4).integers(1 << 22, 1 << 23, V) * 2 + 1           # 24 bits, odd: 5/4 of it is no f32 number
    if dtype == "bf16":
        r = r >> 16 << 16 | 1 << 16
    q = np.ldexp(r.astype(np.float64), -35)
    rest = 1.0 - q.sum()
    # the last entries make the sum 1, in numbers of the type
    parts = []
    while rest > 0:
        m, e = np.frexp(rest)
        x = np.ldexp(np.floor(np.ldexp(m, 8)), e - 8)
        parts.append(x)
        rest -= x
    q = np.concatenate([q, parts])
    assert q.sum() == 1.0
    Q = first_row(q, fell + 1, dtype)
    assert np.array_equal(f64(Q[0]), q)
    P = first_row(1.25 * q, fell + 1, dtype)
    left = Left(P[0], Q[0], fell)
    some = 0
    for x in np.random.default_rng(5).choice(left.at, 60):
        for part in (0.3, 0.5, 0.7):
            below = left.sums[x - 1] if x else 0
            ul = np.float32(float(Fraction(below + int((left.sums[x] - below) * part), left.whole)))
            want, margin = left.drawn(ul)
            if margin > 2.0 ** -41:
                some += 1
                assert siblings_fall(P, Q, fell, ul) == want
    assert some > 30


def test_verify_tiny_numbers():
    """Products of numbers below f32's normal ones: u q < p as real numbers have it."""
    cases = [(u, q, p) for u in (0.25, 0.5, 0.625, 0.75, 0.9375) for q in range(1, 8) for p in range(8)]
    B, V = len(cases), 8
    P, Q = torch.zeros(2 * B, V), torch.zeros(2 * B, V)
    P[:, 5] = Q[:, 5] = 0.5
    P[0::2, 3] = torch.tensor([np.ldexp(float(p), -149) for _, _, p in cases])
    Q[0::2, 3] = torch.tensor([np.ldexp(float(q), -149) for _, q, _ in cases])
    u = torch.tensor([x for x, _, _ in cases], device=DEV).repeat_interleave(2)
    out, path = (torch.empty(B, 2, dtype=torch.int32, device=DEV) for _ in range(2))
    count = torch.empty(B, dtype=torch.int32, device=DEV)
    cq.cq_verify(P.to(DEV), torch.full((2 * B,), 3, dtype=torch.int32, device=DEV), starts([2] * B), 2, u, torch.full((B,), 0.5, device=DEV),
                 out, path, count, Q=Q.to(DEV))
    assert cq.cq_get_device_error() == 0
    assert count.tolist() == [int(x * q < p) for x, q, p in cases]


# ---- what f32 outputs put back of truncated sums ---------------------------------------------------------------------

def few_tokens_decide(n, group, D, out, L, at, B=32, Hkv=16):
    """(outputs, exact ones) of rows whose weights all lie on the tokens `at`, evenly: their scores are 90 above the others', whose
    weights are below 2^-128."""
    s = Setup(66, [L], Hkv, D, 1024, spare=0)
    s.len = [L]
    k, v = torch.zeros(L, Hkv, D, device=DEV), s.rows(L, Hkv, "f32", 0.3)
    k[at] = 90.0 * D ** -0.5
    cq.cq_kv8_write(s.cache, k, v, starts([L]), i32([L]))
    k, v = (f64(x) for x in s.read("f32"))
    assert np.all(np.abs(k[at] * D ** 0.5 - 90.0) < 1.0) and not np.delete(k, at, 0).any()
    s.cache = cq.cq_kv8_cache(s.cache.Kq, s.cache.Ks, s.cache.Vq, s.cache.Vs, s.table.repeat(B, 1))       # all over the same pages
    q, o = torch.ones(B * n, Hkv * group, D, dtype=torch.bfloat16, device=DEV), torch.empty(B * n, Hkv * group, D, dtype=TORCH[out], device=DEV)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(B * n, Hkv * group, Hkv, D, B, n), dtype=torch.uint8, device=DEV)
    mask = torch.full((B * n, (n + 31) // 32), -1, dtype=torch.int32, device=DEV)
    cq.cq_attn_kv8_tree(q, s.cache, starts([n] * B), i32([L] * B), n, mask, o, ws)
    assert cq.cq_get_device_error() == 0
    return f64(o).reshape(B * n, Hkv, group, D), np.broadcast_to(v[at].mean(0)[None, :, None], (B * n, Hkv, group, D))


@pytest.mark.parametrize("n,group", [(1, 4), (4, 4), (5, 5), (16, 4), (32, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token_decides(n, group, D):
    """A row that gives all weight to one token loses nothing to truncation, wherever in a window the token lies.  What is put back for a
    product of 16 tokens and term, 1.1e-8, is then too much: 16 in each of up to 8 steps, 1.41e-6, and three roundings of
    2^-24 (its factor, and two products).  The others' weights come to 4500 2^-128 of values up to 2^6: less than 2^-109."""
    for L, at in ((40, 0), (1024, 3), (1024, 1023), (1152, 500), (4500, 4200)):
        o, want = few_tokens_decide(n, group, D, "f32", L, [at])
        steps = min(-(-L // 128), 8)
        assert np.all(np.abs(o - want) <= np.abs(want) * (steps * 16 * 1.1e-8 + 3 * 2.0 ** -24) + 2.0 ** -109), (L, at)


@pytest.mark.parametrize("counts,group", [([3, 4], 2), ([4, 3], 4), ([6, 4], 5), ([26, 20], 4), ([32, 25], 8)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_chain_has_the_bits_of_the_causal_call(counts, group, out, D):
    """The same arithmetic with a mask as without, whichever kernel: one item a KV head, so that both have the same shares."""
    held = [300, 9000]
    s = Setup(67, [n + h for n, h in zip(counts, held)], 2, D, 64)
    s.len = [n + h for n, h in zip(counts, held)]
    T, Hq, most = sum(counts), 2 * group, max(counts)
    k, v = s.rows(sum(s.len), 2, "bf16", 0.3), s.rows(sum(s.len), 2, "bf16", 0.3)
    cq.cq_kv8_write(s.cache, k, v, starts(s.len), i32(s.len))
    q = s.rows(T, Hq, "bf16", 0.3)
    ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(T, Hq, 2, D, 2, most), dtype=torch.uint8, device=DEV)
    a, b = (torch.empty(T, Hq, D, dtype=TORCH[out], device=DEV) for _ in range(2))
    la, lb = (torch.empty(T, Hq, device=DEV) for _ in range(2))
    mask = torch.from_numpy(draftref.words([(2 << i) - 1 for n in counts for i in range(n)], (most + 31) // 32)).to(DEV)
    cq.cq_attn_kv8(q, s.cache, starts(counts), i32(s.len), most, a, ws, lse=la)
    cq.cq_attn_kv8_tree(q, s.cache, starts(counts), i32(s.len), most, mask, b, ws, lse=lb)
    assert cq.cq_get_device_error() == 0
    assert torch.equal(a, b) and torch.equal(la, lb)
