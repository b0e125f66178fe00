"""A step of drafting over the 8-bit key/value cache, as measured cases: rotary positions, appending rotated keys,
attention for trees of drafted tokens, and the check of drafted tokens against the target's probabilities.

The cache.  Keys and values are int8 codes in pages, Kq and Vq [pages][Hkv][page][D], with one f32 scale per 32
tokens and head, Ks and Vs [pages][Hkv][page / 32]; table[b][i] names the page that holds tokens i * page .. of
sequence b.  A value is code * scale; the scale is the smallest power of two 2^e (e >= -64) with amax <= 127 * 2^e
over the block's tokens, the code the nearest integer (ties to even).  Tokens that are appended to a block with
tokens in it may raise its scale; the codes that stay are then rounded to the new one.

The operators.  "rope": the first `rot` channels of each head turn in pairs by position * frequency, channels i and
i + rot/2 ("half") or 2i and 2i + 1 ("pairs"), times a factor for scaled contexts.  "append": new tokens' keys are
rotated and written to the cache with their values, then read back (the whole of each sequence, or the block that a
single new token went to).  "tree": softmax attention of a sequence's last rows over all tokens before them and, among
themselves, over those that mask bits name.  "verify": drafted tokens, a chain or a tree, stand or fall by given random
numbers; the token after the last that stands is drawn from what the target's probabilities leave.
"""
import math
import random

import torch

own = False

BLOCK = 32
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
DEV = "cuda"


def listed():
    return [
        # Queries of one token of one user: a launch, latency only.
        {"name": "rope_step", "kind": "rope", "rows": 1, "heads": 32, "d": 128, "rot": 128, "layout": "half", "type": "bf16", "out": "bf16",
         "far": 777, "scaled": False},
        # A prompt's queries behind a context of a million tokens, frequencies scaled for it: memory traffic.
        {"name": "rope_prompt", "kind": "rope", "rows": 16384, "heads": 32, "d": 128, "rot": 128, "layout": "half", "type": "bf16", "out": "bf16",
         "far": 1000000, "scaled": True},
        # Half of each head, neighbouring channels, out of the f32 rows that a projection left.
        {"name": "rope_partial", "kind": "rope", "rows": 3001, "heads": 24, "d": 96, "rot": 48, "layout": "pairs", "type": "f32", "out": "bf16",
         "far": 20000, "scaled": False},
        # A decode step of a full batch: one token each, ragged lengths, most in a partly filled block.
        {"name": "append_step", "kind": "append", "batch": 96, "hkv": 8, "d": 128, "rot": 128, "layout": "half", "page": 32, "base_min": 17,
         "base_max": 4000, "new_min": 1, "new_max": 1, "type": "bf16", "out": "bf16", "back": "block", "given": True, "mix": 2},
        # Long prompts of ragged lengths: memory traffic.
        {"name": "append_prompts", "kind": "append", "batch": 4, "hkv": 8, "d": 128, "rot": 128, "layout": "half", "page": 128, "base_min": 0,
         "base_max": 100, "new_min": 20001, "new_max": 32768, "type": "bf16", "out": "bf16", "back": "all", "given": False, "mix": 3},
        # One user's four drafted rows over a short context: latency.
        {"name": "tree_one", "kind": "tree", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "page": 64, "base_min": 776, "base_max": 776, "new_min": 4,
         "new_max": 4, "type": "bf16", "out": "bf16", "lse": False, "mix": 5},
        # Small trees of a batch, a group of five heads.
        {"name": "tree_batch", "kind": "tree", "batch": 24, "hq": 40, "hkv": 8, "d": 128, "page": 64, "base_min": 300, "base_max": 9000, "new_min": 2,
         "new_max": 6, "type": "bf16", "out": "bf16", "lse": False, "mix": 6},
        # Trees of 26 rows over contexts of mixed lengths.
        {"name": "tree_wide", "kind": "tree", "batch": 32, "hq": 32, "hkv": 8, "d": 128, "page": 64, "base_min": 1000, "base_max": 16000, "new_min": 26,
         "new_max": 26, "type": "f16", "out": "f16", "lse": True, "mix": 7},
        # Large trees over two very long contexts, wide groups: many rows, work split over the tokens.
        {"name": "tree_long", "kind": "tree", "batch": 2, "hq": 32, "hkv": 4, "d": 128, "page": 128, "base_min": 70001, "base_max": 100001, "new_min": 64,
         "new_max": 64, "type": "bf16", "out": "f32", "lse": False, "mix": 8},
        # One user's chain of five drawn tokens, a small vocabulary: latency.
        {"name": "verify_one", "kind": "verify", "batch": 1, "new_min": 6, "new_max": 6, "vocab": 32000, "type": "f32", "drawn": True, "tree": False, "mix": 9},
        # Chains of a batch over a large odd vocabulary: one row of the target and one of the draft model per sequence.
        {"name": "verify_batch", "kind": "verify", "batch": 64, "new_min": 2, "new_max": 6, "vocab": 152001, "type": "f32", "drawn": True, "tree": False,
         "mix": 10},
        # Trees of chosen (not drawn) tokens in 16-bit probabilities.
        {"name": "verify_tree", "kind": "verify", "batch": 16, "new_min": 26, "new_max": 26, "vocab": 131072, "type": "bf16", "drawn": False, "tree": True,
         "mix": 11},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["rope", "append", "tree", "tree", "verify", "verify"])
    if kind == "rope":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        rows, heads = log_int(1, 20000), rng.choice([1, 3, 8, 24, 32, 40, 64])
        while rows * heads * d > 16384 * 32 * 128:
            rows = log_int(1, 20000)
        return {"kind": kind, "rows": rows, "heads": heads, "d": d, "rot": 16 * rng.randrange(1, d // 16 + 1), "layout": rng.choice(["half", "pairs"]),
                "type": rng.choice(["f16", "bf16", "f32"]), "out": rng.choice(["f16", "bf16", "f32"]), "far": log_int(rows, 2000000),
                "scaled": rng.random() < 0.5}
    common = {"kind": kind, "page": rng.choice([32, 64, 96, 128, 256]), "type": rng.choice(["f16", "bf16"]), "mix": rng.randrange(1 << 30)}
    if kind == "append":
        d, step = rng.choice([64, 128]), rng.random() < 0.4
        batch = log_int(1, 128) if step else log_int(1, 12)
        base = sorted([log_int(1, 6000), log_int(1, 6000)]) if step else [0, log_int(1, 300)]
        new = [1, 1] if step else sorted([log_int(1, 8000), log_int(1, 8000)])
        if rng.random() < 0.3:
            common["type"] = "f32"
        return {**common, "batch": batch, "hkv": rng.choice([1, 2, 3, 4, 8, 16]), "d": d, "rot": 16 * rng.randrange(1, d // 16 + 1),
                "layout": rng.choice(["half", "pairs"]), "base_min": base[0], "base_max": base[1], "new_min": new[0], "new_max": new[1],
                "out": rng.choice(["f16", "bf16"]), "back": "block" if step else "all", "given": rng.random() < 0.5}
    if kind == "tree":
        hkv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        while hkv * group > 64:
            group = rng.choice([1, 2, 3, 4])
        batch = log_int(1, 48)
        top = max(64, min(60000, 200000 // batch))
        base, new = sorted([log_int(1, top), log_int(1, top)]), sorted([log_int(1, 80), log_int(1, 80)])
        case = {**common, "batch": batch, "hq": hkv * group, "hkv": hkv, "d": rng.choice([64, 128]), "base_min": base[0] - 1, "base_max": base[1],
                "new_min": new[0], "new_max": new[1], "out": rng.choice([common["type"], "f32"]), "lse": rng.random() < 0.3}
        return case if work(case)["flops"] <= 4e11 else draw(rng)
    tree, drawn = rng.random() < 0.5, rng.random() < 0.6
    vocab = log_int(100, 150000 if not (tree and drawn) else 40000)
    new = sorted([log_int(1, 40 if tree else 16), log_int(2, 40 if tree else 16)])
    if tree and drawn:
        new = [min(n, 12) for n in new]
    batch = log_int(1, 64)
    while batch * new[1] * vocab > 60000000:
        batch = log_int(1, 64)
    return {"kind": kind, "batch": batch, "new_min": new[0], "new_max": new[1], "vocab": vocab, "type": rng.choice(["f32", "f32", "bf16", "f16"]),
            "drawn": drawn, "tree": tree, "mix": common["mix"]}


def lengths(case):
    """(tokens held before, new tokens) of each sequence: spread over the case's ranges, both ends among them."""
    rng = random.Random(case["mix"])
    n = case["batch"]
    out = []
    for lo, hi in ((case.get("base_min", 0), case.get("base_max", 0)), (case["new_min"], case["new_max"])):
        v = [lo + (hi - lo) * i // max(n - 1, 1) for i in range(n)]
        v = [x if i in (0, n - 1) else max(lo, min(hi, x - rng.randrange(0, 1 + (hi - lo) // n))) for i, x in enumerate(v)]
        rng.shuffle(v)
        out.append(v)
    return out


def trees(case, new):
    """The parent of each row but the first, per sequence: near ones more often, so that there are chains and siblings."""
    rng = random.Random(case["mix"] + 1)
    chain = case["kind"] == "verify" and not case["tree"]
    return [[-1] + [i - 1 if chain or rng.random() < 0.4 else rng.randrange(max(0, i - 8), i) for i in range(1, n)] for n in new]


def ancestors(parents):
    """Each row's ancestors and itself, as bits."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": n * case["d"] * (SIZE[case["type"]] + SIZE[case["out"]]) + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    base, new = lengths(case)
    if kind == "verify":
        # what is read of the probabilities: one row each (of the draft's as well, mostly), for the token after the last that stands
        per = case["vocab"] * SIZE[case["type"]] * (2 if case["drawn"] else 1)
        return {"bytes": case["batch"] * per + 20 * sum(new), "flops": case["batch"] * case["vocab"] * (3 if case["drawn"] else 1)}
    hkv, d = case["hkv"], case["d"]
    per_key = 2 * hkv * (d + 4 / BLOCK)
    rows = sum(new)
    if kind == "append":
        back = sum((b + n - 1) % BLOCK + 1 if case["back"] == "block" else b + n for b, n in zip(base, new))
        moved = 2 * hkv * d * (rows * SIZE[case["type"]] + back * SIZE[case["out"]]) + per_key * (rows + back)
        return {"bytes": int(moved), "flops": 4 * hkv * d * (rows + back) + 3 * hkv * case["rot"] * rows}
    moved = rows * case["hq"] * (d * (SIZE[case["type"]] + SIZE[case["out"]]) + (4 if case["lse"] else 0))
    moved += per_key * sum(b + n for b, n in zip(base, new)) + rows * (max(new) + 31) // 32 * 4
    pairs = sum(b * n + sum(bin(m).count("1") for m in ancestors(p)) for b, n, p in zip(base, new, trees(case, new)))
    return {"bytes": int(moved), "flops": 4 * d * case["hq"] * pairs}


# ---- what a program has in hand before the call ---------------------------------------------------------------------

def exponent_scale(amax):
    """2^e, e the smallest integer >= -64 with amax <= 127 * 2^e (f32 bit arithmetic)."""
    mant, ex = torch.frexp(amax)                                   # amax = mant * 2^ex, mant in [0.5, 1)
    e = torch.where(mant > 127.0 / 128.0, ex - 6, ex - 7)
    e = torch.where(amax == 0, torch.full_like(e, -64), e).clamp(min=-64)
    return ((e + 127).int() << 23).view(torch.float32)


def rows_of(gen, n, heads, d, values):
    """Keys or values as a model makes them: some channels of the keys are large, the tokens' size drifts."""
    x = torch.randn(n, heads, d, generator=gen, device=DEV)
    if values:
        return x * torch.exp(0.4 * torch.randn(n, 1, 1, generator=gen, device=DEV))
    gain = torch.ones(heads, d, device=DEV)
    gain[:, 3::29] = 5.0
    return x * gain


def filled(gen, case, held, table, pages):
    """A cache that holds `held` tokens of each sequence; what no token was written to is left as found."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    pools = []
    for values in (False, True):
        codes = torch.randint(-127, 128, (pages, hkv, page // BLOCK, BLOCK, d), generator=gen, device=DEV, dtype=torch.int8)
        scales = torch.full((pages, hkv, page // BLOCK), float("nan"), device=DEV)
        for b, n in enumerate(held):
            step = 65536 // page * page
            for at in range(0, n, step):
                m = min(step, n - at)
                blocks = (m + BLOCK - 1) // BLOCK
                x = torch.zeros(blocks * BLOCK, hkv, d, device=DEV)
                x[:m] = rows_of(gen, m, hkv, d, values)
                x = x.view(blocks, BLOCK, hkv, d).permute(0, 2, 1, 3)
                s = exponent_scale(x.abs().amax((2, 3)))
                q = torch.round(x / s[:, :, None, None]).to(torch.int8)
                where = torch.arange(blocks, device=DEV) + at // BLOCK
                p, j = table[b].long()[where // (page // BLOCK)], where % (page // BLOCK)
                if m % BLOCK:
                    q[-1, :, m % BLOCK:] = codes[p[-1], :, j[-1], m % BLOCK:]
                codes[p, :, j] = q
                scales[p, :, j] = s
        pools += [codes.view(pages, hkv, page, d), scales]
    return pools


def starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def frequencies(rot, scaled):
    """(radians per position of each pair, factor on the rotated channels): plain ones of base 10000, or those scaled by 16
    behind a trained context of 8192, the slow ones wholly, the fast ones not at all, those between by a ramp."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if not scaled:
        return f.float().to(DEV), 1.0
    turn = [rot * math.log(8192 / (2 * math.pi * beta)) / (2 * math.log(10000.0)) for beta in (32, 1)]
    lo, hi = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), rot - 1)
    ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (f / 16 * ramp + f * (1 - ramp)).float().to(DEV), 0.1 * math.log(16) + 1


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    st = {"case": case}
    kind = case["kind"]
    if own:
        import block_quantized_weight_02_gb300 as cq
        st["cq"] = cq
    if kind in ("rope", "append"):
        st["freq"], st["mag"] = frequencies(case["rot"], case.get("scaled", False))
        if own:
            st["rope"] = cq.cq_rope_spec(st["freq"], cq.CQ_ROPE_HALF if case["layout"] == "half" else cq.CQ_ROPE_PAIRS, st["mag"])
    if kind == "rope":
        st["x"] = torch.randn(case["rows"], case["heads"], case["d"], generator=gen, device=DEV).to(TYPES[case["type"]])
        first = case["far"] - int(torch.randint(0, max(1, case["far"] - case["rows"] + 1), (1,), generator=gen, device=DEV))
        st["pos"] = torch.arange(first - case["rows"], first, dtype=torch.int32, device=DEV)
        st["y"] = torch.empty(st["x"].shape, dtype=TYPES[case["out"]], device=DEV)
        return st
    base, new = lengths(case)
    st["new"], st["q_start"] = new, ints(starts(new))
    rows = sum(new)
    if kind == "verify":
        return prepare_verify(st, gen, new)
    total = [b + n for b, n in zip(base, new)]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    per = [(t + page - 1) // page for t in total]
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).int()
    table = torch.full((case["batch"], max(per) + 1), -1, dtype=torch.int32, device=DEV)   # unused entries name no page
    at = starts(per)
    for b, n in enumerate(per):
        table[b, :n] = order[at[b]:at[b] + n]
    kq, ks, vq, vs = filled(gen, case, base if kind == "append" else total, table, pages)
    st.update(base=base, total=total, kq=kq, ks=ks, vq=vq, vs=vs, table=table, lens=ints(total))
    if own:
        st["cache"] = cq.cq_kv8_cache(kq, ks, vq, vs, table)
    if kind == "append":
        dt, odt = TYPES[case["type"]], TYPES[case["out"]]
        st["k"], st["v"] = rows_of(gen, rows, hkv, d, False).to(dt), rows_of(gen, rows, hkv, d, True).to(dt)
        place = torch.cat([torch.arange(b, t, device=DEV) for b, t in zip(base, total)]).int()
        # given positions: every sequence behind text of its own that the cache does not hold
        ahead = torch.randint(0, 100000, (case["batch"],), generator=gen, device=DEV).int()
        st["pos"] = place + ahead.repeat_interleave(ints(new)) if case["given"] else None
        first = [(t - 1) // BLOCK * BLOCK if case["back"] == "block" else 0 for t in total]
        back = [t - f for t, f in zip(total, first)]
        st.update(first_host=first, back=back, first=ints(first), out_start=ints(starts(back)))
        st["k_out"], st["v_out"] = (torch.empty(sum(back), hkv, d, dtype=odt, device=DEV) for _ in range(2))
        plan_append(st, place)
        return st
    st["q"] = torch.randn(rows, case["hq"], d, generator=gen, device=DEV).to(TYPES[case["type"]])
    st["o"] = torch.empty(rows, case["hq"], d, dtype=TYPES[case["out"]], device=DEV)
    st["lse"] = torch.empty(rows, case["hq"], dtype=torch.float32, device=DEV) if case["lse"] else None
    st["mask"] = masks(trees(case, new), max(new))
    if own:
        size = cq.cq_attn_kv8_workspace_bytes(rows, case["hq"], hkv, d, case["batch"], max(new))
        st["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    return st


def masks(parents, most):
    """The rows' ancestors as 32-bit words [rows][words]."""
    words = (most + 31) // 32
    bits = [m for p in parents for m in ancestors(p)]
    w = [[(m >> 32 * i & 0xFFFFFFFF) - (m >> 32 * i + 31 & 1) * (1 << 32) for i in range(words)] for m in bits]
    return torch.tensor(w, dtype=torch.int32, device=DEV)


def plan_append(st, place):
    """Where each new token goes, for the plain form: its block, its row there, the blocks that are touched, and the rows that
    are read back."""
    page, table = st["case"]["page"], st["table"].long()
    tok, touched, kept, out, n_blocks = [], [], [], [], 0
    for b, (base, n, first, back) in enumerate(zip(st["base"], st["new"], st["first_host"], st["back"])):
        p = torch.arange(base, base + n, device=DEV)
        blk = torch.arange(base // BLOCK, (base + n - 1) // BLOCK + 1, device=DEV)
        tok.append(torch.stack([table[b][p // page], p % page // BLOCK, p % BLOCK, p // BLOCK - base // BLOCK + n_blocks]))
        touched.append(torch.stack([table[b][blk * BLOCK // page], blk * BLOCK % page // BLOCK], 1))
        kept.append((base - blk * BLOCK).clamp(0, BLOCK))
        n_blocks += blk.shape[0]
        r = torch.arange(first, first + back, device=DEV)
        out.append(torch.stack([table[b][r // page], r % page // BLOCK, r % BLOCK]))
    st["place"] = place
    st["tok"], st["touched"], st["kept"], st["out"] = torch.cat(tok, 1), torch.cat(touched), torch.cat(kept), torch.cat(out, 1)
    st["part"] = st["kept"].nonzero()[:, 0]


def prepare_verify(st, gen, new):
    case = st["case"]
    rows, vocab, dt = sum(new), case["vocab"], TYPES[case["type"]]
    pitch = (vocab + 7) // 8 * 8
    logits = 2.5 * torch.randn(rows, vocab, generator=gen, device=DEV)
    st["p"] = torch.zeros(rows, pitch, dtype=dt, device=DEV)[:, :vocab]
    st["p"].copy_(torch.softmax(logits, 1))
    q = torch.softmax(logits + 0.6 * torch.randn(rows, vocab, generator=gen, device=DEV), 1).to(dt)
    st["q"] = None
    if case["drawn"]:
        st["q"] = torch.zeros(rows, pitch, dtype=dt, device=DEV)[:, :vocab]
        st["q"].copy_(q)
    parents = trees(case, new)
    at = starts(new)
    up = torch.tensor([max(p, 0) + at[b] for b, ps in enumerate(parents) for p in ps], device=DEV)
    # drafted tokens: drawn from the draft's probabilities at their parent
    noise = torch.rand(rows, vocab, generator=gen, device=DEV)
    st["tokens"] = (q[up].float() / -torch.log(noise.clamp(min=1e-30))).argmax(1).int()
    st["mask"] = masks(parents, max(new)) if case["tree"] else None
    st["u"], st["u_last"] = torch.rand(rows, generator=gen, device=DEV), torch.rand(case["batch"], generator=gen, device=DEV)
    st["out"], st["path"] = (torch.empty(case["batch"], max(new), dtype=torch.int32, device=DEV) for _ in range(2))
    st["count"] = torch.empty(case["batch"], dtype=torch.int32, device=DEV)
    # for the plain form: [sequence][place] row numbers, parents' places (none: -2) and whether there is a row
    n = torch.tensor(new, device=DEV)[:, None]
    place = torch.arange(max(new), device=DEV)[None]
    st["there"] = place < n
    st["row"] = (torch.tensor(at[:-1], device=DEV)[:, None] + place).clamp(max=rows - 1)
    st["parent"] = torch.tensor([p + [-2] * (max(new) - len(p)) for p in parents], device=DEV)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    c, kind = st["case"], st["case"]["kind"]
    if own:
        cq = st["cq"]
        if kind == "rope":
            cq.cq_rope(st["x"], st["rope"], st["pos"], st["y"])
            return [st["y"]]
        if kind == "append":
            cq.cq_kv8_write_rope(st["cache"], st["k"], st["v"], st["q_start"], st["lens"], st["rope"], st["pos"])
            cq.cq_kv8_read(st["cache"], st["first"], st["out_start"], st["k_out"], st["v_out"])
            return [st["k_out"], st["v_out"]]
        if kind == "tree":
            cq.cq_attn_kv8_tree(st["q"], st["cache"], st["q_start"], st["lens"], max(st["new"]), st["mask"], st["o"], st["ws"],
                                scale=1.0 / math.sqrt(c["d"]), lse=st["lse"])
            return [st["o"], st["lse"]] if c["lse"] else [st["o"]]
        cq.cq_verify(st["p"], st["tokens"], st["q_start"], max(st["new"]), st["u"], st["u_last"], st["out"], st["path"], st["count"],
                     Q=st["q"], mask=st["mask"])
        return [st["out"], st["path"], st["count"]]
    if kind == "rope":
        return [turned(st["x"], st["pos"], st).to(TYPES[c["out"]])]
    if kind == "append":
        k = turned(st["k"], st["pos"] if c["given"] else st["place"], st)
        return [plain_append(st, k, st["kq"], st["ks"]), plain_append(st, st["v"].float(), st["vq"], st["vs"])]
    return plain_tree(st) if kind == "tree" else plain_verify(st)


def turned(x, pos, st):
    """The rows with their first rot channels rotated, in 32 bits; the angles in 64."""
    rot, half = st["case"]["rot"], st["case"]["layout"] == "half"
    angle = pos.double()[:, None] * st["freq"].double()
    cos, sin = (st["mag"] * torch.cos(angle)).float()[:, None], (st["mag"] * torch.sin(angle)).float()[:, None]
    y = x.to(torch.float32, copy=True)
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if half else (y[..., 0:rot:2], y[..., 1:rot:2])
    p, q = a * cos - b * sin, b * cos + a * sin
    a.copy_(p)
    b.copy_(q)
    return y


def plain_append(st, x, codes, scales):
    case = st["case"]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    c5 = codes.view(-1, hkv, page // BLOCK, BLOCK, d)
    pg, blk, row, slot = st["tok"]
    tp, tb = st["touched"][:, 0], st["touched"][:, 1]
    kept, part = st["kept"], st["part"]
    amax = torch.zeros(tp.shape[0], hkv, device=DEV).index_reduce_(0, slot, x.abs().amax(2), "amax")
    s0 = scales[tp, :, tb]
    s1 = exponent_scale(amax)
    s1 = torch.where(kept[:, None] > 0, torch.maximum(s0, s1), s1)
    if part.numel():
        old = c5[tp[part], :, tb[part]]
        moved = torch.round(old.float() * (s0 / s1)[part][:, :, None, None]).to(torch.int8)
        stays = torch.arange(BLOCK, device=DEV)[None, None, :, None] < kept[part][:, None, None, None]
        c5[tp[part], :, tb[part]] = torch.where(stays, moved, old)
    scales[tp, :, tb] = s1
    c5[pg, :, blk, row] = torch.round(x / s1[slot][:, :, None]).to(torch.int8)
    op, ob, orow = st["out"]
    return (c5[op, :, ob, orow].float() * scales[op, :, ob][:, :, None]).to(TYPES[case["out"]])


def plain_tree(st):
    """All sequences at once, padded to the longest."""
    case = st["case"]
    hq, hkv, d, page, batch = case["hq"], case["hkv"], case["d"], case["page"], case["batch"]
    group, most, long = hq // hkv, max(st["new"]), max(st["total"])
    lens, at, end = st["lens"].long()[:, None], st["q_start"].long()[:-1, None], st["q_start"].long()[1:, None]
    tok = torch.arange(long, device=DEV)[None]                                                       # [1][tokens]
    pg = st["table"].long()[:, (tok[0] // page)].clamp(min=0)                                        # [batch][tokens]
    place = (tok % page).expand(batch, long)
    hold = (tok < lens)[:, :, None, None]
    k, v = (torch.where(hold, codes[pg, :, place].float() * scales[pg, :, place // BLOCK][..., None], 0.0).permute(0, 2, 1, 3)
            for codes, scales in ((st["kq"], st["ks"]), (st["vq"], st["vs"])))                       # [batch][hkv][tokens][d]
    row = at + torch.arange(most, device=DEV)[None]                                                  # [batch][most]
    there = row < end
    row = torch.where(there, row, 0)
    q = st["q"].float()[row].view(batch, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, most * group, d)
    s = torch.matmul(q, k.transpose(2, 3)).view(batch, hkv, most, group, long) * (1.0 / math.sqrt(d))
    # what a row sees: all before the drafted tokens, and those of its mask among them
    j = tok - (lens - (end - at))                                                                    # [batch][tokens]
    word = st["mask"][row].gather(2, (j.clamp(min=0) // 32).clamp(max=st["mask"].shape[1] - 1)[:, None].expand(batch, most, long))
    sees = (j < 0)[:, None] | ((word >> (j % 32).int()[:, None] & 1) != 0)
    sees = (sees & (tok < lens)[:, None])[:, None, :, None]
    s.masked_fill_(~sees, float("-inf"))
    top = s.amax(4, keepdim=True)
    s = torch.exp(s - top)
    z = s.sum(4, keepdim=True)
    o = torch.matmul(s.view(batch, hkv, most * group, long), v).view(batch, hkv, most, group, d) / z
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, most, hq, d)[there].to(TYPES[case["out"]])
    lse = (top + torch.log(z))[..., 0].permute(0, 2, 1, 3).reshape(batch, most, hq)[there]
    return [o, lse] if case["lse"] else [o]


def plain_verify(st):
    """In 64 bits: whole numbers come out, and a draw may lie next to a border."""
    p, q, tokens = st["p"], st["q"], st["tokens"].long()
    row, there = st["row"], st["there"]
    batch, most = row.shape
    every = torch.arange(batch, device=DEV)
    x, u = tokens[row], st["u"][row].double()
    up = row.gather(1, st["parent"].clamp(min=0))
    px = p[up, x].double()
    qx = q[up, x].double() if q is not None else None
    if st["mask"] is None:
        stands = (u * qx < px if q is not None else u < px) & there
        stands[:, 0] = True
        stands = stands.long().cumprod(1).bool()
        last = stands.sum(1) - 1
        ends = last == there.sum(1) - 1
        at = row[every, last]
        rest = p[at].double()
        if q is not None:
            rest = torch.where(ends[:, None], rest, (rest - q[at].double()).clamp(min=0))
        else:
            fell = row[every, (last + 1).clamp(max=most - 1)]
            rest.scatter_(1, tokens[fell][:, None], torch.where(ends[:, None], rest.gather(1, tokens[fell][:, None]), 0.0))
    else:
        # a walk: one step for each place, as each depends on the ones before (children come after their parents)
        last = torch.zeros(batch, dtype=torch.long, device=DEV)
        stands = torch.zeros(batch, most, dtype=torch.bool, device=DEV)
        stands[:, 0] = True
        fell = torch.zeros_like(stands)                                  # rejected children of the last that stands
        mass, less = torch.ones(batch, device=DEV).double(), torch.zeros(batch, device=DEV).double()
        for j in range(1, most):
            child = (st["parent"][:, j] == last) & there[:, j]
            if q is not None:
                ok = u[:, j] * qx[:, j] * mass < (px[:, j] - less * qx[:, j]).clamp(min=0)
                no = child & ~ok
                less = torch.where(no, less + mass, less)
                at = row[every, last]
                mass = torch.where(no, (p[at].double() - less[:, None] * q[at].double()).clamp(min=0).sum(1), mass)
            else:
                again = ((x == x[:, j:j + 1]) & fell).any(1)
                w = torch.where(again, 0.0, px[:, j])
                ok = u[:, j] * mass < w
                no = child & ~ok
                mass = torch.where(no, mass - w, mass)
            yes = child & ok
            fell[:, j] = no
            fell &= ~yes[:, None]
            stands[:, j] = yes
            last = torch.where(yes, j, last)
            mass, less = torch.where(yes, 1.0, mass), torch.where(yes, 0.0, less)
        at = row[every, last]
        rest = p[at].double()
        if q is not None:
            rest = (rest - less[:, None] * q[at].double()).clamp(min=0)
        else:
            gone = torch.zeros_like(rest).scatter_add_(1, x, fell.double())
            rest = torch.where(gone > 0, 0.0, rest)
    rest = torch.where((rest.sum(1) > 0)[:, None], rest, p[at].double())
    cum = rest.cumsum(1)
    new = torch.searchsorted(cum, st["u_last"].double()[:, None] * cum[:, -1:], right=True)[:, 0]
    count = stands.sum(1) - 1
    # the tokens and rows that stand, closed up, then the drawn token
    order = torch.argsort(~stands, dim=1, stable=True)
    keep = torch.arange(most, device=DEV)[None]
    path = torch.where(keep <= count[:, None], row.gather(1, order), -1)
    out = torch.where(keep < count[:, None], x.gather(1, order.roll(-1, 1)), -1)
    out[every, count] = new
    return [out.int(), path.int(), count.int()]


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def exact_turned(st, x, pos):
    rot, half = st["case"]["rot"], st["case"]["layout"] == "half"
    y = x.double()
    z = y.clone()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if half else (2 * i, 2 * i + 1)
        t = pos.double() * float(st["freq"][i])
        turn = st["mag"] * torch.complex(torch.cos(t), torch.sin(t))[:, None]
        w = torch.complex(y[..., a], y[..., b]) * turn
        z[..., a], z[..., b] = w.real, w.imag
    return z


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rope":
        return [exact_turned(st, st["x"], st["pos"])]
    if case["kind"] == "verify":
        return exact_verify(st)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    table = st["table"].cpu().tolist()

    def tokens(codes, scales, b, h, n):
        """The first n tokens of a head, f64 codes and scales of their blocks."""
        ids = torch.tensor(table[b][:(n + page - 1) // page], device=DEV, dtype=torch.long)
        c = codes[ids, h].reshape(-1, d)[:n].double()
        s = scales[ids, h].reshape(-1)[:(n + BLOCK - 1) // BLOCK].double()
        return c, s

    if case["kind"] == "append":
        def least(a):
            e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 127.0))
            e = torch.where(a <= 127.0 * torch.exp2(e - 1), e - 1, e)
            e = torch.where(a > 127.0 * torch.exp2(e), e + 1, e)
            return torch.exp2(e.clamp(min=-64))

        pos = st["pos"]
        if pos is None:
            pos = torch.tensor([p for b, n in zip(st["base"], st["new"]) for p in range(b, b + n)], device=DEV)
        both = []
        for x, codes, scales in ((exact_turned(st, st["k"], pos), st["kq"], st["ks"]), (st["v"].double(), st["vq"], st["vs"])):
            parts, at = [], 0
            for b, (base, n, first) in enumerate(zip(st["base"], st["new"], st["first_host"])):
                heads = []
                for h in range(hkv):
                    c, s0 = tokens(codes, scales, b, h, base) if base else (torch.zeros(0, d, device=DEV).double(), torch.zeros(0, device=DEV).double())
                    total, edge = base + n, base // BLOCK * BLOCK
                    xs = x[at:at + n, h]
                    grown = torch.zeros((total - edge + BLOCK - 1) // BLOCK * BLOCK, device=DEV).double()
                    grown[base - edge:total - edge] = xs.abs().amax(1)
                    s1 = least(grown.view(-1, BLOCK).amax(1))
                    if base % BLOCK:
                        s1[0] = torch.maximum(s1[0], s0[-1])
                        tail = torch.round(c[edge:] * s0[-1] / s1[0]) * s1[0]
                    else:
                        tail = c[edge:]
                    whole = (c[:edge].view(-1, BLOCK, d) * s0[:edge // BLOCK, None, None]).view(-1, d)
                    to = s1[torch.arange(base - edge, total - edge, device=DEV) // BLOCK][:, None]
                    heads.append(torch.cat([whole, tail, torch.round(xs / to) * to])[first:])
                parts.append(torch.stack(heads, 1))
                at += n
            both.append(torch.cat(parts))
        return both

    group = case["hq"] // hkv
    o = torch.zeros(sum(st["new"]), case["hq"], d, device=DEV, dtype=torch.float64)
    z = torch.zeros(sum(st["new"]), case["hq"], device=DEV, dtype=torch.float64)
    at = 0
    for b, (base, n, parents) in enumerate(zip(st["base"], st["new"], trees(case, st["new"]))):
        hide = torch.zeros(n, base + n, dtype=torch.bool)
        for i in range(n):
            hide[i, base:] = True
            j = i
            while j >= 0:
                hide[i, base + j] = False
                j = parents[j]
        hide = hide.to(DEV)
        for h in range(hkv):
            (kc, ksc), (vc, vsc) = tokens(st["kq"], st["ks"], b, h, base + n), tokens(st["vq"], st["vs"], b, h, base + n)
            k = kc * ksc.repeat_interleave(BLOCK)[:base + n, None]
            v = vc * vsc.repeat_interleave(BLOCK)[:base + n, None]
            x = st["q"][at:at + n, h * group:(h + 1) * group].double()
            s = torch.einsum("mgd,kd->mgk", x, k) / math.sqrt(d)
            s = s.masked_fill(hide[:, None], float("-inf"))
            l = torch.logsumexp(s, 2)
            o[at:at + n, h * group:(h + 1) * group] = torch.einsum("mgk,kd->mgd", torch.exp(s - l[..., None]), v)
            z[at:at + n, h * group:(h + 1) * group] = l
        at += n
    return [o, z] if case["lse"] else [o]


def exact_verify(st):
    case, at = st["case"], starts(st["new"])
    most = max(st["new"])
    tokens, u, u_last = st["tokens"].cpu().tolist(), st["u"].double().cpu().tolist(), st["u_last"].double().cpu().tolist()
    outs, paths, counts = [], [], []
    for b, parents in enumerate(trees(case, st["new"])):
        cur, out, path = 0, [], [at[b]]
        while True:
            p = st["p"][at[b] + cur].double().cpu()
            q = st["q"][at[b] + cur].double().cpu() if case["drawn"] else None
            # the target's probabilities less what the rejected children have had, normalised again after each
            left, go = p / 1.0, None
            for j in range(cur + 1, len(parents)):
                if parents[j] != cur:
                    continue
                x, r = tokens[at[b] + j], u[at[b] + j]
                if r * (float(q[x]) if case["drawn"] else 1.0) < float(left[x]):
                    go = j
                    break
                if case["drawn"]:
                    left = (left - q).clamp(min=0)
                    left = left / left.sum()
                else:
                    had = float(left[x])
                    left[x] = 0.0
                    left = left / (1.0 - had)
            if go is None:
                break
            out.append(tokens[at[b] + go])
            path.append(at[b] + go)
            cur = go
        cum = torch.cumsum(left if float(left.sum()) > 0 else p, 0)
        out.append(int((cum <= u_last[b] * cum[-1]).sum()))
        outs.append(out + [-1] * (most - len(out)))
        paths.append(path + [-1] * (most - len(path)))
        counts.append(len(path) - 1)
    return [ints(outs), ints(paths), ints(counts)]
