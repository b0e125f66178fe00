"""The 8-bit key/value cache and the attention over it, as measured cases.

The cache.  Keys and values are int8 codes in pages, Kq and Vq [pages][Hkv][page][D], with one f32 scale per 32
tokens and head, Ks and Vs [pages][Hkv][page / 32]; table[b][i] names the page that holds tokens i * page .. of
sequence b.  A value is code * scale; the scale is the smallest power of two 2^e (e >= -64) with amax <= 127 * 2^e
over the block's tokens, the code the nearest integer (ties to even).  Tokens that are appended to a block with
tokens in it may raise its scale; the codes that stay are then rounded to the new one.

The operators.  "store": new tokens' keys and values are written to the cache, then read back (the whole of each
sequence, or the 32-token block that a single new token went to).  "attend": softmax attention of ragged query rows
over the cache, grouped heads, causal (with or without a window) or not; a sequence's query rows are the last of its
tokens.
"""
import math
import random

import torch

own = False

BLOCK = 32
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # One sequence grows by one token, one layer of a model with 4 KV heads: a launch or two, latency only.
        {"name": "store_step_one", "kind": "store", "batch": 1, "hkv": 4, "d": 128, "page": 64, "base_min": 500, "base_max": 500, "new_min": 1, "new_max": 1,
         "type": "bf16", "out": "bf16", "back": "block", "mix": 1},
        # A decode step of a full batch: one token each, ragged lengths, most in a partly filled block.
        {"name": "store_step_batch", "kind": "store", "batch": 96, "hkv": 8, "d": 128, "page": 32, "base_min": 17, "base_max": 4000, "new_min": 1, "new_max": 1,
         "type": "f16", "out": "f16", "back": "block", "mix": 2},
        # Prompts of odd lengths behind short kept prefixes, f32 rows as a projection may leave them, narrow heads,
        # pages that are no power of two.
        {"name": "store_prompts", "kind": "store", "batch": 7, "hkv": 16, "d": 64, "page": 96, "base_min": 0, "base_max": 45, "new_min": 1, "new_max": 1500,
         "type": "f32", "out": "f32", "back": "all", "mix": 3},
        # Long prompts: four documents of 32768 tokens; memory traffic only.
        {"name": "store_documents", "kind": "store", "batch": 4, "hkv": 8, "d": 128, "page": 128, "base_min": 0, "base_max": 0, "new_min": 32768, "new_max": 32768,
         "type": "bf16", "out": "bf16", "back": "all", "mix": 4},
        # One user, one token, a short context: latency.
        {"name": "decode_one", "kind": "attend", "batch": 1, "hq": 32, "hkv": 4, "d": 128, "page": 64, "base_min": 776, "base_max": 776, "new_min": 1, "new_max": 1,
         "type": "bf16", "out": "bf16", "causal": True, "window": 0, "lse": False, "mix": 5},
        # A serving batch with mixed lengths, grouped heads: the cache is read once, nothing else counts.
        {"name": "decode_batch", "kind": "attend", "batch": 32, "hq": 32, "hkv": 8, "d": 128, "page": 64, "base_min": 1000, "base_max": 32767, "new_min": 1, "new_max": 1,
         "type": "bf16", "out": "bf16", "causal": True, "window": 0, "lse": False, "mix": 6},
        # Few sequences with very long contexts and wide groups: the work has to be split over the tokens.
        {"name": "decode_long", "kind": "attend", "batch": 3, "hq": 64, "hkv": 4, "d": 128, "page": 128, "base_min": 90001, "base_max": 131071, "new_min": 1, "new_max": 1,
         "type": "f16", "out": "f32", "causal": True, "window": 0, "lse": True, "mix": 7},
        # Heads of their own and narrow, with a sliding window over odd lengths.
        {"name": "decode_window", "kind": "attend", "batch": 48, "hq": 16, "hkv": 16, "d": 64, "page": 32, "base_min": 0, "base_max": 6001, "new_min": 1, "new_max": 1,
         "type": "f16", "out": "f16", "causal": True, "window": 1024, "lse": False, "mix": 8},
        # A few guessed tokens per sequence are checked in one pass; a group of five heads.
        {"name": "verify_few", "kind": "attend", "batch": 24, "hq": 40, "hkv": 8, "d": 128, "page": 64, "base_min": 300, "base_max": 9000, "new_min": 5, "new_max": 5,
         "type": "bf16", "out": "bf16", "causal": True, "window": 0, "lse": False, "mix": 9},
        # Prompts of mixed lengths, some behind kept context.
        {"name": "prefill_ragged", "kind": "attend", "batch": 6, "hq": 32, "hkv": 8, "d": 128, "page": 64, "base_min": 0, "base_max": 3000, "new_min": 1, "new_max": 2000,
         "type": "bf16", "out": "bf16", "causal": True, "window": 0, "lse": True, "mix": 10},
        # A block of 1024 rows that are refined together: every row sees its context and the whole block.
        {"name": "refine_block", "kind": "attend", "batch": 2, "hq": 24, "hkv": 24, "d": 128, "page": 128, "base_min": 3500, "base_max": 4100, "new_min": 1024, "new_max": 1024,
         "type": "bf16", "out": "bf16", "causal": False, "window": 0, "lse": False, "mix": 11},
        # A long prompt from its first token: matrix products and exponentials.
        {"name": "prefill_long", "kind": "attend", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "page": 128, "base_min": 0, "base_max": 0, "new_min": 16384, "new_max": 16384,
         "type": "bf16", "out": "bf16", "causal": True, "window": 0, "lse": False, "mix": 12},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def span(base, new):
        return {"base_min": base[0], "base_max": base[1], "new_min": new[0], "new_max": new[1]}

    common = {"page": rng.choice([32, 64, 96, 128, 256]), "type": rng.choice(["f16", "bf16"]), "mix": rng.randrange(1 << 30)}
    if rng.random() < 0.3:
        hkv, d = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128])
        step = rng.random() < 0.5
        if step:
            batch = log_int(1, 128)
            base, new = sorted([log_int(1, 6000), log_int(1, 6000)]), [1, 1]
        else:
            batch = log_int(1, 12)
            base = [0, log_int(1, 300)]
            new = sorted([log_int(1, 8000), log_int(1, 8000)])
        if not step and rng.random() < 0.3:
            common["type"] = "f32"
        return {**common, **span(base, new), "kind": "store", "batch": batch, "hkv": hkv, "d": d, "out": rng.choice([common["type"], "f32"]),
                "back": "block" if step else "all"}
    hkv, d, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    while hkv * group > 64:
        group = rng.choice([1, 2, 3, 4])
    case = {**common, "kind": "attend", "hq": hkv * group, "hkv": hkv, "d": d, "out": rng.choice([common["type"], "f32"]),
            "causal": True, "window": 0, "lse": rng.random() < 0.3}
    which = rng.choice(["decode", "decode", "few", "prompt", "chunk", "block"])
    if which == "decode" or which == "few":
        case["batch"] = log_int(1, 64)
        top = max(64, min(100000, 300000 // case["batch"]))
        base = sorted([log_int(1, top), log_int(1, top)])
        new = [1, 1] if which == "decode" else [1, rng.randrange(2, 17)]
    elif which == "prompt":
        case["batch"] = log_int(1, 8)
        base = [0, log_int(1, 500)]
        new = sorted([log_int(1, 6000), log_int(1, 6000)])
    elif which == "chunk":
        case["batch"] = 1
        base = [log_int(500, 60000)] * 2
        new = [log_int(17, 1000)] * 2
    else:
        case["batch"] = log_int(1, 4)
        case["causal"] = False
        base = sorted([log_int(1, 5000), log_int(1, 5000)])
        new = [log_int(64, 1024)] * 2
    case.update(span(base, new))
    if case["causal"] and rng.random() < 0.3:
        case["window"] = log_int(16, 4096)
    if work(case)["flops"] > 1e12:
        return draw(rng)
    return case


def lengths(case):
    """(tokens held before, new tokens) of each sequence: spread over the case's ranges, both ends among them."""
    rng = random.Random(case["mix"])
    n = case["batch"]
    out = []
    for lo, hi in ((case["base_min"], case["base_max"]), (case["new_min"], case["new_max"])):
        v = [lo + (hi - lo) * i // max(n - 1, 1) for i in range(n)]
        v = [x if i in (0, n - 1) else max(lo, min(hi, x - rng.randrange(0, 1 + (hi - lo) // n))) for i, x in enumerate(v)]
        rng.shuffle(v)
        out.append(v)
    return out


def seen(case, base, new):
    """(visible pairs, keys that any row sees) of one sequence."""
    total = base + new
    if not case["causal"]:
        return new * total, total
    w = case["window"] or total
    pairs = sum(min(p + 1, w) for p in range(base, total)) if w < total else new * base + new * (new + 1) // 2
    return pairs, min(total, w + new - 1)


def work(case):
    base, new = lengths(case)
    hkv, d = case["hkv"], case["d"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    per_key = 2 * hkv * (d + 4 / BLOCK)
    if case["kind"] == "store":
        rows = sum(new)
        back = sum((b + n - 1) % BLOCK + 1 if case["back"] == "block" else b + n for b, n in zip(base, new))
        moved = 2 * hkv * d * (rows * size[case["type"]] + back * size[case["out"]]) + per_key * (rows + back)
        return {"bytes": int(moved), "flops": 4 * hkv * d * (rows + back)}
    both = [seen(case, b, n) for b, n in zip(base, new)]
    rows = sum(new)
    moved = rows * case["hq"] * (d * (size[case["type"]] + size[case["out"]]) + (4 if case["lse"] else 0))
    moved += per_key * sum(k for _, k in both)
    return {"bytes": int(moved), "flops": 4 * d * case["hq"] * sum(p for p, _ in both)}


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


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    base, new = lengths(case)
    total = [b + n for b, n in zip(base, new)]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    per = [(t + page - 1) // page for t in total]
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).int()
    table = torch.full((case["batch"], max(per) + 1), -1, dtype=torch.int32, device=DEV)   # unused entries name no page
    at = starts(per)
    for b, n in enumerate(per):
        table[b, :n] = order[at[b]:at[b] + n]
    held = base if case["kind"] == "store" else total
    kq, ks, vq, vs = filled(gen, case, held, table, pages)
    st = {"case": case, "base": base, "new": new, "total": total, "kq": kq, "ks": ks, "vq": vq, "vs": vs, "table": table,
          "q_start": torch.tensor(starts(new), dtype=torch.int32, device=DEV),
          "lens": torch.tensor(total, dtype=torch.int32, device=DEV)}
    rows, dt, odt = sum(new), TYPES[case["type"]], TYPES[case["out"]]
    if case["kind"] == "store":
        st["k"] = rows_of(gen, rows, hkv, d, False).to(dt)
        st["v"] = rows_of(gen, rows, hkv, d, True).to(dt)
        first = [(t - 1) // BLOCK * BLOCK if case["back"] == "block" else 0 for t in total]
        back = [t - f for t, f in zip(total, first)]
        st["first_host"], st["back"] = first, back
        st["first"] = torch.tensor(first, dtype=torch.int32, device=DEV)
        st["out_start"] = torch.tensor(starts(back), dtype=torch.int32, device=DEV)
        if own:
            st["k_out"] = torch.empty(sum(back), hkv, d, dtype=odt, device=DEV)
            st["v_out"] = torch.empty(sum(back), hkv, d, dtype=odt, device=DEV)
        else:
            plan_store(st)
    else:
        st["q"] = torch.randn(rows, case["hq"], d, generator=gen, device=DEV).to(dt)
        if own:
            st["o"] = torch.empty(rows, case["hq"], d, dtype=odt, device=DEV)
            st["lse"] = torch.empty(rows, case["hq"], dtype=torch.float32, device=DEV) if case["lse"] else None
    if own:
        import block_quantized_weight_02_gb300 as cq
        st["cq"] = cq
        st["cache"] = cq.cq_kv8_cache(kq, ks, vq, vs, table)
        if case["kind"] == "attend":
            size = cq.cq_attn_kv8_workspace_bytes(rows, case["hq"], hkv, d, case["batch"], max(new))
            st["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    return st


def plan_store(st):
    """Where each new token goes, for the plain form: its block, its row there, and the blocks that are touched."""
    page, table = st["case"]["page"], st["table"].long()
    tok, touched, kept = [], [], []
    for b, (base, n) in enumerate(zip(st["base"], st["new"])):
        p = torch.arange(base, base + n, device=DEV)
        blk = torch.arange(base // BLOCK, (base + n - 1) // BLOCK + 1, device=DEV)
        page_of = table[b][p // page]
        tok.append(torch.stack([page_of, p % page // BLOCK, p % BLOCK, p // BLOCK - base // BLOCK + sum(x.shape[0] for x in touched)]))
        touched.append(torch.stack([table[b][blk * BLOCK // page], blk * BLOCK % page // BLOCK], 1))
        kept.append((base - blk * BLOCK).clamp(0, BLOCK))
    st["tok"], st["touched"], st["kept"] = torch.cat(tok, 1), torch.cat(touched), torch.cat(kept)


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        cq = st["cq"]
        if st["case"]["kind"] == "store":
            cq.cq_kv8_write(st["cache"], st["k"], st["v"], st["q_start"], st["lens"])
            cq.cq_kv8_read(st["cache"], st["first"], st["out_start"], st["k_out"], st["v_out"])
            return [st["k_out"], st["v_out"]]
        c = st["case"]
        cq.cq_attn_kv8(st["q"], st["cache"], st["q_start"], st["lens"], max(st["new"]), st["o"], st["ws"],
                       scale=1.0 / math.sqrt(c["d"]), causal=c["causal"], window=c["window"], lse=st["lse"])
        return [st["o"], st["lse"]] if c["lse"] else [st["o"]]
    if st["case"]["kind"] == "store":
        return [plain_store(st, st["k"], st["kq"], st["ks"]), plain_store(st, st["v"], st["vq"], st["vs"])]
    return plain_attend(st)


def plain_store(st, x, codes, scales):
    case = st["case"]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    c5 = codes.view(-1, hkv, page // BLOCK, BLOCK, d)
    x = x.float()
    pg, blk, row, slot = st["tok"]
    tp, tb = st["touched"][:, 0], st["touched"][:, 1]
    kept = st["kept"]
    amax = torch.zeros(tp.shape[0], hkv, device=DEV).index_reduce_(0, slot, x.abs().amax(2), "amax")
    s0 = scales[tp, :, tb]
    s1 = exponent_scale(amax)
    s1 = torch.where(kept[:, None] > 0, torch.maximum(s0, s1), s1)
    part = kept.nonzero()[:, 0]
    if part.numel():
        old = c5[tp[part], :, tb[part]]
        moved = torch.round(old.float() * (s0 / s1)[part][:, :, None, None]).to(torch.int8)
        stays = torch.arange(BLOCK, device=DEV)[None, None, :, None] < kept[part][:, None, None, None]
        c5[tp[part], :, tb[part]] = torch.where(stays, moved, old)
    scales[tp, :, tb] = s1
    c5[pg, :, blk, row] = torch.round(x / s1[slot][:, :, None]).to(torch.int8)
    out = []
    for b, (first, n) in enumerate(zip(st["first_host"], st["back"])):
        keys = plain_keys(st, codes, scales, b, first, first + n)
        out.append(keys.to(TYPES[case["out"]]))
    return torch.cat(out)


def plain_keys(st, codes, scales, b, lo, hi):
    """Tokens lo .. hi - 1 of sequence b as [tokens][Hkv][D] f32."""
    page = st["case"]["page"]
    p = torch.arange(lo, hi, device=DEV)
    pg = st["table"][b].long()[p // page]
    return codes[pg, :, p % page].float() * scales[pg, :, p % page // BLOCK][:, :, None]


def plain_attend(st):
    case = st["case"]
    hq, hkv, d, group = case["hq"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    q = st["q"].float().view(-1, hkv, group, d)
    outs, sums = [], []
    at = 0
    for b, (base, n) in enumerate(zip(st["base"], st["new"])):
        lo = max(0, base - case["window"] + 1) if case["window"] else 0
        total = base + n
        k = plain_keys(st, st["kq"], st["ks"], b, lo, total).transpose(0, 1)             # [Hkv][keys][D]
        v = plain_keys(st, st["vq"], st["vs"], b, lo, total).transpose(0, 1)
        key = torch.arange(lo, total, device=DEV)
        step = max(1, (1 << 29) // (hq * (total - lo)))
        for i in range(0, n, step):
            m = min(step, n - i)
            x = q[at + i:at + i + m].permute(1, 0, 2, 3).reshape(hkv, m * group, d)
            s = torch.bmm(x, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
            if case["causal"]:
                pos = torch.arange(base + i, base + i + m, device=DEV).repeat_interleave(group)[:, None]
                hide = key[None, :] > pos
                if case["window"]:
                    hide |= key[None, :] <= pos - case["window"]
                s.masked_fill_(hide, float("-inf"))
            top = s.amax(2, keepdim=True)
            s = torch.exp(s - top)
            z = s.sum(2, keepdim=True)
            o = torch.bmm(s, v) / z
            outs.append(o.view(hkv, m, group, d).transpose(0, 1).reshape(m, hq, d).to(TYPES[case["out"]]))
            sums.append((top + torch.log(z)).view(hkv, m, group).transpose(0, 1).reshape(m, hq))
        at += n
    return [torch.cat(outs), torch.cat(sums)] if case["lse"] else [torch.cat(outs)]


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    table = st["table"].cpu().tolist()

    def tokens(codes, scales, b, h, n):
        """The first n tokens of a head, f64 codes and scales of their blocks."""
        ids = torch.tensor(table[b][:(n + page - 1) // page], device=DEV, dtype=torch.long)
        c = codes[ids, h].reshape(-1, d)[:n].double()
        s = scales[ids, h].reshape(-1)[:(n + BLOCK - 1) // BLOCK].double()
        return c, s

    if case["kind"] == "store":
        def least(a):
            e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 127.0))
            e = torch.where(a <= 127.0 * torch.exp2(e - 1), e - 1, e)
            e = torch.where(a > 127.0 * torch.exp2(e), e + 1, e)
            return torch.exp2(e.clamp(min=-64))

        both = []
        for x, codes, scales in ((st["k"], st["kq"], st["ks"]), (st["v"], st["vq"], st["vs"])):
            parts, at = [], 0
            for b, (base, n, first) in enumerate(zip(st["base"], st["new"], st["first_host"])):
                heads = []
                for h in range(hkv):
                    c, s0 = tokens(codes, scales, b, h, base) if base else (torch.zeros(0, d, device=DEV).double(), torch.zeros(0, device=DEV).double())
                    total, edge = base + n, base // BLOCK * BLOCK
                    xs = x[at:at + n, h].double()
                    grown = torch.zeros((total - edge + BLOCK - 1) // BLOCK * BLOCK, device=DEV).double()
                    grown[base - edge:total - edge] = xs.abs().amax(1)
                    s1 = least(grown.view(-1, BLOCK).amax(1))
                    if base % BLOCK:
                        s1[0] = torch.maximum(s1[0], s0[-1])
                        tail = torch.round(c[edge:] * s0[-1] / s1[0]) * s1[0]
                    else:
                        tail = c[edge:]
                    whole = (c[:edge].view(-1, BLOCK, d) * s0[:edge // BLOCK, None, None]).view(-1, d)
                    per = s1[torch.arange(base - edge, total - edge, device=DEV) // BLOCK][:, None]
                    heads.append(torch.cat([whole, tail, torch.round(xs / per) * per])[first:])
                parts.append(torch.stack(heads, 1))
                at += n
            both.append(torch.cat(parts))
        return both

    group = case["hq"] // hkv
    o = torch.zeros(sum(st["new"]), case["hq"], d, device=DEV, dtype=torch.float64)
    z = torch.zeros(sum(st["new"]), case["hq"], device=DEV, dtype=torch.float64)
    at = 0
    for b, (base, n) in enumerate(zip(st["base"], st["new"])):
        for h in range(hkv):
            (kc, ksc), (vc, vsc) = tokens(st["kq"], st["ks"], b, h, base + n), tokens(st["vq"], st["vs"], b, h, base + n)
            k = kc * ksc.repeat_interleave(BLOCK)[:base + n, None]
            v = vc * vsc.repeat_interleave(BLOCK)[:base + n, None]
            step = max(1, (1 << 26) // (group * (base + n)))
            for i in range(0, n, step):
                m = min(step, n - i)
                hi = base + i + m if case["causal"] else base + n
                lo = max(0, base + i - case["window"] + 1) if case["causal"] and case["window"] else 0
                x = st["q"][at + i:at + i + m, h * group:(h + 1) * group].double()
                s = torch.einsum("mgd,kd->mgk", x, k[lo:hi]) / math.sqrt(d)
                if case["causal"]:
                    ahead = torch.arange(lo, hi, device=DEV)[None] - torch.arange(base + i, base + i + m, device=DEV)[:, None]
                    bad = ahead > 0
                    if case["window"]:
                        bad = bad | (ahead <= -case["window"])
                    s = torch.where(bad[:, None], torch.full_like(s, float("-inf")), s)
                l = torch.logsumexp(s, 2)
                o[at + i:at + i + m, h * group:(h + 1) * group] = torch.einsum("mgk,kd->mgd", torch.exp(s - l[..., None]), v[lo:hi])
                z[at + i:at + i + m, h * group:(h + 1) * group] = l
        at += n
    return [o, z] if case["lse"] else [o]
