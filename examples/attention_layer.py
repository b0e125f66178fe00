"""One attention layer of a decoder with Q4 weights and the 8-bit paged cache,
run as a server runs it: ragged prompts first, then single tokens out of one
captured CUDA graph.

  x -> cq_gemm_q4 (q, k, v in one product) -> cq_kv8_write -> cq_attn_kv8
    -> cq_gemm_q4 (output projection)

`python examples/attention_layer.py [steps]` prints how far each phase's
attention is from a plain one over the cache as cq_kv8_read gives it back, and
the time of a single-token step.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_weight_02_gb300 as cq  # noqa: E402

HIDDEN, HQ, HKV, D, PAGE = 1024, 8, 2, 128, 64
PROMPTS = [300, 17, 64, 1, 129, 700]


class Layer:
    def __init__(self, room, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        self.dev, self.gen = torch.device(device), gen
        self.B = len(PROMPTS)
        # Q4 weights: nibbles and fp16 block scales
        self.qkv, self.out = self.weight((HQ + 2 * HKV) * D, HIDDEN), self.weight(HIDDEN, HQ * D)
        # pages in any order, room for `room` more tokens each
        per = [-(-(n + room) // PAGE) for n in PROMPTS]
        order = torch.randperm(sum(per), generator=gen, device=device).int()
        table = torch.zeros(self.B, max(per), dtype=torch.int32, device=device)
        for b, part in enumerate(order.split(per)):
            table[b, :len(part)] = part
        self.cache = cq.cq_kv8_cache.empty(sum(per), HKV, PAGE, D, table, device)

    def weight(self, n, k):
        q = torch.randint(0, 256, (n, k // 2), generator=self.gen, device=self.dev, dtype=torch.uint8)
        s = (0.2 + 0.1 * torch.rand(n, k // 32, generator=self.gen, device=self.dev)) / k ** 0.5
        return q, s.half().view(torch.int16)

    def buffers(self, T, max_q):
        """What a call over T rows needs, allocated once."""
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=self.dev)
        size = max(cq.cq_gemm_q4_workspace_bytes(T, HIDDEN), cq.cq_gemm_q4_workspace_bytes(T, HQ * D))
        return {"y": e(T, HQ + 2 * HKV, D), "o": e(T, HQ, D), "out": e(T, HIDDEN), "ws": e(max(size, 1), dtype=torch.uint8),
                "attn_ws": e(cq.cq_attn_kv8_workspace_bytes(T, HQ, HKV, D, self.B, max_q), dtype=torch.uint8), "max_q": max_q}

    def forward(self, x, q_start, lens, buf):
        """x [T][HIDDEN] are the last tokens of sequences that hold lens tokens with them."""
        y, o = buf["y"], buf["o"]
        cq.cq_gemm_q4(x, *self.qkv, y.view(len(x), -1), buf["ws"])
        q, k, v = y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]         # slices: no copies
        cq.cq_kv8_write(self.cache, k, v, q_start, lens)
        cq.cq_attn_kv8(q, self.cache, q_start, lens, buf["max_q"], o, buf["attn_ws"])
        cq.cq_gemm_q4(o.view(len(x), -1), *self.out, buf["out"], buf["ws"])
        return buf["out"]

    def error(self, counts, lens, buf):
        """The attention's distance from a plain one in 64 bits, over what 11-bit weights (the smallest are dropped) and a
        bf16 output allow."""
        start = torch.tensor([0] + lens, device=self.dev).cumsum(0).int()
        k = torch.empty(sum(lens), HKV, D, device=self.dev)
        v = torch.empty_like(k)
        cq.cq_kv8_read(self.cache, None, start, k, v)
        worst, at, tok = 0.0, 0, 0
        for n, L in zip(counts, lens):
            q = buf["y"][at:at + n, :HQ].double().unflatten(1, (HKV, -1))
            kk, vv = k[tok:tok + L].double(), v[tok:tok + L].double()
            s = torch.einsum("ihgd,jhd->hgij", q, kk) * D ** -0.5
            ahead = torch.arange(L, device=self.dev) > torch.arange(L - n, L, device=self.dev)[:, None]
            w = torch.softmax(s.masked_fill(ahead, float("-inf")), -1)
            ref, mass = (torch.einsum("hgij,jhd->ihgd", w, t).flatten(1, 2) for t in (vv, vv.abs()))
            err = (buf["o"][at:at + n].double() - ref).abs()
            worst = max(worst, float((err / (2 ** -8 * ref.abs() + 2 ** -9 * mass + 2 ** -20 * vv.abs().amax())).amax()))
            at, tok = at + n, tok + L
        return worst


def run(steps=32):
    """(prompt error, last step's error, us a step); errors are in units of what the roundings allow."""
    layer = Layer(steps + 8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=layer.dev)
    x = torch.randn(sum(PROMPTS), HIDDEN, generator=layer.gen, device=layer.dev).bfloat16()
    buf = layer.buffers(len(x), max(PROMPTS))
    starts = [0]
    for n in PROMPTS:
        starts.append(starts[-1] + n)
    layer.forward(x, i32(starts), i32(PROMPTS), buf)
    prompt = layer.error(PROMPTS, PROMPTS, buf)

    # single tokens: the step counts the lengths up on the device, so that one graph serves them all
    one = layer.buffers(layer.B, 1)
    tok = torch.randn(layer.B, HIDDEN, generator=layer.gen, device=layer.dev).bfloat16()
    each, lens = i32(list(range(layer.B + 1))), i32(PROMPTS)

    def step():
        lens.add_(1)
        y = layer.forward(tok, each, lens, one)
        tok.copy_(torch.nn.functional.rms_norm(y, (HIDDEN,)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if cq.cq_get_device_error():
        raise RuntimeError("the device reported an error")
    last = layer.error([1] * layer.B, [n + 1 + steps for n in PROMPTS], one)
    return prompt, last, begin.elapsed_time(end) * 1e3 / max(steps, 1)


if __name__ == "__main__":
    p, s, us = run(int(sys.argv[1]) if len(sys.argv) > 1 else 32)
    print(f"prompts of {PROMPTS}: error {p:.3f} of what the roundings allow")
    print(f"single tokens: error {s:.3f}, {us:.1f} us a step for {len(PROMPTS)} sequences")
