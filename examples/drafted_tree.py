"""Steps of drafting over the 8-bit paged cache, as a server runs them: a tree of drafted
tokens a step, checked in one pass, what stands kept.

  token rows -> cq_gemm_q4 (q, k, v) -> cq_rope, cq_kv8_write_rope -> cq_attn_kv8_tree
    -> cq_gemm_q4 (logits) -> softmax -> cq_verify -> cq_kv8_write_rope of the rows that stand

The model is one attention layer with random Q4 weights; its draft is the same layer without
attention, the best two tokens at each of three levels (chosen, not drawn).
`python examples/drafted_tree.py [steps]` prints the drafted tokens that stood a step.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_weight_02_gb300 as cq  # noqa: E402

HIDDEN, HQ, HKV, D, PAGE, VOCAB = 512, 4, 2, 64, 32, 1024
PROMPTS = [30, 5, 64]
# the tree: the root, two children, two more of each, and so on: places 1 to 14
LEVELS, WIDTH = 3, 2
PARENTS = [-1] + [(i - 1) // WIDTH for i in range(1, sum(WIDTH ** n for n in range(LEVELS + 1)))]
ROWS = len(PARENTS)


def bits(parents):
    """Each node's ancestors and itself."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


class Model:
    def __init__(self, room, device="cuda", seed=0):
        self.gen, self.dev, self.B = torch.Generator(device).manual_seed(seed), torch.device(device), len(PROMPTS)
        w = lambda n, k, size: (torch.randint(0, 256, (n, k // 2), generator=self.gen, device=self.dev, dtype=torch.uint8),
                                (size * (0.2 + 0.1 * torch.rand(n, k // 32, generator=self.gen, device=self.dev)) / k ** 0.5).half().view(torch.int16))
        self.qkv, self.out, self.head = w((HQ + 2 * HKV) * D, HIDDEN, 1.0), w(HIDDEN, HQ * D, 2.0), w(VOCAB, HIDDEN, 2.0)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=self.gen, device=self.dev).bfloat16()
        self.rope = cq.cq_rope_spec.make(D, device=self.dev)
        pages = -(-(max(PROMPTS) + room) // PAGE)
        table = torch.randperm(pages * self.B, generator=self.gen, device=self.dev).int().view(self.B, pages)
        self.cache = cq.cq_kv8_cache.empty(pages * self.B, HKV, PAGE, D, table, self.dev)
        self.ws = torch.empty(1 << 24, dtype=torch.uint8, device=self.dev)
        most = max(sum(PROMPTS), self.B * ROWS)
        self.attn_ws = torch.empty(cq.cq_attn_kv8_workspace_bytes(most, HQ, HKV, D, self.B, max(max(PROMPTS), ROWS)), dtype=torch.uint8, device=self.dev)

    def times(self, x, w):
        y = torch.empty(len(x), len(w[0]), dtype=torch.bfloat16, device=self.dev)
        cq.cq_gemm_q4(x.contiguous(), *w, y, self.ws)
        return y

    def rows(self, tokens, q_start, lens, max_q, pos, mask=None):
        """Probabilities of what follows each row, and the rows' keys and values."""
        x = self.embed[tokens.long()]
        y = self.times(x, self.qkv).view(len(x), -1, D)
        q, k, v = y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]
        cq.cq_kv8_write_rope(self.cache, k, v, q_start, lens, self.rope, pos)
        cq.cq_rope(q, self.rope, pos)
        o = torch.empty(len(x), HQ, D, dtype=torch.bfloat16, device=self.dev)
        if mask is None:
            cq.cq_attn_kv8(q, self.cache, q_start, lens, max_q, o, self.attn_ws)
        else:
            cq.cq_attn_kv8_tree(q, self.cache, q_start, lens, max_q, mask, o, self.attn_ws)
        h = x + self.times(o.flatten(1), self.out)
        return torch.softmax(self.times(h, self.head).float(), 1), k, v

    def draft(self, last):
        """The best WIDTH tokens after each of the tree's nodes, as the layer without attention sees them."""
        tree = [last]
        for i in range(ROWS // WIDTH):
            logits = self.times(self.embed[tree[i].long()], self.head)
            tree += list(logits.topk(WIDTH, 1).indices.int().T)
        return torch.stack(tree[:ROWS], 1)                                             # [B][ROWS]


def run(steps=8, seed=0):
    """(tokens per sequence, drafted tokens that stood) after so many steps."""
    m = Model(steps * ROWS + ROWS, seed=seed)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=m.dev)
    start = [0]
    for n in PROMPTS:
        start.append(start[-1] + n)
    prompt = torch.randint(0, VOCAB, (start[-1],), generator=m.gen, device=m.dev).int()
    held = i32(PROMPTS)
    place = torch.cat([torch.arange(n, device=m.dev) for n in PROMPTS]).int()
    p, _, _ = m.rows(prompt, i32(start), held, max(PROMPTS), place)
    last = p[i32(start[1:]).long() - 1].argmax(1).int()

    q_start = i32([b * ROWS for b in range(m.B + 1)])
    mask = i32(bits(PARENTS)).repeat(m.B).view(-1, 1)
    depth = [0] * ROWS
    for i in range(1, ROWS):
        depth[i] = depth[PARENTS[i]] + 1
    depth, stood = i32(depth), 0
    out, path = (torch.empty(m.B, ROWS, dtype=torch.int32, device=m.dev) for _ in range(2))
    count = torch.empty(m.B, dtype=torch.int32, device=m.dev)
    texts = [[int(t)] for t in last]
    for _ in range(steps):
        tokens = m.draft(last).flatten().contiguous()
        pos = (held[:, None] + depth).flatten()
        p, k, v = m.rows(tokens, q_start, held + ROWS, ROWS, pos, mask)
        u, u_last = torch.rand(len(tokens), generator=m.gen, device=m.dev), torch.rand(m.B, generator=m.gen, device=m.dev)
        cq.cq_verify(p, tokens, q_start, ROWS, u, u_last, out, path, count, mask=mask)
        # the rows that stand, closed up, are the sequences' last tokens: the tree's others are written over
        keep = path.flatten()[path.flatten() >= 0].long()
        ends = torch.cat([i32([0]), (count + 1).cumsum(0).int()])
        held = held + count + 1
        cq.cq_kv8_write_rope(m.cache, k[keep].contiguous(), v[keep].contiguous(), ends, held, m.rope)
        last = out.gather(1, count.long()[:, None])[:, 0]
        stood += int(count.sum())
        for b in range(m.B):
            texts[b] += out[b, :int(count[b]) + 1].tolist()
    if cq.cq_get_device_error():
        raise RuntimeError("the device reported an error")
    return texts, stood


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 8
    texts, stood = run(n)
    print(f"{stood} drafted tokens stood in {n} steps of {len(PROMPTS)} sequences; {[len(t) for t in texts]} tokens in all")
