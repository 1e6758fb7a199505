"""An attention block at work: one prompt, eight samples of it, their cache.

The block has the shape of a Qwen3-0.6B layer (hidden size 1024, 16 query heads and 8 key/value heads of 128, q4_K
weights; random, from the repository's generator).  A prompt goes through it once (prefill).  The sequence is then forked
into eight samples: they share the prompt's pages and get a copy of its partly filled last one.  Each step every sample
adds a token: q8_K activations, the packed products, rotary positions with the keys and values going straight to the
sample's slots, attention over the shared prompt and the sample's own tokens, the output product.  Half of the samples
then end, their pages are given back and the pool is packed, and the others go on.

    python examples/shared_prefix_decode.py

Every attention result is compared with its definition in f64, on keys and values that the example keeps for itself in
plain tensors.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gen  # noqa: E402
import quant_packed_gemv_gb300 as q  # noqa: E402

HIDDEN, HEADS, KV_HEADS, D, PAGE = 1024, 16, 8, 128, 16
PAGES, SEQS, WIDTH = 256, 16, 48          # the pool, and the table of its sequences
GROUP = HEADS // KV_HEADS


class Block:
    """The four packed matrices, the rotary frequencies, the pages and their tables."""

    def __init__(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = {"q": HEADS * D, "k": KV_HEADS * D, "v": KV_HEADS * D}
        self.w = {n: torch.from_numpy(gen.q4K_blocks(7, j, r, HIDDEN)).cuda() for j, (n, r) in enumerate(rows.items())}
        self.wo = torch.from_numpy(gen.q4K_blocks(7, 3, HIDDEN, HEADS * D)).cuda()
        self.rows = rows
        self.freqs, _ = q.plm_rope_freqs(D, 1e6, device="cuda")
        self.pool = torch.zeros(PAGES, 2, KV_HEADS, PAGE, D, dtype=torch.bfloat16, device="cuda")
        self.table, self.lens, self.refs = torch.full((SEQS, WIDTH), -1, **i32), torch.zeros(SEQS, **i32), torch.zeros(PAGES, **i32)
        self.status, self.live = torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.kv = q.plm_kv_state(self.pool, self.table, self.lens, self.refs, PAGE, self.status)
        self.workspace = torch.empty(max(q.plm_kv_workspace_size(PAGES, SEQS), 1 << 26), dtype=torch.uint8, device="cuda")

    def product(self, w, x, n):
        m, k = x.shape
        xq, y = torch.empty(m * (k // 256) * q.Q8K_BYTES, dtype=torch.uint8, device="cuda"), torch.empty(m, n, device="cuda")
        q.plm_quantize_q8K(x, xq, m, k)
        q.plm_gemm_q4K(w, xq, y, m, n, k)
        return y

    def forward(self, x, seqs, tokens, positions, prefix, max_len):
        """x [len(seqs) * tokens][HIDDEN]: each sequence's next tokens.  Returns the block's output, the attention's
        before the output product, and q, k, v as the products gave them."""
        n = len(seqs)
        ids = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        slots = torch.empty(n, tokens, dtype=torch.int64, device="cuda")
        q.plm_kv_reserve(self.kv, ids, torch.full((n,), tokens, dtype=torch.int32, device="cuda"), slots, self.workspace)
        y = {name: self.product(self.w[name], x, r).view(n * tokens, -1, D) for name, r in self.rows.items()}
        qr = torch.empty(n * tokens, HEADS, D, dtype=torch.bfloat16, device="cuda")
        slots = slots.view(-1)
        q.plm_rope([q.plm_rope_tensor(y["q"], qr), q.plm_rope_tensor(y["k"], self.pool[:, 0], slots=slots),
                    q.plm_rope_tensor(y["v"], self.pool[:, 1], slots=slots, rotate=False)], positions, self.freqs, D)
        o = torch.empty(n * tokens, HEADS, D, device="cuda")
        need = q.plm_attn_workspace_size(n, tokens, HEADS, KV_HEADS, D, prefix, max_len)
        assert need <= self.workspace.numel()
        q.plm_attn_shared_prefix(qr, o, self.pool[:, 0], self.pool[:, 1], self.table, self.lens, tokens, prefix, max_len, D ** -0.5,
                                 self.workspace, seqs=ids)
        return self.product(self.wo, o.view(n * tokens, -1), HIDDEN), o, y


class Record:
    """The same keys, values and attention by the definition: whole tensors per sequence, f64."""

    def __init__(self, freqs):
        self.k, self.v = {}, {}
        self.turns = torch.tensor([int(f) / 2.0 ** 64 for f in freqs.tolist()], dtype=torch.float64, device="cuda")

    def turned(self, x, positions):
        angle = 2 * torch.pi * torch.frac(positions.double()[:, None] * self.turns)[:, None]
        a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1).bfloat16().double()

    def step(self, seqs, tokens, y, positions):
        out, empty = [], torch.empty(0, KV_HEADS, D, dtype=torch.float64, device="cuda")
        turned_q, turned_k = self.turned(y["q"], positions), self.turned(y["k"], positions)
        for i, s in enumerate(seqs):
            rows = slice(i * tokens, (i + 1) * tokens)
            self.k[s] = torch.cat((self.k.get(s, empty), turned_k[rows]))
            self.v[s] = torch.cat((self.v.get(s, empty), y["v"][rows].bfloat16().double()))
            n = self.k[s].shape[0]
            x = torch.einsum("thgd,nhd->hgtn", turned_q[rows].view(tokens, KV_HEADS, GROUP, D), self.k[s]) * D ** -0.5
            late = torch.arange(n, device="cuda") > torch.arange(n - tokens, n, device="cuda")[:, None]
            p = torch.softmax(x.masked_fill(late, float("-inf")), -1)
            out.append(torch.einsum("hgtn,nhd->thgd", p, self.v[s]).reshape(tokens, HEADS, D))
        return torch.cat(out)

    def fork(self, parent, children):
        for c in children:
            self.k[c], self.v[c] = self.k[parent], self.v[parent]


def run(prompt=333, steps=24, samples=8, say=lambda *a: None):
    """Returns (largest relative error of an attention result, pages in use at the end, the outputs)."""
    torch.manual_seed(5)
    block, worst, outputs = Block(), 0.0, []
    record = Record(block.freqs)

    def forward(seqs, tokens, start, prefix, max_len):
        nonlocal worst
        x = torch.randn(len(seqs) * tokens, HIDDEN, device="cuda")
        positions = (start + torch.arange(tokens, device="cuda", dtype=torch.int32)).repeat(len(seqs))
        out, o, y = block.forward(x, seqs, tokens, positions, prefix, max_len)
        want = record.step(seqs, tokens, y, positions)
        worst = max(worst, float((o.double() - want).norm() / want.norm()))
        outputs.append(out)

    forward([0], prompt, 0, 0, prompt)
    children = list(range(1, samples + 1))
    c = torch.tensor(children, dtype=torch.int32, device="cuda")
    q.plm_kv_fork(block.kv, torch.zeros_like(c), c, block.workspace)
    record.fork(0, children)
    shared = prompt // PAGE * PAGE        # the full pages are the same for all samples
    for t in range(steps):
        if t == steps // 2:               # half of the samples end; the pool is packed
            q.plm_kv_free(block.kv, c[: samples // 2].contiguous())
            q.plm_kv_compact(block.kv, block.live, block.workspace)
            children = children[samples // 2:]
            say("after %d steps %d pages are in use" % (t, int(block.live)))
        forward(children, 1, prompt + t, shared, prompt + t + 1)
    q.plm_kv_compact(block.kv, block.live, block.workspace)
    if int(block.status):
        raise RuntimeError("the page calls flagged %d" % int(block.status))
    say("%d tokens of prompt, %d steps: largest error of an attention result %.1e" % (prompt, steps, worst))
    return worst, int(block.live), outputs


if __name__ == "__main__":
    run(say=print)
