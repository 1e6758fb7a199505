"""A whole decoder on packed weights: a prompt, then a batch of samples of it, token by token.

The model is small and random (hidden size 1024, 16 query heads and 8 key/value heads of 128, q4_K matrices, a q6_K head;
from the repository's generator), its steps are those of a Qwen3 layer.  Between the packed products everything runs in this
package: residual sums and norms into q8_K activations, norms of the heads, rotary positions, a cache in 8 bits whose pages
hold all layers, attention over it with the prompt shared by all samples, and the choice of each sample's next token by its
own temperature, top-k, top-p and min-p.

    python examples/packed_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gen  # noqa: E402
import quant_packed_gemv_gb300 as q  # noqa: E402

HIDDEN, HEADS, KV_HEADS, D, FFN, VOCAB, LAYERS = 1024, 16, 8, 128, 2048, 8192, 2
PAGE, PAGES, SEQS, WIDTH, EPS = 16, 256, 16, 48, 1e-6
ROWS = {"q": (HEADS * D, HIDDEN), "k": (KV_HEADS * D, HIDDEN), "v": (KV_HEADS * D, HIDDEN), "o": (HIDDEN, HEADS * D),
        "gate": (FFN, HIDDEN), "up": (FFN, HIDDEN), "down": (HIDDEN, FFN)}


class Model:
    def __init__(self, seed=11):
        torch.manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        near_one = lambda n: 1 + 0.1 * torch.randn(n, device="cuda")  # noqa: E731
        self.packed = [{name: gen.q4K_blocks(seed, 16 * l + j, n, k) for j, (name, (n, k)) in enumerate(ROWS.items())} for l in range(LAYERS)]
        self.packed_head = gen.q6K_blocks(seed, 1000, VOCAB, HIDDEN)
        self.w = [{name: torch.from_numpy(b).cuda() for name, b in layer.items()} for layer in self.packed]
        self.head = torch.from_numpy(self.packed_head).cuda()
        self.norms = [{"in": near_one(HIDDEN), "q": near_one(D), "k": near_one(D), "ffn": near_one(HIDDEN)} for _ in range(LAYERS)]
        self.last_norm, self.embedding = near_one(HIDDEN), torch.randn(VOCAB, HIDDEN, device="cuda")
        self.freqs, _ = q.plm_rope_freqs(D, 1e6, device="cuda")
        # a page holds every layer's keys and values of 16 tokens
        size = q.plm_kv8_page_bytes(KV_HEADS, PAGE, D)
        self.pool = torch.zeros(PAGES, LAYERS * size, dtype=torch.uint8, device="cuda")
        self.cache = [q.plm_kv8_views(self.pool[:, l * size:(l + 1) * size], KV_HEADS, PAGE, D) for l in range(LAYERS)]
        self.table, self.lens, self.refs = torch.full((SEQS, WIDTH), -1, **i32), torch.zeros(SEQS, **i32), torch.zeros(PAGES, **i32)
        self.status = torch.zeros(1, **i32)
        self.kv = q.plm_kv_state(self.pool, self.table, self.lens, self.refs, PAGE, self.status)
        self.workspace = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def product(self, w, xq, n, k):
        m = xq.shape[0]
        y = torch.empty(m, n, device="cuda")
        q.plm_gemm_q4K(w, xq, y, m, n, k)
        return y

    def blocks(self, m, k):
        return torch.empty(m, k // 256 * q.Q8K_BYTES, dtype=torch.uint8, device="cuda")

    def forward(self, ids, seqs, tokens, positions, prefix, max_len):
        """Logits behind the last of each sequence's next `tokens` tokens, ids [len(seqs) * tokens]."""
        n = len(seqs)
        m, which = n * tokens, torch.tensor(seqs, dtype=torch.int32, device="cuda")
        slots = torch.empty(n, tokens, dtype=torch.int64, device="cuda")
        q.plm_kv_reserve(self.kv, which, torch.full((n,), tokens, dtype=torch.int32, device="cuda"), slots, self.workspace)
        slots = slots.view(-1)
        h, delta, xq = self.embedding[ids.long()], None, self.blocks(m, HIDDEN)
        assert q.plm_attn_kv8_workspace_size(n, tokens, HEADS, KV_HEADS, D, prefix, max_len) <= self.workspace.numel()
        for w, norm, (ck, cv, ek, ev) in zip(self.w, self.norms, self.cache):
            if delta is None:
                q.plm_rmsnorm(h, norm["in"], EPS, xq=xq)
            else:   # the last layer's output joins the residual, in its place
                q.plm_rmsnorm(delta, norm["in"], EPS, residual=h, sum=h, xq=xq)
            y = {name: self.product(w[name], xq, *ROWS[name]) for name in "qkv"}
            for name in "qk":   # every head by itself, in place
                rows = y[name].view(-1, D)
                q.plm_rmsnorm(rows, norm[name], EPS, y=rows)
            y = {name: x.view(m, -1, D) for name, x in y.items()}
            turned = torch.empty(m, HEADS, D, dtype=torch.bfloat16, device="cuda")
            q.plm_rope([q.plm_rope_tensor(y["q"], turned)], positions, self.freqs, D)
            q.plm_kv8_write([q.plm_kv8_tensor(y["k"], ck, ek, slots), q.plm_kv8_tensor(y["v"], cv, ev, slots, rotate=False)], positions,
                            self.freqs, D)
            o = torch.empty(m, HEADS, D, device="cuda")
            q.plm_attn_kv8(turned, o, ck, cv, ek, ev, self.table, self.lens, tokens, prefix, max_len, D ** -0.5, self.workspace, seqs=which)
            oq = self.blocks(m, HEADS * D)
            q.plm_quantize_q8K(o, oq, m, HEADS * D)
            delta = self.product(w["o"], oq, *ROWS["o"])
            q.plm_rmsnorm(delta, norm["ffn"], EPS, residual=h, sum=h, xq=xq)
            act = torch.empty(m, FFN, device="cuda")
            q.plm_gemm_q4K_swiglu(w["gate"], w["up"], xq, act, m, FFN, HIDDEN)
            aq = self.blocks(m, FFN)
            q.plm_quantize_q8K(act, aq, m, FFN)
            delta = self.product(w["down"], aq, *ROWS["down"])
        ends = slice(tokens - 1, None, tokens)
        xq = self.blocks(n, HIDDEN)
        q.plm_rmsnorm(delta[ends], self.last_norm, EPS, residual=h[ends], xq=xq)
        logits = torch.empty(n, VOCAB, device="cuda")
        q.plm_gemm_q6K(self.head, xq, logits, n, VOCAB, HIDDEN)
        return logits


def run(prompt=75, steps=20, samples=6, say=lambda *a: None):
    """Returns the tokens of each sample [samples][steps + 1], their probabilities, the prompt, and the model."""
    model, f32 = Model(), dict(dtype=torch.float32, device="cuda")
    ids = torch.randint(0, VOCAB, (prompt,), device="cuda", dtype=torch.int32)
    logits = model.forward(ids, [0], prompt, torch.arange(prompt, dtype=torch.int32, device="cuda"), 0, prompt)
    children = list(range(1, samples + 1))
    c = torch.tensor(children, dtype=torch.int32, device="cuda")
    q.plm_kv_fork(model.kv, torch.zeros_like(c), c, model.workspace)
    shared = prompt // PAGE * PAGE
    # the first sample is greedy, the others differ
    rules = dict(temperature=torch.tensor(([0.0, 1.0, 0.7, 0.7, 1.2, 1.0] * samples)[:samples], **f32),
                 top_k=torch.tensor(([0, 0, 20, 0, 50, 0] * samples)[:samples], dtype=torch.int32, device="cuda"),
                 top_p=torch.tensor(([1.0, 1.0, 1.0, 0.9, 0.95, 1.0] * samples)[:samples], **f32),
                 min_p=torch.tensor(([0.0, 0.0, 0.0, 0.0, 0.02, 0.1] * samples)[:samples], **f32))
    spread = logits.std()   # random weights give large logits; a trained model's need no such thing
    logits, found, probs = logits.expand(samples, VOCAB).contiguous(), [], []
    for t in range(steps + 1):
        tokens, prob, u = torch.empty(samples, dtype=torch.int32, device="cuda"), torch.empty(samples, **f32), torch.rand(samples, device="cuda")
        q.plm_sample(logits * (3.0 / spread), tokens, u=u, prob=prob, **rules)
        found.append(tokens)
        probs.append(prob)
        if t < steps:
            positions = torch.full((samples,), prompt + t, dtype=torch.int32, device="cuda")
            logits = model.forward(tokens, children, 1, positions, shared, prompt + t + 1)
    if int(model.status):
        raise RuntimeError("the page calls flagged %d" % int(model.status))
    found, probs = torch.stack(found, 1), torch.stack(probs, 1)
    for row, p in zip(found.tolist(), probs.tolist()):
        say(" ".join("%d" % v for v in row[:10]), "..  mean probability %.3f" % (sum(p) / len(p)))
    return found, probs, ids, model


if __name__ == "__main__":
    run(say=print)
