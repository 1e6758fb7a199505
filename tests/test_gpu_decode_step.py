"""The steps of a decoder together: examples/packed_decode.py against the same chain in f64.

The chain here takes the packed products from the oracle on its own q8_K activations, and the norms, positions, the cache's
rounding, attention and residuals from their definitions in f64.  Both round at the same places (q8_K activations, q in bf16,
the cache in 8 bits), so they differ where a value next to a border is rounded the other way: a code in some hundred, each off
by a 128th of its block's largest value, and the second product of the attention by 2^-11.  Over the products' sums of 1024 and
more terms that is below 1e-3 of a result's norm per layer, and 1e-2 leaves room for five times as much over two layers."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import quant_packed_gemv_gb300 as q
from tests.test_gpu_kv8 import decode, encode

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "packed_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("packed_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def chain(E, model, ids):
    """Logits behind the last of the tokens ids, all numpy f64."""
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    norm = lambda x, w: x / np.sqrt((x ** 2).mean(-1, keepdims=True) + E.EPS) * host(w)  # noqa: E731

    def product(w, x, n, k, kind="q4K"):
        xq = oracle.quantize_q8K(np.ascontiguousarray(x.astype(np.float32)))
        return np.asarray(getattr(oracle, "gemm_%s_f64" % kind)(w, xq, x.shape[0], n, k)).reshape(x.shape[0], n)

    m = len(ids)
    turns = np.array([int(f) / 2.0 ** 64 for f in model.freqs.tolist()])
    angle = 2 * np.pi * ((np.arange(m)[:, None] * turns) % 1.0)[:, None]

    def turned(x):
        a, b = x[..., :E.D // 2], x[..., E.D // 2:]
        return np.concatenate((a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)), -1)

    stored = lambda x: decode(*encode(x.astype(np.float32)))  # noqa: E731
    h = host(model.embedding)[ids]
    for w, n in zip(model.packed, model.norms):
        x = norm(h, n["in"])
        y = {name: product(w[name], x, *E.ROWS[name]).reshape(m, -1, E.D) for name in "qkv"}
        qv = torch.from_numpy(turned(norm(y["q"], n["q"]))).bfloat16().double().numpy()
        k, v = stored(turned(norm(y["k"], n["k"]))), stored(y["v"])
        s = np.einsum("thgd,nhd->hgtn", qv.reshape(m, E.KV_HEADS, -1, E.D), k) * E.D ** -0.5
        s[..., np.arange(m)[None] > np.arange(m)[:, None]] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        o = np.einsum("hgtn,nhd->thgd", p / p.sum(-1, keepdims=True), v).reshape(m, -1)
        h = h + product(w["o"], o, *E.ROWS["o"])
        x = norm(h, n["ffn"])
        g, u = (product(w[name], x, *E.ROWS[name]) for name in ("gate", "up"))
        h = h + product(w["down"], g / (1 + np.exp(-g)) * u, *E.ROWS["down"])
    return product(model.packed_head, norm(h[-1:], model.last_norm), E.VOCAB, E.HIDDEN, "q6K")[0]


def test_a_prompt_and_a_step_against_the_chain():
    E = example()
    model = E.Model()
    ids = np.random.RandomState(3).randint(0, E.VOCAB, 22)
    dev = torch.from_numpy(ids.astype(np.int32)).cuda()
    at = torch.arange(22, dtype=torch.int32, device="cuda")
    for cut in (21, 20):   # a prompt, then a token of two samples that share it
        got = model.forward(dev[:cut], [0], cut, at[:cut], 0, cut)[0].double().cpu().numpy() if cut == 21 else None
        if got is None:
            both = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
            q.plm_kv_fork(model.kv, torch.zeros_like(both), both, model.workspace)
            out = model.forward(dev[21:].repeat(2), [1, 2], 1, at[21:].repeat(2), 16, 22)
            assert torch.equal(out[0], out[1])
            got, cut = out[0].double().cpu().numpy(), 22
        want = chain(E, model, ids[:cut])
        assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)
    assert int(model.status) == 0 and q.plm_device_fault() == 0


def test_the_example_runs():
    E = example()
    found, probs, ids, model = E.run(prompt=40, steps=6, samples=6)
    assert found.shape == probs.shape == (6, 7) and bool((found >= 0).all()) and bool((found < E.VOCAB).all())
    assert bool((probs[0] == 1).all())                       # greedy
    assert bool((probs > 0).all()) and bool((probs <= 1).all())
    again, _, _, _ = E.run(prompt=40, steps=6, samples=6)    # the same seed, the same tokens
    assert torch.equal(found, again)


class Step:
    """The calls of a step on tensors of its own, captured into a graph on a stream of its own."""

    def __init__(self, seed, tokens):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        b, heads, kv_heads, d, page, prefix, most = 40, 8, 2, 128, 16, 8192, 8192 + 128
        m, pages, own = b * tokens, 40 * 8 + prefix // page, (most - prefix) // page
        self.x, self.r, w = rand(m, 2048), rand(m, 2048), rand(2048)
        self.h, self.xq = torch.empty_like(self.x), torch.zeros(m * 8 * q.Q8K_BYTES, dtype=torch.uint8, device="cuda")
        pool = torch.zeros(pages, q.plm_kv8_page_bytes(kv_heads, page, d), dtype=torch.uint8, device="cuda")
        pool[:, :2 * kv_heads * page * d] = torch.randint(0, 256, (pages, 2 * kv_heads * page * d), generator=g, device="cuda", dtype=torch.uint8)
        pool[:, 2 * kv_heads * page * d:] = 121   # steps of 2^-6
        self.parts = q.plm_kv8_views(pool, kv_heads, page, d)
        shared = torch.arange(prefix // page, dtype=torch.int32, device="cuda")
        table = torch.cat((shared.expand(b, -1), len(shared) + torch.arange(b * own, dtype=torch.int32, device="cuda").view(b, own)), 1).contiguous()
        lens = torch.full((b,), prefix + 90, dtype=torch.int32, device="cuda")
        positions = (prefix + 90 - tokens + torch.arange(tokens, dtype=torch.int32, device="cuda")).repeat(b)
        slots = (table.long().gather(1, (positions // page).long().view(b, tokens)) * page + (positions % page).view(b, tokens)).reshape(-1)
        k, v, qx = rand(m, kv_heads, d), rand(m, kv_heads, d), rand(m, heads, d).bfloat16()
        self.back, self.o = torch.empty(m, kv_heads, d, device="cuda"), torch.empty(m, heads, d, device="cuda")
        freqs, _ = q.plm_rope_freqs(d, 1e6, device="cuda")
        need = q.plm_attn_kv8_workspace_size(b, tokens, heads, kv_heads, d, prefix, most)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        logits, u, p = rand(b, 32000), torch.rand(b, generator=g, device="cuda"), torch.full((b,), 0.9, device="cuda")
        self.token, self.prob = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, device="cuda")

        def call():
            q.plm_rmsnorm(self.x, w, 1e-6, residual=self.r, sum=self.h, xq=self.xq)
            q.plm_kv8_write([q.plm_kv8_tensor(k, self.parts[0], self.parts[2], slots), q.plm_kv8_tensor(v, self.parts[1], self.parts[3], slots, rotate=False)],
                            positions, freqs, d)
            q.plm_kv8_read([q.plm_kv8_tensor(self.back, self.parts[0], self.parts[2], slots)])
            q.plm_attn_kv8(qx, self.o, *self.parts, table, lens, tokens, prefix, most, d ** -0.5, ws)
            q.plm_sample(logits, self.token, u=u, top_p=p, prob=self.prob)

        self.keep = (pool, w, table, lens, positions, slots, k, v, qx, freqs, ws, logits, u, p)
        self.stream = torch.cuda.Stream()
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            call()
            self.stream.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=self.stream):
                call()

    def results(self):
        return [t.clone() for t in (self.h, self.xq, self.back, self.o, self.token, self.prob)]

    def run(self, times):
        with torch.cuda.stream(self.stream):
            for _ in range(times):
                self.graph.replay()


def test_two_captured_steps_replayed_at_once():
    # with workspaces of their own, neither sees anything of the other
    steps = [Step(1, 4), Step(2, 20)]
    want = []
    for s in steps:
        s.run(1)
        torch.cuda.synchronize()
        want.append(s.results())
    for t in (t for s in steps for t in (s.h, s.back, s.o, s.token, s.prob)):
        t.fill_(-3)
    torch.cuda.synchronize()
    for _ in range(10):
        for s in steps:
            s.run(2)
    torch.cuda.synchronize()
    assert q.plm_device_fault() == 0
    for s, w in zip(steps, want):
        for a, b in zip(s.results(), w):
            assert not a.float().isnan().any() and torch.equal(a, b)
