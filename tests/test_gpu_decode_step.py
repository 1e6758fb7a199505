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
