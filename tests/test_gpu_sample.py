"""The sampler on the GPU against its definition in f64, row by row.

Tokens have to be equal.  A weight is off by 2^-29 of itself, or 2^-40 of the largest, at most, a sum of n by n 2^-40 of the
largest besides.  So a token may differ only where u, top_p or min_p lies within that of a border: 1e-8 of the sum for the
rows here.  For such a row (none is expected among the seeds used, and the reference says if one is) the neighbour is right too.
prob is a quotient of a weight and such a sum, rounded once: 2^-28 + 2^-24 of itself, and n 2^-40 where it is small.  A small
weight's own bits below 2^-40 are not lost in it."""
import math

import numpy as np
import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEAR = 1e-8


def define(x, u, t, k, p, low):
    """(token, probability, whether a border is nearer than NEAR) of one row (numpy, f64)."""
    x = np.where(np.isnan(x), -math.inf, x.astype(np.float64))
    if x.max() == -math.inf:
        return -1, 0.0, False
    if not t > 0 or u is None:
        return int(np.argmax(x)), 1.0, False
    order = np.argsort(-x, kind="stable")
    z = np.zeros_like(x) if math.isinf(x.max()) else (x - x.max()) / t
    w = np.where(x == x.max(), 1.0, 0.0 if math.isinf(x.max()) else np.exp(np.maximum(z, -800)))
    w[x == -math.inf] = 0.0
    w[w < 2.0 ** -40] = 0.0
    order = order[w[order] > 0]
    if k > 0:
        order = order[:k]
    close = False
    if p < 1:
        mass = np.cumsum(w[order])
        before, target = mass - w[order], max(p, 0.0) * mass[-1]
        keep = before < target
        keep[0] = True
        close |= bool((np.abs(before[1:] - target) < NEAR * mass[-1]).any())
        order = order[keep]
    if low > 0:
        close |= bool((np.abs(w[order] / min(low, 1.0) - 1) < NEAR).any() and low < 1)
        order = order[w[order] >= min(low, 1.0) * (1 - 1e-12)]
    order = np.sort(order)
    mass = np.cumsum(w[order])
    target = min(max(0.0 if math.isnan(u) else u, 0.0), 1.0) * mass[-1]
    close |= bool((np.abs(mass[:-1] - target) < NEAR * mass[-1]).any())
    i = min(int((mass <= target).sum()), len(order) - 1)
    while w[order[i]] == 0:
        i -= 1
    return int(order[i]), float(w[order[i]] / mass[-1]), close


class Rows:
    def __init__(self, x, seed=0, dtype=torch.float32, **params):
        """x [m][n] on the GPU or as numpy; params: temperature, top_k, top_p, min_p, u as a number, a list or None."""
        x = torch.as_tensor(np.asarray(x.cpu() if isinstance(x, torch.Tensor) else x)).cuda().to(dtype)
        m, n = x.shape
        buf = torch.full((m, n + 5), 100.0, dtype=dtype, device="cuda")   # rows apart: what lies between would win
        buf[:, :n] = x
        self.x = buf[:, :n]
        self.m, self.n = m, n
        g = np.random.RandomState(seed)
        self.p = {"u": g.rand(m).astype(np.float32)}
        for name, v in params.items():
            kind = np.int32 if name == "top_k" else np.float32
            self.p[name] = None if v is None else np.broadcast_to(np.asarray(v, kind), (m,)).copy()

    def run(self, stream=None, prob=True):
        dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in self.p.items()}
        out = torch.full((self.m + 2,), -9, dtype=torch.int32, device="cuda")
        pr = torch.full((self.m + 2,), -9.0, device="cuda") if prob else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        q.plm_sample(self.x, out[1:-1], prob=pr[1:-1] if prob else None, stream=stream, **dev)
        torch.cuda.synchronize()
        assert out[0] == -9 and out[-1] == -9 and (not prob or (pr[0] == -9 and pr[-1] == -9))
        return out[1:-1].cpu().numpy(), pr[1:-1].cpu().numpy() if prob else None

    def check(self, got=None):
        tokens, prob = got or self.run()
        x, near = self.x.float().cpu().numpy(), 0
        at = lambda name, i, off: off if self.p.get(name) is None else self.p[name][i].item()  # noqa: E731
        for i in range(self.m):
            t, p, close = define(x[i], at("u", i, None), at("temperature", i, 1.0), at("top_k", i, 0), at("top_p", i, 1.0), at("min_p", i, 0.0))
            near += close
            if close:
                continue
            assert tokens[i] == t, (i, tokens[i], t, {k: None if v is None else v[i] for k, v in self.p.items()})
            assert abs(float(prob[i]) - p) <= (2.0 ** -28 + 2.0 ** -24) * p + self.n * 2.0 ** -40, (i, prob[i], p)
        assert near <= self.m // 50, near


def normal(seed, m, n, spread=3.0):
    return spread * np.random.RandomState(seed).randn(m, n).astype(np.float32)


SIZES = [(1, 1), (3, 2), (5, 31), (40, 32), (33, 1000), (7, 4097), (300, 513), (2, 32000), (5, 40001), (1, 151936), (160, 5000)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("params", [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=20), dict(top_p=0.9, temperature=0.8), dict(min_p=0.05),
                                    dict(temperature=1.3, top_k=200, top_p=0.95, min_p=0.02), dict(temperature=0.0), dict(u=None)])
def test_against_the_definition(m, n, params):
    Rows(normal(n, m, n), seed=m, **params).check()


@pytest.mark.parametrize("spread", [0.0, 1e-6, 0.3, 10.0])
@pytest.mark.parametrize("params", [dict(top_k=37), dict(top_p=0.5), dict(top_p=0.97), dict(top_k=3000, top_p=0.7), dict(min_p=0.5)])
def test_flat_and_peaked_rows(spread, params):
    Rows(normal(5, 6, 20011, spread), **params).check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("params", [dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=300, top_p=0.8, min_p=0.01), dict(temperature=0.0)])
def test_16_bit_logits_have_many_ties(dtype, params):
    Rows(normal(2, 30, 9000, 1.0), dtype=T[dtype], **params).check()


def test_probability_of_a_small_weight_keeps_its_bits():
    # One token of weight 1 and one of 2^-32 or so, which u = 1 takes.  The weight is off by 2^-29 of itself, the sum, 1 + 2^-32,
    # by 2^-29 too (the large one is exact but for 2^-40), and the quotient is rounded once: 2^-24 + 2^-28
    for z in (-10.0, -17.3, -22.1803, -25.0, -27.5):
        r = Rows(np.array([[0.0, z, -math.inf]] * 2, np.float32), u=1.0)
        tokens, prob = r.run()
        want = math.exp(float(np.float32(z))) / (1 + math.exp(float(np.float32(z))))
        assert tokens.tolist() == [1, 1]
        assert abs(float(prob[0]) - want) <= (2.0 ** -24 + 2.0 ** -28) * want, (z, prob[0], want)


def test_ties_go_to_the_lowest_index():
    x = np.full((8, 3000), -5.0, np.float32)
    x[:, 1000:1900:3] = 2.0    # 300 equal ones
    x[:, 2500] = 2.5
    for params in (dict(top_k=1), dict(top_k=2), dict(top_k=101), dict(top_k=301), dict(top_k=302), dict(top_p=0.5), dict(top_p=0.999),
                   dict(top_k=200, top_p=0.5)):
        r = Rows(x, u=np.linspace(0, 0.999, 8), **params)
        r.check()
    assert Rows(x, temperature=0.0).run()[0].tolist() == [2500] * 8
    x[:, 2500] = 2.0
    tokens, prob = Rows(x, temperature=0.0).run()
    assert tokens.tolist() == [1000] * 8 and prob.tolist() == [1.0] * 8
    assert Rows(x, top_k=1).run()[0].tolist() == [1000] * 8
    signed = np.zeros((2, 100), np.float32)
    signed[:, ::2] = -0.0      # equal to 0
    assert Rows(signed, top_k=1).run()[0].tolist() == [0, 0]
    # two equal ones, half of the sum before the second
    assert set(Rows(np.zeros((64, 2)), top_p=0.5).run()[0].tolist()) == {0}


def test_rows_with_infinities_and_nan():
    inf, nan = math.inf, math.nan
    x = normal(1, 9, 500)
    x[0] = -inf
    x[1] = nan
    x[2, :499] = -inf
    x[3, 7], x[3, 400] = inf, inf
    x[4, ::2] = nan
    x[5, ::3] = -inf
    x[6, 0] = nan
    x[7, 3], x[7, 9] = inf, nan
    x[8] = -3e38
    x[8, 77] = 3e38
    for params in (dict(), dict(temperature=0.0), dict(top_k=3), dict(top_p=0.8), dict(min_p=0.2), dict(top_k=100, top_p=0.9, min_p=0.01, temperature=2.0)):
        r = Rows(x, **params)
        got = r.run()
        r.check(got)
        assert got[0][0] == got[0][1] == -1 and got[1][0] == got[1][1] == 0 and got[0][2] == 499 and got[0][3] in (7, 400) and got[0][7] == 3


def test_parameters_at_their_ends():
    x = normal(3, 1, 3001)
    nan, inf = math.nan, math.inf
    settings = [dict(temperature=t) for t in (1e-30, 1e-38, 1e-3, 1e3, 1e30, inf, -1.0, nan)]
    settings += [dict(top_k=k) for k in (-1, 0, 3000, 3001, 2 ** 31 - 1)]
    settings += [dict(top_p=p) for p in (0.0, -1.0, 1e-30, 1.0, 2.0, nan, 1 - 2 ** -24)]
    settings += [dict(min_p=p) for p in (-1.0, 1e-30, 1.0, 5.0, nan, 1e-12)]
    settings += [dict(u=u) for u in (0.0, 1.0, -3.0, 7.0, nan, 1 - 2 ** -24)]
    settings += [dict(u=1.0, top_p=0.9), dict(u=0.0, top_k=5), dict(u=1.0, min_p=0.3)]
    for s in settings:
        if s.get("top_p") == 1 - 2 ** -24:   # what is left is below what f64 sums of another order tell apart
            Rows(x, **s).run()
            continue
        Rows(x, seed=7, **s).check()


def test_weights_that_the_bins_bounds_tell_apart_badly():
    # one value holds nearly all the sum, the border lies far below it among many small ones
    n = 20000
    x = np.full((4, n), 0.0, np.float32)
    x[:, 5] = 9.0
    x[:, 100:] = np.linspace(-1, -0.99, n - 100)
    for p in (0.3, 0.301, 0.5, 0.9999):
        Rows(x, top_p=p).check()
    x = np.zeros((4, n), np.float32)          # 10000 equal ones, and as many an ulp or so beside them
    x[:, ::2] = 1.0 + np.arange(n // 2, dtype=np.float32) * 2.0 ** -23
    for p in (0.2, 0.5, 0.73, 0.7313, 0.9):
        Rows(x, top_p=p).check()
    for k in (1, 2, 9999, 10000, 10001, 15000):
        Rows(x, top_k=k).check()


@pytest.mark.parametrize("n", [500001, 1 << 20, 1 << 22])
def test_rows_too_long_for_shared_memory(n):
    x = (2 * torch.randn(2, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    x[:, n - 3] = 12.0
    for params in (dict(top_k=10), dict(top_p=0.6), dict(temperature=0.0), dict(min_p=0.01)):
        Rows(x, **params).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_that_fit_shared_memory_in_part(dtype):
    # more CTAs than SMs: two share one, and a row's rest stays in L2
    m, n = 24, 200063
    x = normal(12, m, n, 2.5)
    Rows(x, dtype=T[dtype], top_p=np.repeat([0.9, 1.0, 0.5], 8), top_k=np.tile([0, 0, 50, 1000], 6), min_p=np.tile([0.0, 0.1], 12),
         temperature=np.linspace(0.0, 1.5, m)).check()


def test_each_row_has_its_own_parameters():
    m, n = 240, 6007
    g = np.random.RandomState(4)
    r = Rows(normal(9, m, n, 2.0), temperature=g.choice([0.0, 0.5, 0.7, 1.0, 1.5], m), top_k=g.choice([0, 1, 5, 40, 2000], m),
             top_p=g.choice([1.0, 0.3, 0.9, 0.99], m), min_p=g.choice([0.0, 0.05, 0.3], m))
    got = r.run()
    r.check(got)
    one = Rows(r.x[17:18].clone(), **{k: v[17:18] for k, v in r.p.items()}).run()   # a row does not depend on the others
    assert one[0][0] == got[0][17] and one[1][0] == got[1][17]


def test_every_token_is_met_as_often_as_it_should_be():
    m, n = 5000, 50
    x = np.repeat(normal(4, 1, n, 1.5), m, 0)
    tokens, prob = Rows(x, u=((np.arange(m) + 0.5) / m), top_p=0.95, temperature=0.9).run()
    assert (np.diff(tokens) >= 0).all()                      # in the order of the indices
    for t in np.unique(tokens):
        here = tokens == t
        assert abs(here.sum() - m * prob[here][0]) <= 1.01   # u in even steps
    assert abs(prob[np.unique(tokens, return_index=True)[1]].sum() - 1) < 1e-6


def test_streams_graphs_and_no_probabilities():
    x = normal(6, 20, 30011)
    r = Rows(x, top_p=0.9, temperature=0.8)
    want = r.run()
    got = r.run(stream=torch.cuda.Stream(), prob=False)
    assert (got[0] == want[0]).all()
    u, t = torch.from_numpy(r.p["u"]).cuda(), torch.full((20,), 0.8, device="cuda")
    p, out, prob = torch.full((20,), 0.9, device="cuda"), torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(20, device="cuda")
    call = lambda: q.plm_sample(r.x, out, u=u, temperature=t, top_p=p, prob=prob)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for seed in (1, 2):
        r.p["u"] = np.random.RandomState(seed).rand(20).astype(np.float32)
        u.copy_(torch.from_numpy(r.p["u"]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        r.check((out.cpu().numpy(), prob.cpu().numpy()))
    q.plm_sample(r.x[:0], out[:0], u=u[:0])
