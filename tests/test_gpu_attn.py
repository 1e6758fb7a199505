"""Attention over a shared prefix and pages on the GPU against the definition in f64.

Tolerance, per output value, with p the exact probabilities, A = sum p |v| and
S = scale sum |q k| <= the largest over the row's keys:
  scores: products exact in f32, a sum of d terms and two roundings: |ds| <=
    (d + 4) 2^-24 S; the exponential's argument and its own error add
    2^-22 (1 + S): dp/p <= e = 2 ((d + 4) 2^-24 + 2^-22) (1 + S)
  p rounded to the cache's type: u = 2^-8 (bf16) or 2^-11 (f16); f16 also loses
    what is below 2^-25 of the row's largest p: n 2^-25 max|v|
  sums of n terms in f32: n 2^-24 relative to A, for sum p and sum p v
  |error| <= (u + e + 2 n 2^-24) A + [f16] n 2^-25 max|v| + half an ulp of o.
lse: e + n 2^-24 + 2^-22 |lse| + 2^-22."""
import math
import random

import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
T = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Case:
    """Pages with NaN wherever nothing may be read; rows in a shuffled table."""

    def __init__(self, lens, nq, hq, hkv, d, prefix, page, dtype, order="heads first", seed=0, extra_rows=2, qscale=1.5, kscale=1.0):
        r, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nq, self.hq, self.hkv, self.d, self.prefix, self.page = lens, nq, hq, hkv, d, prefix, page
        b, shared = len(lens), prefix // page
        width = max(1, max(-(-n // page) for n in lens)) + r.randrange(3)
        count = shared + sum(max(0, -(-n // page) - shared) for n in lens) + 3
        order_ = list(range(count))
        r.shuffle(order_)
        first = [order_.pop() for _ in range(shared)]
        rows = []
        for n in lens:
            k = -(-n // page)
            rows.append((first[:k] + [order_.pop() for _ in range(max(0, k - shared))] + [-1] * width)[:width])
        used = torch.zeros(count, page, dtype=torch.bool)
        for n, row in zip(lens, rows):
            for j in range(n):
                used[row[j // page], j % page] = True
        self.scale = 1.0 / math.sqrt(d)
        shape = (count, 2, hkv, page, d) if order == "heads first" else (count, 2, page, hkv, d)
        pool = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
        self.k, self.v = pool[:, 0], pool[:, 1]
        if order != "heads first":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k.mul_(kscale)
        for x in (self.k, self.v):
            x.transpose(1, 2)[~used.cuda()] = float("nan")
        big = torch.randn(b * nq, hq + 2 * hkv, d, generator=g, device="cuda") * qscale   # q is a part of a product's rows
        self.q = big.to(dtype)[:, :hq]
        # the sequences are rows of a larger table, in another order
        n_rows = b + extra_rows
        self.seq = r.sample(range(n_rows), b)
        table, ls = [[-1] * width for _ in range(n_rows)], [3 * page] * n_rows
        for i, s in enumerate(self.seq):
            table[s], ls[s] = rows[i], lens[i]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.row_lens, self.seqs = torch.tensor(table, **i32), torch.tensor(ls, **i32), torch.tensor(self.seq, **i32)
        self.rows = rows

    def run(self, o_type=None, max_len=None, prefix=None, stream=None):
        n, prefix = self.q.shape[0], self.prefix if prefix is None else prefix
        most = max(1, max(self.lens), prefix) if max_len is None else max_len
        buf = torch.full((n * self.hq * self.d + 64,), float("nan"), dtype=o_type or self.q.dtype, device="cuda")
        buf[-64:] = 7
        o, lse = buf[:-64].view(n, self.hq, self.d), torch.full((n, self.hq), float("nan"), device="cuda")
        size = q.plm_attn_workspace_size(len(self.lens), self.nq, self.hq, self.hkv, self.d, prefix, most)
        ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN if read as f32 before it is written
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        q.plm_attn_shared_prefix(self.q, o, self.k, self.v, self.table, self.row_lens, self.nq, prefix, most, self.scale,
                                 ws[:size], lse=lse, seqs=self.seqs, stream=stream)
        torch.cuda.synchronize()
        assert bool((buf[-64:] == 7).all()) and bool((ws[size:] == 255).all())
        assert q.plm_device_fault() == 0
        return o, lse

    def check(self, o, lse):
        g, u = self.hq // self.hkv, U[self.q.dtype]
        for b, n in enumerate(self.lens):
            pages = [p for p in self.rows[b] if p >= 0]
            take = lambda x: x[pages].transpose(1, 2).reshape(-1, self.hkv, self.d)[:n].double()  # noqa: E731
            k, v = take(self.k), take(self.v)
            rows = slice(b * self.nq, (b + 1) * self.nq)
            x = self.q[rows].double().view(self.nq, self.hkv, g, self.d)
            s = torch.einsum("thgd,nhd->thgn", x, k) * self.scale
            size = (torch.einsum("thgd,nhd->thgn", x.abs(), k.abs()) * self.scale)
            pos = torch.arange(n - self.nq, n, device="cuda")
            hidden = torch.arange(n, device="cuda")[None] > pos[:, None]
            s = s.masked_fill(hidden[:, None, None], -math.inf)
            size = size.masked_fill(hidden[:, None, None], 0.0)
            size = size.amax(-1) if n else torch.zeros(self.nq, self.hkv, g, dtype=torch.float64, device="cuda")
            empty = pos < 0
            p = torch.softmax(s, -1).nan_to_num(0.0) if n else s
            want, A = torch.einsum("thgn,nhd->thgd", p, v), torch.einsum("thgn,nhd->thgd", p, v.abs())
            top = v.abs().amax() if n else 0.0
            e = 2 * ((self.d + 4) * 2.0 ** -24 + 2.0 ** -22) * (1 + size)
            tol = (u + e[..., None] + 2 * n * 2.0 ** -24) * A + 1e-30
            if self.q.dtype == torch.float16:
                tol = tol + n * 2.0 ** -25 * top
            tol = tol + U[o.dtype] * (want.abs() + tol) + (2.0 ** -25 if o.dtype == torch.float16 else 0)
            got = o[rows].double().view(want.shape)
            assert not got.isnan().any()
            err = (got - want).abs()
            assert bool((err <= tol).all()), (b, n, float((err / tol).max()))
            assert bool((got[empty] == 0).all())
            ref = torch.logsumexp(s, -1) if n else s.sum(-1) - math.inf
            got = lse[rows].double().view(ref.shape)
            assert bool((got[empty] == -math.inf).all())
            err = (got - ref).abs()[~empty]
            bound = (e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + ref.abs()))[~empty]
            assert bool((err <= bound).all()), (b, n, float(err.max()))


HEADS = [(16, 8, 128), (14, 2, 64), (8, 8, 64), (32, 8, 128), (5, 1, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,nq,prefix,page", [
    ([1], 1, 0, 16), ([15, 16, 17, 33], 1, 0, 16), ([130, 0, 64, 1, 129, 257], 1, 0, 32),         # no prefix
    ([32, 33, 48, 0, 95, 300], 1, 32, 16), ([640, 641, 705, 1100, 650], 1, 640, 64),              # decode behind one
    ([128, 131, 260, 0, 4], 4, 64, 16), ([700, 513, 512, 600], 5, 512, 32),                       # a few tokens each
    ([64, 40, 10, 100, 0], 1, 64, 16),                                                            # shorter than the prefix
    ([2], 7, 0, 16), ([5, 0, 9], 9, 0, 16),                                                       # more queries than keys
    ([100, 333, 260, 128], 100, 128, 64), ([1000, 640], 333, 512, 128), ([515], 515, 0, 16),      # prompts
])
def test_against_the_definition(hq, hkv, d, dtype, lens, nq, prefix, page):
    c = Case(lens, nq, hq, hkv, d, prefix, page, T[dtype], seed=nq + prefix)
    c.check(*c.run())


@pytest.mark.parametrize("order", ["heads first", "tokens first"])
@pytest.mark.parametrize("nq", [1, 3, 70])
def test_orders_of_the_cache_and_f32_output(order, nq):
    c = Case([257, 300, 512 + nq, 256 + nq], nq, 8, 2, 128, 256, 16, torch.bfloat16, order=order, seed=3)
    o, lse = c.run(o_type=torch.float32)
    c.check(o, lse)


@pytest.mark.parametrize("batch,nq", [(200, 1), (65, 2), (40, 9), (3, 150)])
def test_the_prefix_length_does_not_change_the_result(batch, nq):
    # the same sequences told to share 0, some and all of their common pages
    r = random.Random(batch)
    c = Case([1024 + r.randrange(nq, 200) for _ in range(batch)], nq, 8, 2, 128, 1024, 16, torch.bfloat16, seed=batch)
    for prefix in (0, 16, 496, 1024):
        c.check(*c.run(prefix=prefix))


@pytest.mark.parametrize("nq", [1, 4, 64])
def test_long_rows_and_loose_bounds(nq):
    c = Case([20000, 17, 9000, 20000 - 3], nq, 4, 2, 128, 0, 64, torch.bfloat16, seed=8)
    c.check(*c.run())
    c.check(*c.run(max_len=90000))     # a bound far above the lengths (the rows of the table end first)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nq,prefix", [(1, 4096), (1, 0), (130, 4096), (130, 0)])
def test_sharp_and_rising_scores(dtype, nq, prefix):
    # scores of +-60: one key takes all; later keys score higher, so the running maximum moves again and again
    c = Case([4096 + nq + 70, 4096 + nq + 1], nq, 4, 2, 64, prefix, 16, T[dtype], seed=4, qscale=6.0, kscale=2.0)
    c.check(*c.run())
    ramp = torch.linspace(0.05, 3.0, c.k.shape[0], device="cuda").to(c.k.dtype)
    c.k.mul_(ramp[:, None, None, None])
    c.check(*c.run())


@pytest.mark.parametrize("nq,prefix", [(1, 0), (1, 512), (40, 512), (130, 0), (130, 512)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scales_of_zero_and_below(dtype, nq, prefix):
    c = Case([600 + nq, 516 + nq, 130, 0], nq, 8, 2, 64, prefix, 16, T[dtype], seed=11)
    scale, c.scale = c.scale, 0.0      # the mean of the values
    c.check(*c.run())
    c.scale = -scale                   # as the opposite queries under the opposite scale
    o, lse = c.run()
    c.q.neg_()
    c.scale = scale
    c.check(o, lse)


@pytest.mark.parametrize("hidden", [100, 128, 300])
def test_prompts_with_scores_of_minus_infinity(hidden):
    # the first keys score -inf for positive queries, as if they were not there
    nq, n = 130, 400
    c = Case([n], nq, 2, 1, 128, 0, 16, torch.bfloat16, seed=6)
    c.q.copy_(c.q.abs() + 0.1)
    whole = Case([n], nq, 2, 1, 128, 0, 16, torch.bfloat16, seed=6)
    for j in range(hidden):
        c.k[c.rows[0][j // 16], :, j % 16] = -math.inf
    o, lse = c.run()
    pages = c.rows[0][:n // 16]
    take = lambda x: x[pages].transpose(1, 2).reshape(-1, 128)[:n].double()  # noqa: E731
    k, v, x = take(whole.k)[hidden:], take(c.v)[hidden:], c.q.double()
    s, size = x @ k.T * c.scale, x.abs() @ k.abs().T * c.scale
    seen = torch.arange(hidden, n, device="cuda")[None] <= torch.arange(n - nq, n, device="cuda")[:, None]
    s, size = s.masked_fill(~seen[:, None], -math.inf), size.masked_fill(~seen[:, None], 0.0).amax(-1)
    some = seen.any(-1)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    want, A = p @ v, p @ v.abs()
    e = 2 * ((128 + 4) * 2.0 ** -24 + 2.0 ** -22) * (1 + size)
    tol = (2.0 ** -8 + e[..., None] + 2 * n * 2.0 ** -24) * A + 1e-30
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((o.double() - want).abs() <= tol).all())
    assert bool((o[~some] == 0).all()) and bool((lse[~some] == -math.inf).all())
    ref = torch.logsumexp(s, -1)[some]
    assert bool(((lse.double()[some] - ref).abs() <= e[some] + n * 2.0 ** -24 + 2.0 ** -22 * (1 + ref.abs())).all())


def test_scores_of_minus_infinity():
    # keys of -inf score -inf for positive queries: as if hidden; a row of nothing else is empty
    c = Case([40, 20], 1, 2, 1, 64, 0, 16, torch.bfloat16, seed=5)
    c.q.copy_(c.q.abs() + 0.1)
    for j in range(10, 40):
        c.k[c.rows[0][j // 16], :, j % 16] = -math.inf
    for j in range(20):
        c.k[c.rows[1][j // 16], :, j % 16] = -math.inf
    o, lse = c.run()
    assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    c.lens, c.row_lens = [10, 0], None
    c.check(o, lse)


def test_pages_out_of_range_read_as_zeros():
    c = Case([64, 64], 1, 4, 2, 128, 0, 16, torch.bfloat16, seed=6)
    good, _ = c.run()
    page = c.rows[1][2]
    c.k[page], c.v[page] = 0, 0
    want, wl = c.run()
    for bad in (-1, -2 ** 31, c.k.shape[0], 2 ** 31 - 1):
        c.table[c.seq[1], 2] = bad
        o, lse = c.run()
        assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(o[0], good[0])


def test_sequences_out_of_range_have_no_keys():
    c = Case([64, 64, 64], 1, 4, 2, 128, 0, 16, torch.bfloat16, seed=6)
    for bad in (-1, 99, 2 ** 31 - 1):
        c.seqs[1] = bad
        o, lse = c.run()
        assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all()) and not o.isnan().any()


def test_lengths_are_cut_to_the_bound_and_the_row():
    c = Case([64, 48], 1, 4, 2, 128, 0, 16, torch.bfloat16, seed=7)
    short, sl = c.run(max_len=48)
    c.lens[0] = 48
    c.check(short, sl)
    c.row_lens[c.seq[1]] = 10 ** 9
    c.row_lens[c.seq[0]] = -5
    o, lse = c.run(max_len=48)
    assert torch.equal(o[1], short[1]) and bool((o[0] == 0).all()) and bool((lse[0] == -math.inf).all())


def test_offsets_past_32_bits():
    # the pages in use are the last of a pool of more than 2^32 elements
    hkv, page, d = 8, 64, 128
    pages = (1 << 32) // (hkv * page * d) + 30
    pool = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    for nq, n, prefix in ((1, 700, 512), (90, 700, 512), (1, 300, 0)):
        c = Case([n, n], nq, 16, hkv, d, prefix, page, torch.bfloat16, seed=9)
        shift = pages - c.k.shape[0]
        k, v = pool.clone(), pool
        k[shift:], v[shift:] = c.k, c.v
        want, wl = c.run()
        c.k, c.v, c.rows = k, v, None
        c.table = torch.where(c.table >= 0, c.table + shift, c.table)
        o, lse = c.run()
        assert torch.equal(o, want) and torch.equal(lse, wl)
        del k


def test_the_same_bits_every_time_and_on_another_stream():
    for nq, batch in ((1, 33), (4, 20), (80, 3)):
        r = random.Random(nq)
        c = Case([2048 + r.randrange(nq, 900) for _ in range(batch)], nq, 16, 4, 128, 2048, 16, torch.bfloat16, seed=nq)
        o, lse = c.run()
        for stream in (None, torch.cuda.Stream()):
            o2, l2 = c.run(stream=stream)
            assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_in_a_graph_with_new_lengths():
    # the launches do not depend on the lengths: a captured call serves a growing batch
    c = Case([512 + 60, 512 + 90, 512 + 3], 1, 8, 2, 128, 512, 16, torch.bfloat16, seed=11)
    final, most = list(c.lens), 640
    o, lse = torch.empty_like(c.q, memory_format=torch.contiguous_format), torch.empty(3, 8, device="cuda")
    ws = torch.empty(q.plm_attn_workspace_size(3, 1, 8, 2, 128, 512, most), dtype=torch.uint8, device="cuda")
    call = lambda: q.plm_attn_shared_prefix(c.q, o, c.k, c.v, c.table, c.row_lens, 1, 512, most, c.scale, ws, lse=lse, seqs=c.seqs)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([520, 513, 515], [530, 0, 512], final):
        c.lens = lens
        for s, n in zip(c.seq, lens):
            c.row_lens[s] = n
        graph.replay()
        torch.cuda.synchronize()
        c.check(o, lse)


def test_binding_refuses():
    c = Case([64, 64], 1, 4, 2, 128, 0, 16, torch.bfloat16)
    o, ws = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    ok = dict(q=c.q, o=o, k=c.k, v=c.v, table=c.table, lens=c.row_lens, tokens=1, prefix_len=0, max_len=64, scale=0.1, workspace=ws)
    q.plm_attn_shared_prefix(**ok)
    for bad in (dict(o=o[:1]), dict(q=c.q.half()), dict(v=c.v.half()), dict(v=c.v[:, :1]), dict(v=c.v.contiguous()), dict(table=c.table.long()),
                dict(lens=c.row_lens[:1]), dict(tokens=3), dict(tokens=0), dict(lse=o), dict(seqs=c.seqs[:1]), dict(q=c.q[..., :64])):
        with pytest.raises(ValueError):
            q.plm_attn_shared_prefix(**{**ok, **bad})
    for bad in (dict(prefix_len=8), dict(max_len=0), dict(prefix_len=128)):
        with pytest.raises(q.PlmError):
            q.plm_attn_shared_prefix(**{**ok, **bad})
