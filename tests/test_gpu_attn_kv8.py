"""Attention over 8-bit pages on the GPU against the definition in f64, on the values that the pages stand for.

The cases, their poisoned pages and the terms of the tolerance are those of the 16-bit pages (test_gpu_attn): a code times
its power of two is exact in bf16 and here in f16 (steps of 2^-14 and more), so both operands of the first product are
exact.  Few rows have their second product in f16 whatever the type.  There
  p is held as 2^7 .. 2^15 times what it is relative to the row's largest, so what f16 loses below its steps of 2^-24 is
    2^-25 / 2^7 = 2^-32 of the largest p at most, n of them: n 2^-32 max|v|;
  a value is held relative to the largest power of two 2^j of its 32 dims so far, to 2^-24 of it: a block of steps of 2^(j - 25)
    or less may be lost, 127 2^(j - 25) a value, where a code of 2^j is 64 at least: 2^-24 max|v|, as sum p = 1.
Both are added to the bound.  Where nothing may be read the codes are arbitrary and the exponents 255, which would give
infinite values."""
import math
import random

import pytest
import torch

import quant_packed_gemv_gb300 as q
from tests import test_gpu_attn

pytestmark = pytest.mark.gpu
T = test_gpu_attn.T


def encode(x):
    """Codes and exponents of x [..][d], whose values are 0 or normal; NaN counts as 0."""
    x = x.float().nan_to_num(0.0)
    b = x.reshape(*x.shape[:-1], -1, 32)
    m, k = torch.frexp(b.abs().amax(-1))       # m 2^k, m in 1/2 .. 1
    j = k - 7 + (m * 128 >= 127.5).int()
    codes = torch.round(b * torch.exp2(-j.float())[..., None])
    return codes.reshape(x.shape).to(torch.int8), torch.where(m == 0, 0, j + 127).to(torch.uint8)


def decode(codes, exps):
    return (codes.float().reshape(*exps.shape, 32) * torch.where(exps == 0, 0.0, torch.exp2(exps.float() - 127))[..., None]).reshape(codes.shape)


class Case8(test_gpu_attn.Case):
    """The same case over 8-bit pages: k and v are the values that they stand for."""

    def __init__(self, *args, order="heads first", loud=1.0, **kw):
        super().__init__(*args, order=order, **kw)
        pages, hkv, page, d = self.k.shape
        if loud != 1.0:   # blocks of very different sizes
            g = torch.Generator(device="cuda").manual_seed(3)
            for x in (self.k, self.v):
                x.copy_((x.float().view(pages, hkv, page, -1, 32) * torch.exp2(torch.randint(-5, 5, (pages, hkv, page, d // 32, 1), generator=g, device="cuda") *
                                                                               math.log2(loud))).view(x.shape).to(x.dtype))
        self.order = order
        if order == "heads first":
            self.pool = torch.empty(pages, q.plm_kv8_page_bytes(hkv, page, d), dtype=torch.uint8, device="cuda")
            self.parts = q.plm_kv8_views(self.pool, hkv, page, d)
        else:
            self.pool = torch.empty(pages, 2, page, hkv, d, dtype=torch.int8, device="cuda")
            exps = torch.empty(2, pages, hkv, page, d // 32, dtype=torch.uint8, device="cuda")
            self.parts = (self.pool[:, 0].transpose(1, 2), self.pool[:, 1].transpose(1, 2), exps[0], exps[1])
        self.encode()

    def encode(self):
        """The pages from k and v, which become what the pages stand for."""
        for x, codes, exps in ((self.k, self.parts[0], self.parts[2]), (self.v, self.parts[1], self.parts[3])):
            unused = x.isnan().any(-1)
            c, e = encode(x)
            values = decode(c, e)
            assert torch.equal(values.to(x.dtype).float(), values)   # exact in the cache's type
            c[unused], e[unused] = 77, 255
            codes.copy_(c)
            exps.copy_(e)
            x.copy_(values.masked_fill(unused[..., None], float("nan")))

    def check(self, o, lse):
        g, u = self.hq // self.hkv, test_gpu_attn.U[self.q.dtype]
        for b, n in enumerate(self.lens):
            pages = [p for p in self.rows[b] if p >= 0]
            k, v = (x[pages].transpose(1, 2).reshape(-1, self.hkv, self.d)[:n].double() for x in (self.k, self.v))
            rows = slice(b * self.nq, (b + 1) * self.nq)
            x = self.q[rows].double().view(self.nq, self.hkv, g, self.d)
            pos = torch.arange(n - self.nq, n, device="cuda")
            hidden = (torch.arange(n, device="cuda")[None] > pos[:, None])[:, None, None]
            s = (torch.einsum("thgd,nhd->thgn", x, k) * self.scale).masked_fill(hidden, -math.inf)
            size = (torch.einsum("thgd,nhd->thgn", x.abs(), k.abs()) * abs(self.scale)).masked_fill(hidden, 0.0)
            size = size.amax(-1) if n else torch.zeros(self.nq, self.hkv, g, dtype=torch.float64, device="cuda")
            empty = pos < 0
            p = torch.softmax(s, -1).nan_to_num(0.0) if n else s
            want, A = torch.einsum("thgn,nhd->thgd", p, v), torch.einsum("thgn,nhd->thgd", p, v.abs())
            top = float(v.abs().amax()) if n else 0.0
            e = 2 * ((self.d + 4) * 2.0 ** -24 + 2.0 ** -22) * (1 + size)
            tol = (u + e[..., None] + 2 * n * 2.0 ** -24) * A + 1e-30 + (n * 2.0 ** -32 + 2.0 ** -24) * top
            if self.q.dtype == torch.float16:
                tol = tol + n * 2.0 ** -25 * top
            tol = tol + test_gpu_attn.U[o.dtype] * (want.abs() + tol) + (2.0 ** -25 if o.dtype == torch.float16 else 0)
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

    def size(self, prefix, most):
        return q.plm_attn_kv8_workspace_size(len(self.lens), self.nq, self.hq, self.hkv, self.d, prefix, most)

    def run(self, o_type=None, max_len=None, prefix=None, stream=None):
        n, prefix = self.q.shape[0], self.prefix if prefix is None else prefix
        most = max(1, max(self.lens), prefix) if max_len is None else max_len
        buf = torch.full((n * self.hq * self.d + 64,), float("nan"), dtype=o_type or self.q.dtype, device="cuda")
        buf[-64:] = 7
        o, lse = buf[:-64].view(n, self.hq, self.d), torch.full((n, self.hq), float("nan"), device="cuda")
        size = self.size(prefix, most)
        ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN if read before it is written
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        q.plm_attn_kv8(self.q, o, *self.parts, self.table, self.row_lens, self.nq, prefix, most, self.scale, ws[:size], lse=lse, seqs=self.seqs,
                       stream=stream)
        torch.cuda.synchronize()
        assert bool((buf[-64:] == 7).all()) and bool((ws[size:] == 255).all())
        assert q.plm_device_fault() == 0
        return o, lse


@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (14, 2, 64), (8, 8, 64), (32, 8, 128), (5, 1, 128)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,nq,prefix,page", [
    ([1], 1, 0, 16), ([15, 16, 17, 33], 1, 0, 16), ([130, 0, 64, 1, 129, 257], 1, 0, 32),         # no prefix
    ([32, 33, 48, 0, 95, 300], 1, 32, 16), ([640, 641, 705, 1100, 650], 1, 640, 64),              # decode behind one
    ([128, 131, 260, 0, 4], 4, 64, 16), ([700, 513, 512, 600], 5, 512, 32),                       # a few tokens each
    ([64, 40, 10, 100, 0], 1, 64, 16),                                                            # shorter than the prefix
    ([2], 7, 0, 16), ([5, 0, 9], 9, 0, 16), ([60, 41], 20, 32, 16),                               # more queries than keys
    ([100, 333, 260, 128], 100, 128, 64), ([1000, 640, 20], 333, 512, 128), ([515], 515, 0, 16),  # prompts
])
def test_against_the_definition(hq, hkv, d, dtype, lens, nq, prefix, page):
    c = Case8(lens, nq, hq, hkv, d, prefix, page, T[dtype], seed=nq + prefix)
    c.check(*c.run())


@pytest.mark.parametrize("order", ["heads first", "tokens first"])
@pytest.mark.parametrize("nq", [1, 3, 30, 70])
def test_orders_of_the_cache_f32_output_and_unequal_blocks(order, nq):
    c = Case8([257, 300, 512 + nq, 256 + nq], nq, 8, 2, 128, 256, 16, torch.bfloat16, order=order, seed=3, loud=2.0)
    c.check(*c.run(o_type=torch.float32))


# what the workspace size says a call does: nothing apart, the prefix, everything read back
@pytest.mark.parametrize("batch,nq,prefix,d,dtype", [(64, 1, 4096, 128, "bf16"), (40, 5, 4080, 64, "f16"), (30, 9, 2032, 128, "bf16"), (24, 20, 3088, 64, "bf16")])
def test_the_prefix_apart(batch, nq, prefix, d, dtype):
    r = random.Random(batch)
    lens = [prefix + r.randrange(nq, 200) for _ in range(batch)]
    lens[3], lens[7], lens[0] = 0, prefix + nq - 2, 5   # idle, and too short to share it
    c = Case8(lens, nq, 8, 2, d, prefix, 16, T[dtype], seed=batch)
    # a prefix that every one of 2000 such streams reads is done apart
    if c.size(prefix, max(lens)) > 0:
        c.check(*c.run())
    for part in (0, 16, prefix // 32 * 16):   # the same sequences told to share less
        c.check(*c.run(prefix=part))


def test_which_calls_read_back():
    size = q.plm_attn_kv8_workspace_size
    assert size(4, 1, 16, 8, 128, 0, 5000) == 0 and size(100, 8, 32, 8, 128, 0, 5000) == 0
    assert size(256, 1, 32, 8, 128, 32768, 34000) > 2 * 32768 * 8 * 128 * 2    # the prefix
    assert size(8, 509, 32, 8, 128, 0, 17000) > 8 * 2 * 17000 * 8 * 128 * 2    # all


@pytest.mark.parametrize("batch,nq", [(3, 150), (5, 60)])
def test_the_prefix_length_does_not_change_the_result(batch, nq):
    r = random.Random(batch)
    c = Case8([1024 + r.randrange(nq, 200) for _ in range(batch)] + [300], nq, 8, 2, 128, 1024, 16, torch.bfloat16, seed=batch)
    for prefix in (0, 16, 496, 1024):
        c.check(*c.run(prefix=prefix))


@pytest.mark.parametrize("nq", [1, 4, 64])
def test_long_rows_and_loose_bounds(nq):
    c = Case8([20000, 17, 9000, 20000 - 3], nq, 4, 2, 128, 0, 64, torch.bfloat16, seed=8)
    c.check(*c.run())
    c.check(*c.run(max_len=90000))     # a bound far above the lengths (the rows of the table end first)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nq,prefix", [(1, 4096), (1, 0), (130, 4096), (130, 0)])
def test_sharp_and_rising_scores(dtype, nq, prefix):
    c = Case8([4096 + nq + 70, 4096 + nq + 1], nq, 4, 2, 64, prefix, 16, T[dtype], seed=4, qscale=6.0, kscale=2.0)
    c.check(*c.run())
    c.k.mul_(torch.linspace(0.05, 3.0, c.k.shape[0], device="cuda").to(c.k.dtype)[:, None, None, None])
    c.encode()
    c.check(*c.run())


@pytest.mark.parametrize("nq,prefix", [(1, 0), (1, 512), (40, 512), (130, 0)])
def test_scales_of_zero_and_below(nq, prefix):
    c = Case8([600 + nq, 516 + nq, 130, 0], nq, 8, 2, 64, prefix, 16, torch.bfloat16, seed=11)
    scale, c.scale = c.scale, 0.0      # the mean of the values
    c.check(*c.run())
    c.scale = -scale                   # as the opposite queries under the opposite scale
    o, lse = c.run()
    c.q.neg_()
    c.scale = scale
    c.check(o, lse)


def test_exponents_at_their_ends():
    # blocks of zeros, of 2^-100 steps and of huge values in bf16; none of them costs the others anything
    c = Case8([40, 33], 1, 4, 2, 128, 0, 16, torch.bfloat16, seed=2)
    first = c.rows[0][0]
    c.v[first, :, 3, :32] = 0.0
    c.k[first, :, 4, 32:64] = 0.0
    c.v[first, :, 5, 64:96] *= 2.0 ** -90
    c.k[first, :, 6, :32] *= 2.0 ** -90
    c.v[first, :, 7, 96:] *= 2.0 ** 60
    c.encode()
    c.check(*c.run())


def test_pages_out_of_range_read_as_zeros():
    for nq in (1, 60):
        c = Case8([80, 80], nq, 4, 2, 128, 0, 16, torch.bfloat16, seed=6)
        good, _ = c.run()
        page = c.rows[1][2]
        for x in c.parts:
            x[page] = 0
        want, wl = c.run()
        for bad in (-1, -2 ** 31, c.k.shape[0], 2 ** 31 - 1):
            c.table[c.seq[1], 2] = bad
            o, lse = c.run()
            assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(o[:nq], good[:nq])


def test_sequences_out_of_range_have_no_keys():
    for nq in (1, 60):
        c = Case8([64, 64, 64], nq, 4, 2, 128, 0, 16, torch.bfloat16, seed=6)
        for bad in (-1, 99, 2 ** 31 - 1):
            c.seqs[1] = bad
            o, lse = c.run()
            assert bool((o[nq:2 * nq] == 0).all()) and bool((lse[nq:2 * nq] == -math.inf).all()) and not o.isnan().any()


def test_lengths_are_cut_to_the_bound_and_the_row():
    for nq in (1, 60):
        c = Case8([64, 48], nq, 4, 2, 128, 0, 16, torch.bfloat16, seed=7)
        short, sl = c.run(max_len=48)
        c.lens[0] = 48
        c.check(short, sl)
        c.row_lens[c.seq[1]] = 10 ** 9
        c.row_lens[c.seq[0]] = -5
        o, lse = c.run(max_len=48)
        assert torch.equal(o[nq:], short[nq:]) and bool((o[:nq] == 0).all()) and bool((lse[:nq] == -math.inf).all())


def test_offsets_past_32_bits():
    hkv, page, d = 8, 64, 128
    size = q.plm_kv8_page_bytes(hkv, page, d)
    pages = (1 << 32) // size + 30
    pool = torch.empty(pages, size, dtype=torch.uint8, device="cuda")
    for nq, n, prefix in ((1, 700, 512), (90, 700, 512), (1, 300, 0)):
        c = Case8([n, n], nq, 16, hkv, d, prefix, page, torch.bfloat16, seed=9)
        shift = pages - c.k.shape[0]
        pool[shift:] = c.pool
        want, wl = c.run()
        c.parts = q.plm_kv8_views(pool, hkv, page, d)
        c.table = torch.where(c.table >= 0, c.table + shift, c.table)
        o, lse = c.run()
        assert torch.equal(o, want) and torch.equal(lse, wl)


def test_the_same_bits_every_time_and_on_another_stream():
    for nq, batch in ((1, 33), (4, 20), (80, 3)):
        r = random.Random(nq)
        c = Case8([2048 + r.randrange(nq, 900) for _ in range(batch)], nq, 16, 4, 128, 2048, 16, torch.bfloat16, seed=nq)
        o, lse = c.run()
        for stream in (None, torch.cuda.Stream()):
            o2, l2 = c.run(stream=stream)
            assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("nq", [1, 60])
def test_in_a_graph_with_new_lengths(nq):
    # the launches do not depend on the lengths: a captured call serves a growing batch
    c = Case8([512 + 60, 512 + 90, 512 + 63], nq, 8, 2, 128, 512, 16, torch.bfloat16, seed=11)
    final, most = list(c.lens), 640
    o, lse = torch.empty_like(c.q, memory_format=torch.contiguous_format), torch.empty(3 * nq, 8, device="cuda")
    ws = torch.empty(c.size(512, most), dtype=torch.uint8, device="cuda")
    call = lambda: q.plm_attn_kv8(c.q, o, *c.parts, c.table, c.row_lens, nq, 512, most, c.scale, ws, lse=lse, seqs=c.seqs)  # noqa: E731
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
    c = Case8([64, 64], 1, 4, 2, 128, 0, 16, torch.bfloat16)
    k, v, ke, ve = c.parts
    o, ws = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    ok = dict(q=c.q, o=o, k=k, v=v, k_exps=ke, v_exps=ve, table=c.table, lens=c.row_lens, tokens=1, prefix_len=0, max_len=64, scale=0.1, workspace=ws)
    q.plm_attn_kv8(**ok)
    for bad in (dict(o=o[:1]), dict(v=v[:, :1]), dict(v=v.contiguous()), dict(v=c.v), dict(k=ke), dict(k_exps=ke[..., :2]), dict(v_exps=ve.contiguous()),
                dict(table=c.table.long()), dict(lens=c.row_lens[:1]), dict(tokens=3), dict(tokens=0), dict(lse=o), dict(seqs=c.seqs[:1]),
                dict(q=c.q[..., :64])):
        with pytest.raises(ValueError):
            q.plm_attn_kv8(**{**ok, **bad})
    for bad in (dict(prefix_len=8), dict(max_len=0), dict(prefix_len=128), dict(q=c.q.half())):
        with pytest.raises(q.PlmError):
            q.plm_attn_kv8(**{**ok, **bad})
