"""Attention over 8-bit pages at the ends of its ranges (tests/test_gpu_attn_kv8.py has the definition, the cases and the
terms of the tolerance)."""
import math

import pytest
import torch

import quant_packed_gemv_gb300 as q
from tests import test_gpu_attn_kv8 as base

pytestmark = pytest.mark.gpu


def test_more_heads_than_a_grid_has_rows():
    # 97 rows a head are read back; compared with the same call on a few of the heads
    heads, n, d, page = 65600, 97, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    pages = -(-n // page)
    pool = torch.randint(0, 256, (pages, q.plm_kv8_page_bytes(heads, page, d)), generator=g, dtype=torch.uint8, device="cuda")
    parts = q.plm_kv8_views(pool, heads, page, d)
    for exps in parts[2:]:
        exps.fill_(121)                         # steps of 2^-6
    for codes in parts[:2]:
        codes.clamp_(min=-127)
    x = torch.randn(n, heads, d, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None], torch.tensor([n], **i32)

    def run(h0, h1):
        few = h1 - h0
        o = torch.full((n, few, d), float("nan"), dtype=torch.float32, device="cuda")
        size = q.plm_attn_kv8_workspace_size(1, n, few, few, d, 0, n)
        assert size > 2 * 2 * 128 * few * d
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        q.plm_attn_kv8(x[:, h0:h1], o, *(p[:, h0:h1] for p in parts), table, lens, n, 0, n, 0.1, ws)
        torch.cuda.synchronize()
        assert q.plm_device_fault() == 0
        return o

    o = run(0, heads)
    for h0 in (0, 65533, heads - 4):
        few = run(h0, h0 + 4)
        k, v = (base.decode(c[:, h0:h0 + 4], e[:, h0:h0 + 4])[table[0].long()].transpose(1, 2).reshape(-1, 4, d)[:n].double() for c, e in
                ((parts[0], parts[2]), (parts[1], parts[3])))
        s = torch.einsum("thd,nhd->thn", x[:, h0:h0 + 4].double(), k) * 0.1
        hidden = torch.arange(n, device="cuda")[None] > torch.arange(n, device="cuda")[:, None]
        p = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1)
        want, A = torch.einsum("thn,nhd->thd", p, v), torch.einsum("thn,nhd->thd", p, v.abs())
        size = torch.einsum("thd,nhd->thn", x[:, h0:h0 + 4].double().abs(), k.abs()).amax(-1, keepdim=True) * 0.1
        tol = (2.0 ** -8 + 2 * ((d + 4) * 2.0 ** -24 + 2.0 ** -22) * (1 + size) + 2 * n * 2.0 ** -24) * A   # (p is rounded to bf16)
        for got in (o[:, h0:h0 + 4], few):
            assert bool(((got.double() - want).abs() <= tol + 1e-30).all())


def sized(c, k=0, v=0):
    """The case with keys and values of up to 2^(k + 1), 2^(v + 1), and queries as much smaller as the keys are larger."""
    c.k.copy_((c.k.float().clamp(-1.99, 1.99) * 2.0 ** k).to(c.k.dtype))
    c.v.copy_((c.v.float().clamp(-1.99, 1.99) * 2.0 ** v).to(c.v.dtype))
    c.q.mul_(2.0 ** -k)
    c.q[c.q.abs() < 2.0 ** -126] = 0   # (that a product takes numbers below that is not promised)
    c.encode()
    return c


# rows a sequence and head: up to 32 in four kernels, in chunks, and read back
ROWS = [(1, 8, 4), (6, 2, 1), (9, 4, 2), (24, 2, 2), (30, 4, 4), (20, 4, 2), (60, 4, 2)]


@pytest.mark.parametrize("nq,hq,hkv", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [119, 112, 105, 96, -90])
def test_keys_of_any_size(nq, hq, hkv, d, power):
    c = sized(base.Case8([40 + nq, 33 + nq, nq, 3], nq, hq, hkv, d, 0, 16, torch.bfloat16, seed=power + 200), k=power)
    c.check(*c.run(o_type=torch.float32))
    if power > 0 and c.size(0, max(c.lens)) == 0:   # queries of the usual size, in the rows that take any score: the largest has all of the sum
        c.q.mul_(2.0 ** power)
        c.check(*c.run())


def test_keys_of_unlike_sizes():
    # blocks of 2^119 and of 2^-90 beside ordinary ones in the same key: where the queries are zero they cost the others nothing
    c = base.Case8([77, 50, 61], 4, 4, 2, 128, 0, 16, torch.bfloat16, seed=4)
    c.k[..., :32] = (c.k[..., :32].float().clamp(-1.9, 1.9) * 2.0 ** 119).to(c.k.dtype)
    c.k[..., 96:] *= 2.0 ** -90
    c.q[..., :32] = 0
    c.encode()
    c.check(*c.run(o_type=torch.float32))


@pytest.mark.parametrize("nq,hq,hkv", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k,v", [(0, 119), (119, 119), (-90, 112), (0, -90)])
def test_values_of_any_size(nq, hq, hkv, d, k, v):
    c = sized(base.Case8([40 + nq, 33 + nq, nq, 3], nq, hq, hkv, d, 0, 16, torch.bfloat16, seed=nq + v + 200), k, v)
    c.check(*c.run(o_type=torch.float32))
    c.check(*c.run())


@pytest.mark.parametrize("nq", [1, 4, 10])
def test_large_values_of_many_keys(nq):
    # several CTAs a sequence, scores that rise so that the running reference lags: sums of 5000 p up to 2^8 before they are divided
    c = base.Case8([5000 + nq, 5000, 4000], nq, 4, 2, 128, 0, 16, torch.bfloat16, seed=3)
    assert c.size(0, max(c.lens)) == 0
    for row, n in zip(c.rows, c.lens):
        pages = [p for p in row if p >= 0]
        c.k[pages] = (c.q[0, 0] * torch.linspace(0.0, 3.0, len(pages), device="cuda")[:, None, None, None] + 0.1 * c.k[pages].float().nan_to_num(0.0)).to(c.k.dtype)
    sized(c, 0, 119)
    c.check(*c.run(o_type=torch.float32))
    c.q.zero_()          # the mean of all of them
    c.check(*c.run())


def check_beside(c, o):
    """The output where values differ by far more than an f16 holds.  As in Case8.check, but that what is lost of p is relative to
    the values that have a share in the row (a key below 2^-100 of the row's largest has none: its p is 0), and what is
    lost of small values below 2^-126 of the largest step: 2^-149 of it in each sum, which is divided by 2^7 at least."""
    g = c.hq // c.hkv
    for b, n in enumerate(c.lens):
        pages = [p for p in c.rows[b] if p >= 0]
        k, v = (x[pages].transpose(1, 2).reshape(-1, c.hkv, c.d)[:n].double() for x in (c.k, c.v))
        rows = slice(b * c.nq, (b + 1) * c.nq)
        x = c.q[rows].double().view(c.nq, c.hkv, g, c.d)
        hidden = (torch.arange(n, device="cuda")[None] > torch.arange(n - c.nq, n, device="cuda")[:, None])[:, None, None]
        s = (torch.einsum("thgd,nhd->thgn", x, k) * c.scale).masked_fill(hidden, -math.inf)
        size = (torch.einsum("thgd,nhd->thgn", x.abs(), k.abs()) * c.scale).masked_fill(s < s.amax(-1, keepdim=True) - 70, 0.0).amax(-1)
        p = torch.softmax(s, -1)
        p = p.masked_fill(p < 2.0 ** -100 * p.amax(-1, keepdim=True), 0.0)
        want, A = torch.einsum("thgn,nhd->thgd", p, v), torch.einsum("thgn,nhd->thgd", p, v.abs())
        # (of each key/value head and dim: the largest value with a share)
        top = ((p > 0).permute(1, 3, 0, 2)[..., None] * v.abs().transpose(0, 1)[:, :, None, None]).amax(1).permute(1, 0, 2, 3)
        e = 2 * ((c.d + 4) * 2.0 ** -24 + 2.0 ** -22) * (1 + size)
        tol = (2.0 ** -11 + e[..., None] + 3 * n * 2.0 ** -24) * A + n * 2.0 ** -32 * top + n * 2.0 ** -149 * float(v.abs().amax())
        tol = tol + half_step(o.dtype) * (want.abs() + tol)
        got = o[rows].double().view(want.shape)
        assert not got.isnan().any()
        err = (got - want).abs()
        assert bool((err <= tol).all()), (b, n, float((err / tol).max()))


def half_step(dtype):
    return {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}[dtype]


@pytest.mark.parametrize("nq,hq,hkv", [(2, 8, 4), (6, 2, 1), (9, 4, 2), (20, 2, 2), (24, 2, 2), (30, 4, 4), (20, 4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [119, 40, 25])
@pytest.mark.parametrize("lens", [[40, 33, 97], [3000, 1711]])
def test_values_beside_others_that_a_row_does_not_see(nq, hq, hkv, d, power, lens):
    # drafted tokens: the last one's value is huge, as after an overflow; the queries before it do not see it
    c = base.Case8([n + nq for n in lens], nq, hq, hkv, d, 0, 16, torch.bfloat16, seed=nq + power)
    assert c.size(0, max(c.lens)) == 0
    for row, n in zip(c.rows, c.lens):
        c.v[row[(n - 1) // 16], :, (n - 1) % 16] = 1.5 * 2.0 ** power
    c.encode()
    o, _ = c.run(o_type=torch.float32)
    check_beside(c, o)


@pytest.mark.parametrize("nq,hq,hkv", [(1, 8, 4), (6, 4, 2), (9, 4, 2), (24, 2, 2), (20, 4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [True, False])
def test_values_beside_others_without_probability(nq, hq, hkv, d, first):
    # keys whose score leaves them no share, with values of 2^100, 2^60 and 2^30 beside those of the others, of 1 and 2^-30
    c = base.Case8([48 + nq, 2000 + nq], nq, hq, hkv, d, 0, 16, torch.bfloat16, seed=nq)
    c.q[..., 0] = 8.0
    c.k[..., 0] = 0.0
    for row, n in zip(c.rows, c.lens):
        for i, power in enumerate((100, 60, 30)):
            j = i if first else n - nq - 1 - 17 * i
            at = (row[j // 16], slice(None), j % 16)
            c.k[at] = 0.0
            c.k[at + (slice(0, 1),)] = -2000.0
            c.v[at] = c.v[at] * 2.0 ** power
        c.v[[p for p in row if p >= 0], :, 5] *= 2.0 ** -30
    c.encode()
    o, _ = c.run(o_type=torch.float32)
    check_beside(c, o)


@pytest.mark.parametrize("nq,hq,hkv,prefix,lens", [(60, 4, 2, 0, [100, 61, 300]), (130, 2, 2, 0, [140, 700]), (1, 8, 2, 4096, [4096 + 17 + i for i in range(128)])])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [16, 40, 119])
def test_f16_beside_values_that_it_does_not_hold(nq, hq, hkv, prefix, lens, d, power):
    # pages that are read back; keys and values of 2^16 and more count as 65504, and nothing where a row does not see them:
    # the last token of each sequence for all queries but its own (of the prefix: behind its end)
    c = base.Case8(lens, nq, hq, hkv, d, prefix, 16, torch.float16, seed=power)
    assert c.size(prefix, max(lens)) > 0
    if nq == 1:
        # a query each: one more token behind the one that asks, which the page holds and nobody sees
        c.lens = [n - 1 for n in lens]
        for b, n in enumerate(c.lens):
            c.row_lens[c.seq[b]] = n
    last = [(row[(n - 1) // 16], slice(None), (n - 1) % 16) for row, n in zip(c.rows, lens)]
    for codes, exps in (c.parts[::2], c.parts[1::2]):
        for at in last:
            codes[at] = 127 - 254 * (torch.arange(d, device="cuda") % 2).to(torch.int8)
            exps[at] = 127 + power - 6
    o, lse = c.run(o_type=torch.float32)
    assert not o.isnan().any() and not o.isinf().any()
    for at in last:   # what the rows that do not see it get, they get without it
        c.parts[2][at] = 0
        c.parts[3][at] = 0
        c.k[at] = 0
        c.v[at] = 0
    want, _ = c.run(o_type=torch.float32)
    c.check(want, _)
    seeing = torch.arange(o.shape[0], device="cuda") % nq == nq - 1 if nq > 1 else torch.zeros(o.shape[0], dtype=torch.bool, device="cuda")
    assert torch.equal(o[~seeing], want[~seeing])
