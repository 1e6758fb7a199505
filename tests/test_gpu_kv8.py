"""The 8-bit cache on the GPU: rows written and read back, against the format's definition.

What is not turned is one exact scaling and one rounding: codes, exponents and values are equal to those formed here on the
CPU, bit for bit.  A turned value y = a c - b s has c and s to 2^-21 (2^-24 of a turn as f32 is 2 pi 2^-25 of c; sincospi
and the scale add 2^-23) and three roundings of at most 2^-24 (|a| + |b|): it is off by at most w = 2^-20 (|a| + |b|) scale, and
what is stored by that and half a step more, where the step may also be the next one at a border that w reaches."""
import math

import numpy as np
import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def encode(x):
    """Codes and exponents of x [..][d] (numpy f32), by the definition."""
    x = np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=2.0 ** 120, neginf=-2.0 ** 120), -2.0 ** 120, 2.0 ** 120)
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    j = np.full(top.shape, -100)
    while True:
        up = top * 2.0 ** -j.astype(np.float64) >= 127.5
        if not up.any():
            break
        j = j + up
    codes = np.rint(b * 2.0 ** -j.astype(np.float64)[..., None])   # to nearest, ties to even
    assert np.abs(codes).max() <= 127
    return codes.reshape(x.shape).astype(np.int8), np.where(top == 0, 0, j + 127).astype(np.uint8)


def decode(codes, exps):
    scale = np.where(exps == 0, 0.0, 2.0 ** (exps.astype(np.float64) - 127))
    return (codes.reshape(*exps.shape, 32) * scale[..., None]).reshape(codes.shape)


class Pages:
    """A pool with a byte of its own wherever nothing may be written."""

    def __init__(self, tokens, heads, d, page, seed=0, order="pool", gone=0):
        self.heads, self.d, self.page = heads, d, page
        n = -(-tokens // page) + 3
        g = np.random.RandomState(seed)
        self.slots_np = g.permutation(n * page)[:tokens].astype(np.int64)
        for i in range(gone):
            self.slots_np[g.randint(tokens)] = (-1, n * page, -7, 1 << 40)[i % 4]
        self.slots = torch.from_numpy(self.slots_np).cuda()
        self.n = n
        if order == "pool":
            self.pool = torch.full((n, q.plm_kv8_page_bytes(heads, page, d)), 165, dtype=torch.uint8, device="cuda")
            self.k, self.v, self.ke, self.ve = q.plm_kv8_views(self.pool, heads, page, d)
        else:   # tokens first, and pages apart
            self.pool = torch.full((n, 2, page + 1, heads, d), 165, dtype=torch.uint8, device="cuda").view(torch.int8)
            self.exps = torch.full((n, 2, heads, page, d // 32), 165, dtype=torch.uint8, device="cuda")
            self.k, self.v = (self.pool[:, i, :page].transpose(1, 2) for i in (0, 1))
            self.ke, self.ve = self.exps[:, 0], self.exps[:, 1]

    def at(self, codes, exps):
        """(codes, exponents) of the slots as numpy, zeros where there is none."""
        good = (self.slots_np >= 0) & (self.slots_np < self.n * self.page)
        s = np.where(good, self.slots_np, 0)
        c, e = (x.permute(0, 2, 1, 3).reshape(self.n * self.page, self.heads, -1).cpu().numpy()[s] for x in (codes, exps))
        return np.where(good[:, None, None], c, 0).astype(c.dtype), np.where(good[:, None, None], e, 0).astype(e.dtype)

    def untouched(self):
        """Whether every other slot is as it was."""
        good = self.slots_np[(self.slots_np >= 0) & (self.slots_np < self.n * self.page)]
        rest = np.setdiff1d(np.arange(self.n * self.page), good)
        for x in (self.k, self.v, self.ke, self.ve):
            flat = x.permute(0, 2, 1, 3).reshape(self.n * self.page, self.heads, -1).cpu().numpy().view(np.uint8)
            if not (flat[rest] == 165).all():
                return False
        return True


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("tokens,heads,d,page,order", [(1, 1, 32, 16, "pool"), (1, 8, 128, 16, "pool"), (61, 8, 128, 16, "pool"), (333, 2, 64, 64, "tokens"),
                                                       (7, 3, 96, 12, "tokens"), (1025, 5, 160, 32, "pool"), (40, 1, 1024, 1, "tokens"), (2000, 8, 128, 1024, "pool")])
@pytest.mark.parametrize("t", list(T))
def test_written_as_defined_and_read_back(tokens, heads, d, page, order, t):
    P = Pages(tokens, heads, d, page, seed=tokens, order=order, gone=0 if tokens < 3 else 2)
    x = (rand(tokens, tokens, 2 * heads + 1, d) * torch.exp(3 * rand(5, tokens, 2 * heads + 1, 1))).to(T[t])   # k and v in a product's rows
    xk, xv = x[:, :heads], x[:, heads + 1:]
    q.plm_kv8_write([q.plm_kv8_tensor(xk, P.k, P.ke, P.slots, rotate=False), q.plm_kv8_tensor(xv, P.v, P.ve, P.slots, rotate=False)])
    torch.cuda.synchronize()
    good = ((P.slots_np >= 0) & (P.slots_np < P.n * page))[:, None, None]
    for x_, codes, exps in ((xk, P.k, P.ke), (xv, P.v, P.ve)):
        c, e = P.at(codes, exps)
        wc, we = encode(x_.float().cpu().numpy())
        assert np.array_equal(c, np.where(good, wc, 0)) and np.array_equal(e, np.where(good, we, 0))
    assert P.untouched()
    for out in T.values():
        y = torch.full((2, tokens, heads + 1, d), float("nan"), dtype=out, device="cuda")
        q.plm_kv8_read([q.plm_kv8_tensor(y[i][:, :heads], codes, exps, P.slots) for i, (codes, exps) in enumerate(((P.k, P.ke), (P.v, P.ve)))])
        for i, (codes, exps) in enumerate(((P.k, P.ke), (P.v, P.ve))):
            want = torch.from_numpy(decode(*P.at(codes, exps))).cuda()
            assert torch.equal(y[i][:, :heads], want.float().to(out))
            assert out is not torch.bfloat16 or torch.equal(y[i][:, :heads].double(), want)   # exact
        assert bool(y[:, :, heads].isnan().all())


def test_borders_of_the_format():
    d = 32
    rows = []
    for top in (127.0, 127.49, 127.5, 127.75, 128.0, 63.75, 63.7, 64.0, 1.9921875, 1.9921874, 2.0, 0.0, 1e-38, 2.0 ** -100, 2.0 ** -94 * 1.99, 2.0 ** 120, 2.0 ** 119,
                3.4e38, math.inf):
        for sign in (1, -1):
            row = np.linspace(-0.5, 0.5, d) * (0 if math.isinf(top) else min(top, 1e30))
            row[11] = sign * top
            rows.append(row)
    rows.append(np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5, 127.0] * 4))   # ties go to the even code
    rows.append(np.array([np.nan] * 31 + [3.0]))
    rows.append(np.array([np.nan] * 32))
    rows.append(np.array([-0.0] * 32))
    rows.append(np.array([np.inf, -np.inf] + [1.0] * 30))
    rows.append(np.array([2.0 ** -149] * 32))
    x = np.array(rows).astype(np.float32)[:, None]
    P = Pages(len(rows), 1, d, 16)
    xd = torch.from_numpy(x).cuda()
    q.plm_kv8_write([q.plm_kv8_tensor(xd, P.k, P.ke, P.slots, rotate=False)])
    c, e = P.at(P.k, P.ke)
    wc, we = encode(x)
    assert np.array_equal(c, wc) and np.array_equal(e, we)
    y = torch.empty_like(xd)
    q.plm_kv8_read([q.plm_kv8_tensor(y, P.k, P.ke, P.slots)])
    assert np.array_equal(y.cpu().numpy().astype(np.float64), decode(wc, we)) and bool(y.isfinite().all())


def turned(x, positions, rot, base, half, scale):
    """x [tokens][heads][d] in f64, turned, and |a| + |b| of each value's pair."""
    x = x.double()
    w = torch.tensor([base ** (-2.0 * i / rot) / (2 * math.pi) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    w = torch.round(w * 2.0 ** 52) * 2.0 ** -52   # the frequencies given are the same; p w in f64 is off by 2^-36 of a turn at most
    angle = 2 * math.pi * torch.frac(positions.double()[:, None] * w)[:, None]
    out, size = x.clone(), torch.zeros_like(x)
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., one], x[..., two]
    out[..., one], out[..., two] = scale * (a * angle.cos() - b * angle.sin()), scale * (b * angle.cos() + a * angle.sin())
    size[..., one] = size[..., two] = scale * (a.abs() + b.abs())
    freqs = [int(v) << 12 for v in (w * 2.0 ** 52).tolist()]
    return out, size, torch.tensor([f - 2 ** 64 if f >= 2 ** 63 else f for f in freqs], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("tokens,heads,d,rot", [(1, 8, 128, 128), (61, 8, 128, 64), (700, 2, 64, 64), (130, 3, 96, 50), (9, 1, 160, 2), (33, 2, 128, 126), (5, 1, 1024, 1024)])
@pytest.mark.parametrize("half", [True, False])
def test_turned_rows(tokens, heads, d, rot, half):
    for t, skip in ((torch.float32, 0), (torch.bfloat16, 0), (torch.float32, 1)):
        P = Pages(tokens, heads, d, 16, seed=rot, gone=0 if tokens == 1 else 1)
        buf = rand(rot, tokens * 2 * heads * d + 8).to(t)
        x = buf[skip:skip + tokens * 2 * heads * d].view(tokens, 2 * heads, d)   # skip: no access of four values is aligned
        xk, xv = x[:, :heads], x[:, heads:]
        positions = torch.randint(0, 1 << 20, (tokens,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.int32)
        want, size, freqs = turned(xk, positions, rot, 1e6, half, 1.5)
        q.plm_kv8_write([q.plm_kv8_tensor(xk, P.k, P.ke, P.slots), q.plm_kv8_tensor(xv, P.v, P.ve, P.slots, rotate=False)], positions, freqs, rot,
                        "half" if half else "interleaved", scale=1.5)
        good = torch.from_numpy((P.slots_np >= 0) & (P.slots_np < P.n * 16)).cuda()[:, None, None]
        c, e = P.at(P.k, P.ke)
        got, step = torch.from_numpy(decode(c, e)).cuda(), torch.from_numpy(2.0 ** (e.astype(np.float64) - 127)).cuda().repeat_interleave(32, -1)
        w = 2.0 ** -20 * size
        assert bool((((got - want).abs() <= w + step / 2) | ~good).all())
        # the step is the smallest that holds the block, give or take w
        most = torch.maximum(want.abs() + w, torch.zeros_like(w)).view(tokens, heads, -1, 32).amax(-1)
        least = (want.abs() - w).view(tokens, heads, -1, 32).amax(-1)
        s = torch.from_numpy(2.0 ** (e.astype(np.float64) - 127)).cuda()
        assert bool(((least < 127.5 * s) & (most >= 127.5 * s / 2) | ~good[..., 0, None]).all())
        vc, ve = P.at(P.v, P.ve)
        wc, we = encode(xv.float().cpu().numpy())
        g = good.cpu().numpy()
        assert np.array_equal(vc, np.where(g, wc, 0)) and np.array_equal(ve, np.where(g, we, 0))
        assert P.untouched()


def test_one_launch_of_eight_tensors_and_a_replayed_one():
    tokens, heads, d = 50, 2, 64
    P = [Pages(tokens, heads, d, 16, seed=i) for i in range(4)]
    x = rand(3, 8, tokens, heads, d)
    parts = [q.plm_kv8_tensor(x[2 * i + j], (p.k, p.v)[j], (p.ke, p.ve)[j], p.slots, rotate=False) for i, p in enumerate(P) for j in (0, 1)]
    y = torch.empty_like(x)
    back = [q.plm_kv8_tensor(y[2 * i + j], (p.k, p.v)[j], (p.ke, p.ve)[j], p.slots) for i, p in enumerate(P) for j in (0, 1)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q.plm_kv8_write(parts)
        q.plm_kv8_read(back)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q.plm_kv8_write(parts)
            q.plm_kv8_read(back)
    torch.cuda.synchronize()
    for factor in (1.0, 0.01):
        x.mul_(factor)
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = decode(*encode(x.cpu().numpy()))
        assert np.array_equal(y.cpu().numpy().astype(np.float64), want)
    none = torch.empty(0, heads, d, device="cuda")
    empty = q.plm_kv8_tensor(none, P[0].k, P[0].ke, torch.empty(0, dtype=torch.int64, device="cuda"), rotate=False)
    q.plm_kv8_write([empty])
    q.plm_kv8_read([empty])


def test_slots_beyond_32_bits():
    # a pool of more than 2^32 bytes: places are worked out in 64 bits
    heads, page, d = 8, 64, 128
    size = q.plm_kv8_page_bytes(heads, page, d)
    pages = (1 << 32) // size + 40
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    k, v, ke, ve = q.plm_kv8_views(pool, heads, page, d)
    x = rand(1, 5, heads, d)
    slots = torch.tensor([0, (pages - 1) * page + 63, (pages - 20) * page + 1, pages * page, 17], dtype=torch.int64, device="cuda")
    q.plm_kv8_write([q.plm_kv8_tensor(x, k, ke, slots, rotate=False), q.plm_kv8_tensor(-x, v, ve, slots, rotate=False)])
    y = torch.empty(2, 5, heads, d, device="cuda")
    q.plm_kv8_read([q.plm_kv8_tensor(y[0], k, ke, slots), q.plm_kv8_tensor(y[1], v, ve, slots)])
    want = decode(*encode(x.cpu().numpy()))
    want[3] = 0.0
    assert np.array_equal(y[0].cpu().numpy().astype(np.float64), want) and torch.equal(y[1], -y[0])
    where = pool[pages - 1].view(torch.int8)[:heads * page * d].view(heads, page, d)[:, 63]
    assert np.array_equal(where.cpu().numpy(), encode(x.cpu().numpy())[0][1])


def test_pages_are_forked_and_compacted_as_one():
    # the page calls move codes and exponents together
    heads, page, d = 2, 16, 64
    pool = torch.zeros(12, q.plm_kv8_page_bytes(heads, page, d), dtype=torch.uint8, device="cuda")
    k, v, ke, ve = q.plm_kv8_views(pool, heads, page, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, refs, status = torch.full((4, 6), -1, **i32), torch.zeros(4, **i32), torch.zeros(12, **i32), torch.zeros(1, **i32)
    kv = q.plm_kv_state(pool, table, lens, refs, page, status)
    ws = torch.empty(q.plm_kv_workspace_size(12, 4), dtype=torch.uint8, device="cuda")
    one = lambda *a: torch.tensor(a, **i32)  # noqa: E731
    x = rand(1, 40, heads, d)
    slots = torch.empty(1, 40, dtype=torch.int64, device="cuda")
    q.plm_kv_reserve(kv, one(0), one(40), slots, ws)
    q.plm_kv8_write([q.plm_kv8_tensor(x, k, ke, slots[0], rotate=False), q.plm_kv8_tensor(2 * x, v, ve, slots[0], rotate=False)])
    q.plm_kv_fork(kv, one(0), one(1), ws)
    q.plm_kv_free(kv, one(0))
    q.plm_kv_compact(kv, None, ws)
    at = torch.arange(40, device="cuda")
    slots = table[1, at // page].long() * page + at % page
    y = torch.empty(2, 40, heads, d, device="cuda")
    q.plm_kv8_read([q.plm_kv8_tensor(y[0], k, ke, slots), q.plm_kv8_tensor(y[1], v, ve, slots)])
    want = decode(*encode(x.cpu().numpy()))
    assert np.array_equal(y[0].cpu().numpy().astype(np.float64), want) and np.array_equal(y[1].cpu().numpy().astype(np.float64), 2 * want)
    assert int(status) == 0 and int(refs[:3].sum()) == 3 and int(refs[3:].sum()) == 0
