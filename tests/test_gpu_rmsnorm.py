"""Residual sum, norm and q8_K blocks on the GPU against the definition in f64.

The sum h is one addition and one rounding: equal bit for bit.  y, per value, relative to itself: the sum of squares of
k <= 16384 values is of positive terms, each in 8 fused steps of a lane, 5 of a warp and at most 1 + 5 over the chunks (20 of
them beyond): 24 roundings at most, of which the root leaves half; a division by k, + eps (halved as well), the root, a
division, two products: (24 + 2) / 2 + 4 = 17 half steps of 2^-24, then one of y's type.
The blocks are those that plm_quantize_q8K makes of y, byte for byte."""
import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a step at 0
EPS = 1e-6


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def rows(values, dtype, pitch=0, skip=0):
    """values as rows `pitch` apart that begin `skip` values into an allocation, NaN around them."""
    m, k = values.shape
    pitch = pitch or k
    buf = torch.full((skip + m * pitch + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[skip:skip + m * pitch].view(m, pitch)[:, :k]
    view.copy_(values)
    return view


def expect(x, residual, weight, eps=EPS):
    h = x.float() if residual is None else (x.float() + residual.float()).to(residual.dtype)
    d = h.double()
    y = d / (d.square().sum(-1, keepdim=True) / x.shape[1] + eps).sqrt()
    return h, y if weight is None else y * weight.double()


def near(y, want):
    u, t = HALF[y.dtype], TINY[y.dtype]
    off = (y.double() - want).abs()
    assert not off.isnan().any()
    assert bool((off <= (17 * 2.0 ** -24 * (1 + u) + u) * want.abs() + t).all()), float((off / (want.abs() + 1e-30)).max())


def blocks_of(y):
    m, k = y.shape
    xq = torch.empty(m, k // 256 * 292, dtype=torch.uint8, device="cuda")
    q.plm_quantize_q8K(y, xq, m, k)
    return xq


# rows of one warp, of several, of several chunks a warp, in one CTA or many, beyond the registers; few and many
SHAPES = [(1, 256), (1, 1024), (3, 2048), (5, 4096), (9, 6144), (2, 12288), (1, 16384), (700, 256), (1300, 512), (901, 1024), (640, 4096), (2, 16640), (1, 40192)]


@pytest.mark.parametrize("m,k", SHAPES)
def test_sum_norm_and_blocks(m, k):
    x, r, w = rand(m, m, k), 3 * rand(k, m, k), 1 + 0.3 * rand(1, k)
    xq = torch.full((m * (k // 256) * 292 + 64,), 171, dtype=torch.uint8, device="cuda")
    h, y = torch.full((m, k), float("nan"), device="cuda"), torch.full((m, k), float("nan"), device="cuda")
    q.plm_rmsnorm(x, w, EPS, residual=r, sum=h, xq=xq[:-64], y=y)
    sum_, want = expect(x, r, w)
    assert torch.equal(h, sum_)
    near(y, want)
    assert torch.equal(xq[:-64].view(m, -1), blocks_of(y)) and bool((xq[-64:] == 171).all())
    # the blocks alone are the same ones, with and without the sum
    for kw in (dict(), dict(sum=torch.empty_like(h))):
        only = torch.zeros_like(xq[:-64])
        q.plm_rmsnorm(x, w, EPS, residual=r, xq=only, **kw)
        assert torch.equal(only, xq[:-64])


@pytest.mark.parametrize("k", [1, 2, 3, 31, 64, 100, 127, 128, 129, 255, 257, 1000, 1023, 4100, 16385, 20001])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_rows_of_any_length(t, k):
    for m, pitch, skip in ((1, 0, 0), (7, k + 3, 1), (40, k + (-k) % 4 + 8, 4)):
        x, y = rows(rand(k, m, k), T[t], pitch, skip), rows(torch.zeros(m, k, device="cuda"), T[t], pitch and pitch + 1, skip)
        q.plm_rmsnorm(x, None, EPS, y=y)
        near(y, expect(x, None, None)[1])
        if pitch:   # what lies between the rows is left as it was
            whole = torch.as_strided(y, (m, pitch + 1), (pitch + 1, 1), skip)
            assert bool(whole[:-1, k:].isnan().all())


@pytest.mark.parametrize("xt", list(T))
@pytest.mark.parametrize("rt", list(T))
@pytest.mark.parametrize("wt,yt", [("f32", "bf16"), ("bf16", "f16"), ("f16", "f32")])
def test_types(xt, rt, wt, yt):
    m, k = 6, 768
    x, r, w = rand(1, m, k).to(T[xt]), rand(2, m, k).to(T[rt]), (1 + rand(3, k)).to(T[wt])
    y, h, f32 = torch.empty(m, k, dtype=T[yt], device="cuda"), torch.empty_like(r), torch.empty(m, k, device="cuda")
    xq = torch.empty(m, k // 256 * 292, dtype=torch.uint8, device="cuda")
    q.plm_rmsnorm(x, w, EPS, residual=r, sum=h, y=y, xq=xq)
    sum_, want = expect(x, r, w)
    assert torch.equal(h, sum_)   # the norm is of the sum as it is stored
    near(y, want)
    q.plm_rmsnorm(x, w, EPS, residual=r, y=f32)   # the same without storing it
    near(f32, want)
    assert torch.equal(f32.to(T[yt]), y) and torch.equal(blocks_of(f32), xq)


@pytest.mark.parametrize("k", [512, 1000, 16640])
def test_in_place(k):
    m, w = 5, 1 + 0.1 * rand(9, k)
    x, r = rand(1, m, k), rand(2, m, k)
    sum_, want = expect(x, r, w)
    for place in ("residual", "x"):
        a, b, y = x.clone(), r.clone(), torch.empty(m, k, device="cuda")
        q.plm_rmsnorm(a, w, EPS, residual=b, sum=b if place == "residual" else a, y=y)
        assert torch.equal(b if place == "residual" else a, sum_) and torch.equal(a if place == "residual" else b, x if place == "residual" else r)
        near(y, want)
    for place in ("x", "residual"):   # the result over an input, the sum kept or not
        for keep in (False, True):
            a, b, h = x.clone(), r.clone(), torch.empty(m, k, device="cuda")
            y = a if place == "x" else b
            q.plm_rmsnorm(a, w, EPS, residual=b, sum=h if keep else None, y=y)
            near(y, want)
            assert not keep or torch.equal(h, sum_)
    a, b = x.clone(), r.clone()   # both: the layer's next residual and its input, in the places of the last ones
    q.plm_rmsnorm(a, w, EPS, residual=b, sum=b, y=a)
    assert torch.equal(b, sum_)
    near(a, want)


def test_a_row_does_not_depend_on_the_others():
    for k in (256, 1000, 4096, 20000):
        x, r, y = rand(1, 3000, k), rand(2, 3000, k), torch.empty(3000, k, device="cuda")
        q.plm_rmsnorm(x, None, EPS, residual=r, y=y)
        for m in (1, 7, 200):
            part = torch.empty(m, k, device="cuda")
            q.plm_rmsnorm(x[:m], None, EPS, residual=r[:m], y=part)
            assert torch.equal(part, y[:m])


def test_rows_of_zeros_and_extremes():
    k = 512
    x = torch.zeros(6, k, device="cuda")
    x[1, 5] = -3.0           # one value
    x[2, :] = 2.0            # the block's maximum occurs everywhere
    x[3, 7], x[3, 300] = -1e18, 1e18
    x[4, :] = 1e-30          # eps decides
    x[5, 255], x[5, 256] = 1.0, -1.0
    y, xq = torch.empty_like(x), torch.empty(6, k // 256 * 292, dtype=torch.uint8, device="cuda")
    q.plm_rmsnorm(x, None, EPS, y=y, xq=xq)
    near(y, expect(x, None, None)[1])
    assert torch.equal(xq, blocks_of(y))
    assert bool((y[0] == 0).all()) and bool((xq[0] == 0).all())
    q.plm_rmsnorm(torch.zeros(1, k, device="cuda"), None, 0.0, y=y[:1])   # 0 / 0: NaN, and no more than that
    assert bool(y[0].isnan().all())
    empty = torch.empty(0, k, device="cuda")
    q.plm_rmsnorm(empty, None, EPS, y=torch.empty_like(empty))


def test_streams_and_graphs():
    m, k = 33, 2048
    x, r, w = rand(1, m, k), rand(2, m, k), rand(3, k)
    h, xq = torch.empty_like(x), torch.empty(m, k // 256 * 292, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q.plm_rmsnorm(x, w, EPS, residual=r, sum=h, xq=xq, stream=stream)
    torch.cuda.synchronize()
    want, sums = xq.clone(), h.clone()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q.plm_rmsnorm(x, w, EPS, residual=r, sum=h, xq=xq)
    for factor in (1.0, -2.0):
        x.mul_(factor)
        r.mul_(factor)
        xq.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, sums * factor)
        y = torch.empty_like(x)
        q.plm_rmsnorm(x, w, EPS, residual=r, y=y)
        assert torch.equal(xq, blocks_of(y))
        assert factor != 1.0 or torch.equal(xq, want)
