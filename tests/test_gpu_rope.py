"""Rotary positions on the GPU against the definition in f64.

Tolerance, per value of a turned pair (a, b): the turns are exact to 2^-32 and
rounded to 24 bits (angle error <= pi 2^-24 + 2 pi 2^-32), sincospi is within 2
ulp, so cos and sin are off by <= 3.3e-7; their scaling, two products and a sum
round by 2^-24 each: |error| <= 6e-7 scale (|a| + |b|), taken as 8e-7.  A
rounding to f16 or bf16 adds half an ulp: 2^-11 or 2^-8 of the value."""
import math

import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def turned(x, positions, freqs, rot, layout, scale, inverse):
    """(values, bound on their f32 error) in f64, by the definition."""
    w = torch.tensor([(int(f) % 2 ** 64) / 2.0 ** 64 for f in freqs], dtype=torch.float64, device=x.device)
    turns = positions.double()[:, None] * w     # positions < 2^24 below: fractions exact to 2^-28
    angle = 2 * math.pi * (turns - turns.round())
    c, s = scale * angle.cos()[:, None], scale * angle.sin()[:, None] * (-1 if inverse else 1)
    x = x.double()
    y, bound = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    bound[..., ia] = bound[..., ib] = 8e-7 * scale * (a.abs() + b.abs())
    return y, bound


def check(got, want, bound, yt):
    err = (got.double() - want).abs()
    assert bool((err <= bound + HALF_ULP[yt] * (want.abs() + bound) + 2.0 ** -24 * (yt == "f16")).all()), float(err.max())


@pytest.mark.parametrize("tokens,heads,d,rot", [(1, 16, 128, 128), (5, 3, 64, 64), (67, 7, 128, 64), (9, 2, 64, 6), (300, 32, 128, 128),
                                                (33, 5, 80, 24), (4, 1, 1024, 1024), (2, 3, 2, 2), (1500, 4, 96, 50)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f16")])
def test_rows(tokens, heads, d, rot, layout, xt, yt):
    g = torch.Generator(device="cuda").manual_seed(tokens + d)
    x = torch.randn(tokens, heads, d, generator=g, device="cuda").to(T[xt])
    pos = torch.randint(0, 1 << 17, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    freqs, scale = q.plm_rope_freqs(rot, 1e4, "ramp" if rot > 8 else "none", 4.0, 4096, device="cuda")
    buf = torch.full((tokens * heads * d + 64,), 7.0, dtype=T[yt], device="cuda")
    y = buf[:-64].view(tokens, heads, d)
    for inverse in (False, True):
        buf[:-64] = float("nan")
        q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs, rot, layout, scale=scale, inverse=inverse)
        want, bound = turned(x, pos, freqs, rot, layout, scale, inverse)
        check(y, want, bound, yt)
        if xt == yt:
            assert torch.equal(y[..., rot:], x[..., rot:])
        assert bool((buf[-64:] == 7.0).all())


def test_far_positions_stay_exact():
    # 2^30 + i and i differ by a whole number of 2^30 steps: the fractions of a turn are integer arithmetic
    freqs, _ = q.plm_rope_freqs(128, 1e6, device="cuda")
    pos = torch.tensor([0, 1, 2 ** 20 + 3, 2 ** 30 + 7, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    x = torch.randn(6, 2, 128, device="cuda")
    y = torch.empty_like(x)
    q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs, 128)
    for t, p in enumerate(pos.tolist()):
        frac = [((p * int(f)) % 2 ** 64) / 2.0 ** 64 for f in freqs.tolist()]
        angle = 2 * math.pi * torch.tensor(frac, dtype=torch.float64, device="cuda")
        a, b = x[t, :, :64].double(), x[t, :, 64:].double()
        want = torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)
        assert bool(((y[t].double() - want).abs() <= 8e-7 * (a.abs() + b.abs()).repeat(1, 2)).all())


def test_gradient_is_the_inverse():
    # L = sum w y(x): dL/dx against central differences of the f32 forward call, and the inverse undoes the forward
    freqs, _ = q.plm_rope_freqs(12, 1e4, device="cuda")
    pos = torch.tensor([3, 900], dtype=torch.int32, device="cuda")
    x, w = torch.randn(2, 2, 16, device="cuda"), torch.randn(2, 2, 16, device="cuda")
    y, grad = torch.empty_like(x), torch.empty_like(x)
    for layout in ("half", "interleaved"):
        q.plm_rope([q.plm_rope_tensor(w, grad)], pos, freqs, 12, layout, scale=1.25, inverse=True)
        for t in range(2):
            for h in range(2):
                for i in range(16):
                    side = []
                    for e in (0.5, -0.5):   # linear: any step is exact
                        z = x.clone()
                        z[t, h, i] += e
                        q.plm_rope([q.plm_rope_tensor(z, y)], pos, freqs, 12, layout, scale=1.25)
                        side.append(float((y.double() * w.double()).sum()))
                    # 64 values, each within 8e-7 * 1.25 * (|a| + |b|) < 1e-5
                    assert abs(side[0] - side[1] - float(grad[t, h, i])) < 64 * 2e-5
        back = torch.empty_like(x)
        q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs, 12, layout)
        q.plm_rope([q.plm_rope_tensor(y, back)], pos, freqs, 12, layout, inverse=True)
        assert float((back - x).abs().max()) < 2e-5


def test_in_place_equals_out_of_place():
    for dt, d, rot, layout in ((torch.bfloat16, 128, 128, "half"), (torch.float32, 64, 30, "interleaved"), (torch.float16, 128, 64, "half")):
        x = torch.randn(37, 6, d, device="cuda").to(dt)
        pos = torch.arange(100, 137, dtype=torch.int32, device="cuda")
        freqs, _ = q.plm_rope_freqs(rot, 1e4, device="cuda")
        y = torch.empty_like(x)
        q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs, rot, layout)
        q.plm_rope([q.plm_rope_tensor(x, x)], pos, freqs, rot, layout)
        assert torch.equal(x, y)


@pytest.mark.parametrize("order", ["heads first", "tokens first"])
@pytest.mark.parametrize("page", [1, 5, 16])
def test_q_k_v_of_one_product_into_the_cache(order, page):
    hq, hkv, d, tokens, pages = 6, 2, 64, 41, 60
    qkv = torch.randn(tokens, (hq + 2 * hkv) * d + 3, device="cuda")[:, :(hq + 2 * hkv) * d].unflatten(1, (-1, d))  # ragged rows
    shape = (pages, 2, hkv, page, d) if order == "heads first" else (pages, 2, page, hkv, d)
    pool = torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda")
    k, v = pool[:, 0], pool[:, 1]
    if order == "tokens first":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    slots = torch.randperm(pages * page, device="cuda")[:tokens]
    slots[7], slots[11] = -1, pages * page   # padding tokens: not written
    pos = torch.randint(0, 9999, (tokens,), device="cuda", dtype=torch.int32)
    freqs, _ = q.plm_rope_freqs(d, 1e4, device="cuda")
    y = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    xk, xv = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q.plm_rope([q.plm_rope_tensor(qkv[:, :hq], y), q.plm_rope_tensor(xk, k, slots=slots),
                q.plm_rope_tensor(xv, v, slots=slots, rotate=False)], pos, freqs, d)
    want, bound = turned(qkv[:, :hq], pos, freqs, d, "half", 1.0, False)
    check(y, want, bound, "bf16")
    want, bound = turned(xk, pos, freqs, d, "half", 1.0, False)
    seen = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            check(k[s // page, :, s % page], want[t], bound[t], "bf16")
            assert torch.equal(v[s // page, :, s % page], xv[t].bfloat16())
            seen[s // page, s % page] = True
    assert bool((k.transpose(1, 2)[~seen] == 9.0).all()) and bool((v.transpose(1, 2)[~seen] == 9.0).all())


def test_offsets_past_32_bits():
    d, hkv, page = 128, 8, 16
    pages = (1 << 32) // (hkv * page * d) + 40       # the last pages start past 2^32 elements
    pool = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, hkv, d, device="cuda")
    pool[-1] = 0
    slots = torch.tensor([pages * page - 1, pages * page - 16, 5], device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")   # no turn
    freqs, _ = q.plm_rope_freqs(d, 1e4, device="cuda")
    q.plm_rope([q.plm_rope_tensor(x, pool, slots=slots)], pos, freqs, d)
    assert torch.equal(pool[-1, :, 15], x[0].bfloat16()) and torch.equal(pool[-1, :, 0], x[1].bfloat16())
    assert torch.equal(pool[0, :, 5], x[2].bfloat16()) and bool((pool[-1, :, 1:15] == 0).all())


def test_temporaries_of_a_nested_call():
    # each part's input is made, and forgotten, within the call: none may take another's place
    x = torch.randn(3, 50, 4, 64, device="cuda")
    y, want = torch.empty(3, 50, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 50, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos, freqs = torch.arange(50, dtype=torch.int32, device="cuda"), q.plm_rope_freqs(64, 1e4, device="cuda")[0]
    held = [x[i].bfloat16() for i in range(3)]
    for i in range(3):
        q.plm_rope([q.plm_rope_tensor(held[i], want[i])], pos, freqs, 64)
    q.plm_rope([q.plm_rope_tensor(x[0].bfloat16(), y[0]), q.plm_rope_tensor(x[1].bfloat16(), y[1]),
                q.plm_rope_tensor(x[2].bfloat16(), y[2])], pos, freqs, 64)
    assert torch.equal(y, want)


def test_side_stream_and_empty_call():
    side = torch.cuda.Stream()
    x = torch.randn(1000, 8, 128, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    pos = torch.arange(1000, dtype=torch.int32, device="cuda")
    freqs, _ = q.plm_rope_freqs(128, 1e4, device="cuda")
    q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs, 128)
    side.wait_stream(torch.cuda.current_stream())
    q.plm_rope([q.plm_rope_tensor(x, z)], pos, freqs, 128, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    q.plm_rope([q.plm_rope_tensor(x[:0], y[:0])], pos[:0], freqs, 128)


def test_binding_refuses():
    x, freqs = torch.randn(4, 2, 64, device="cuda"), q.plm_rope_freqs(64, 1e4, device="cuda")[0]
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    for bad in (lambda: q.plm_rope_tensor(x, y[:3]), lambda: q.plm_rope_tensor(x.cpu(), y), lambda: q.plm_rope_tensor(x.double(), y),
                lambda: q.plm_rope_tensor(x.transpose(1, 2), y.transpose(1, 2)),
                lambda: q.plm_rope_tensor(x, y[None], slots=pos),                       # int32 slots
                lambda: q.plm_rope([q.plm_rope_tensor(x, y)], pos.long(), freqs, 64),   # int64 positions
                lambda: q.plm_rope([q.plm_rope_tensor(x, y)], pos[:3], freqs, 64),
                lambda: q.plm_rope([q.plm_rope_tensor(x, y)], pos, freqs[:3], 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.PlmError):
        q.plm_rope([], pos, freqs, 64)
