"""The norm's q8_K blocks are those of plm_quantize_q8K byte for byte, for values that no model should have too
(tests/test_gpu_rmsnorm.py has the ordinary ones)."""
import math

import pytest
import torch

import quant_packed_gemv_gb300 as q
from tests.test_gpu_rmsnorm import EPS, blocks_of, rand

pytestmark = pytest.mark.gpu
NAN, INF = math.nan, math.inf


def run(x, w, r=None):
    m, k = x.shape
    y, xq = torch.empty(m, k, device="cuda"), torch.full((m, k // 256 * 292), 171, dtype=torch.uint8, device="cuda")
    q.plm_rmsnorm(x, w, EPS, residual=r, y=y, xq=xq)
    only = torch.zeros_like(xq)
    q.plm_rmsnorm(x, w, EPS, residual=r, xq=only)
    assert torch.equal(xq, blocks_of(y)) and torch.equal(only, xq)
    return y, xq.view(m, k // 256, 292)


# one chunk a row, several of a warp, rows that are read twice
@pytest.mark.parametrize("m,k", [(3, 256), (700, 1024), (5, 4096), (2, 16640)])
def test_nan_and_infinities(m, k):
    x, w = rand(m, m, k), 1 + 0.3 * rand(1, k)
    for bad in (NAN, INF, -INF):
        # in a row: all of its values are NaN (or 0, where an infinity has made the others nothing), and no other row's
        xs = x.clone()
        xs[1, 200] = bad
        y, blocks = run(xs, w, 0.5 * x)
        assert bool(y[1, 200].isnan()) and not bool(y[[i for i in range(m) if i != 1]].isnan().any())
        assert bool((blocks[1] == 0).all())   # a block of nothing but NaN and zeros: scale 0, codes 0
        # in the weight: one value of each row, which gets code 0, and the others of its block as if it were not there
        ws = w.clone()
        ws[100] = bad
        y, blocks = run(x, ws)
        if math.isnan(bad):
            zero = w.clone()
            zero[100] = 0.0
            _, want = run(x, zero)
            assert bool(y[:, 100].isnan().all()) and torch.equal(blocks, want)
    ws = torch.full_like(w, NAN)              # all of them
    assert bool((run(x, ws)[1] == 0).all())
    ws[::3] = INF
    ws[1::3] = -INF
    run(x, ws)


def test_values_of_one_block_alone():
    m, k = 4, 1024
    x, w = rand(1, m, k), torch.ones(k, device="cuda")
    w[256:512] = NAN
    w[256 + 255] = -2.0                       # the only one of its block
    y, blocks = run(x, w)
    assert not bool(y[:, 511].isnan().any()) and bool(y[:, 256:511].isnan().all())
    d = blocks[:, 1, :4].contiguous().view(torch.float32)[:, 0]
    assert torch.equal(d, 1.0 / (-128.0 / y[:, 511])) and bool((blocks[:, 1, 4 + 255] == 128).all()) and bool((blocks[:, 1, 4:4 + 255] == 0).all())


@pytest.mark.parametrize("m,k", [(3, 256), (700, 1024), (5, 4096), (2, 16640)])
@pytest.mark.parametrize("size", [1e-36, 3e-38, 1e-40, 1.5e-45])
def test_blocks_of_the_smallest_values(m, k, size):
    # -128 / max is infinite from 128 / 2^128 downwards: codes are 127, 0 or what is left of -2^31 in a byte
    x, w = rand(m, m, k), torch.full((k,), size, device="cuda")
    x[:, 7] = 0.0
    y, blocks = run(x, w)
    assert size > 1e-37 or bool((blocks[:, :, 4:260] == 127).any())
