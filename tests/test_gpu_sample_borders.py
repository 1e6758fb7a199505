"""Rows whose border of a top-p or top-k lies at zero, among logits of both signs that share one bin, so that the
sampler cuts ranges of keys until a bin is one value (tests/test_gpu_sample.py has the definition and the tolerances)."""
import numpy as np
import pytest

from tests.test_gpu_sample import Rows

pytestmark = pytest.mark.gpu
LOG2E = np.float32(1.4426950408889634)   # a temperature of which a step of the histogram is 1/64 of a logit


def around_zero(zeros, tiny, each=6000):
    """Logits from just below 2^-7 down to above -2^-7, all in the bin of 1/64, with zeros and the smallest negative ones between.  The
    largest's key ends in ones, so that one of the bins of keys begins at that of -0."""
    top = np.uint32(0x3BFFFFFF).view(np.float32)
    x = np.concatenate([np.linspace(0.003, top, each), np.zeros(zeros), -1e-41 * np.arange(1, tiny + 1), np.linspace(-0.0077, -0.003, each)]).astype(np.float32)
    assert x.max() == top and (np.abs(x) < 2.0 ** -7).all()
    return x


@pytest.mark.parametrize("zeros,tiny", [(2, 50), (1, 50), (300, 50), (2, 1), (2000, 1500)])
def test_borders_next_to_zero(zeros, tiny):
    x = around_zero(zeros, tiny)
    order = np.argsort(-x, kind="stable")
    w = np.exp((x[order].astype(np.float64) - x.max()) / LOG2E)
    mass = np.cumsum(w)
    last = [6000 - 2, 6000, 6000 + zeros - 1, 6000 + zeros, 6000 + zeros + tiny // 2, 6000 + zeros + tiny - 1, 6000 + zeros + tiny]
    ps = [(mass[j] - 0.5 * w[j]) / mass[-1] for j in last]   # the border is the j-th in order
    us = [0.0, 0.4, 1.0]                                     # (1: the last of those kept, by index)
    shuffled = np.random.RandomState(zeros).permutation(len(x))
    for p in ps:
        for row in (x, x[shuffled]):
            Rows(np.repeat(row[None], 3, 0), u=us, temperature=LOG2E, top_p=p).check()
    for k in [j + 1 for j in last]:
        Rows(np.repeat(x[shuffled][None], 3, 0), u=us, temperature=LOG2E, top_k=k).check()
    Rows(np.repeat(x[shuffled][None], 3, 0), u=us, temperature=LOG2E, top_k=9000, top_p=ps[3], min_p=0.99).check()
