"""The sampler's weights wherever it forms them (sums over a row, short lists, the probability that is given back), to 2^-29
of themselves: by prob, which is a quotient of a weight and a sum, off by 2^-28 for both and rounded once (2^-24).  At
these temperatures the product of a logit and log2(e) / T has a rounding error of its own, up to 2^-19 of 1 in the
exponent, which a weight that took it twice or not at all would show."""
import numpy as np
import pytest

from tests.test_gpu_sample import Rows

pytestmark = pytest.mark.gpu
# all of it is kept: without a look, by a list, by a border that is found among equals
KEPT = [dict(), dict(top_k=4000), dict(top_k=900), dict(top_p=1 - 2.0 ** -24), dict(min_p=1e-11)]


@pytest.mark.parametrize("kept", KEPT)
@pytest.mark.parametrize("t", [0.37, 0.71, 1.0, 1.3, 2.9])
@pytest.mark.parametrize("top", [0.0, 3.0, 17.7, 300.0, -41.3])
def test_sums_of_equal_weights(kept, t, top):
    # one largest logit and n equal ones below it, at many distances: probabilities are 1 / (1 + n w) and w / (1 + n w)
    t = float(np.float32(t))
    for n in (1, 500, 3000):
        if n > kept.get("top_k", n):
            continue
        z = (-np.random.RandomState(n).uniform(0.05, 12.0, 40) * t).astype(np.float32)
        x = np.repeat((np.float32(top) + z)[:, None], n + 1, 1)
        x[:, 0] = top
        w = np.exp((x[:, 1].astype(np.float64) - x[:, 0]) / t)
        for u, token, share in ((0.0, 0, 1 / (1 + n * w)), (1.0, n, w / (1 + n * w))):
            tokens, prob = Rows(x, u=u, temperature=t, **kept).run()
            assert (tokens == token).all()
            assert (np.abs(prob - share) <= (2.0 ** -24 + 2.0 ** -28) * share + (n + 1) * 2.0 ** -40).all()
