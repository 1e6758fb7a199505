"""The example that uses rotary positions, cache pages and shared-prefix attention together, between the packed products.

Its attention results are compared with f64 on keys and values rounded to bf16 once: what separates them is the rounding
of the probabilities to bf16 (2^-9 in the mean square sense at most) and keys that the f32 rotation rounds the other way
(2^-8 of a few of them): 1e-2 of the norm covers both."""
import importlib.util
import os

import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prefix_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("shared_prefix_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("prompt,steps,samples", [(333, 24, 8), (16, 9, 3), (5, 20, 8)])
def test_samples_of_one_prompt(prompt, steps, samples):
    e = example()
    worst, live, outputs = e.run(prompt, steps, samples)
    assert worst < 1e-2
    assert all(bool(torch.isfinite(o).all()) for o in outputs)
    # pages in use: the prompt's own, and for each sample that goes on its tokens past the shared full pages
    full, rest = prompt // e.PAGE, prompt % e.PAGE
    going = samples - samples // 2
    assert live == full + (rest > 0) + going * -(-(rest + steps) // e.PAGE)
    assert q.plm_device_fault() == 0


def test_the_same_bits_in_every_launch_mode():
    # early launch must not let a kernel read what the one before has not written
    runs = []
    before = q.plm_set_overlap(q.PLM_OVERLAP_OFF)
    try:
        for mode in (q.PLM_OVERLAP_OFF, q.PLM_OVERLAP_LAUNCH, q.PLM_OVERLAP_PREFETCH, q.PLM_OVERLAP_LAUNCH):
            q.plm_set_overlap(mode)
            runs.append(example().run(100, 40, 6)[2])
    finally:
        q.plm_set_overlap(before)
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
