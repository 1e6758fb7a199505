"""Attention over 8-bit pages, way by way: which one a case takes is asserted by the workspace that it asks for (nothing:
few rows, all keys in their kernel; something, and nothing without a prefix: the prefix apart; something without one: all
read back)."""
import random

import pytest
import torch

from tests.test_gpu_attn_kv8 import Case8, T
from tests.test_gpu_attn_kv8_range import check_beside

pytestmark = pytest.mark.gpu


def way(c, prefix):
    most = max(max(c.lens), prefix)
    return "read back" if c.size(0, most) > 0 else "prefix apart" if c.size(prefix, most) > 0 else "few rows"


# the prefix costs twice as much unshared as apart, or so: a rule that moves a little still takes it apart
@pytest.mark.parametrize("batch,nq,prefix,d,dtype,expected", [
    (128, 1, 4096, 128, "bf16", "prefix apart"), (80, 5, 4080, 64, "f16", "prefix apart"), (60, 9, 2032, 128, "bf16", "prefix apart"), (64, 12, 2048, 64, "bf16", "prefix apart"),
    (24, 30, 3088, 64, "bf16", "read back"), (4, 1, 512, 128, "f16", "few rows")])
def test_ways_with_a_prefix(batch, nq, prefix, d, dtype, expected):
    r = random.Random(batch)
    lens = [prefix + r.randrange(nq, 200) for _ in range(batch)]
    lens[3], lens[1], lens[0] = 0, prefix + nq - 2 if nq > 1 else prefix - 1, 5   # idle, and too short to share it
    c = Case8(lens, nq, 8, 2, d, prefix, 16, T[dtype], seed=batch)
    assert way(c, prefix) == expected
    c.check(*c.run())
    c.check(*c.run(o_type=torch.float32))


@pytest.mark.parametrize("nq,hq,hkv", [(1, 8, 4), (1, 14, 2), (6, 2, 1), (9, 4, 2), (24, 2, 2), (30, 4, 4), (20, 4, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_p_of_few_rows_is_rounded_to_f16(nq, hq, hkv, d, dtype):
    # whatever the type of q: 2^-11 of itself, which an output in f32 shows (a p in bf16 would be off by 2^-8 of it); over
    # few keys, whose roundings do not even out, and over many
    lens = [nq, nq + 1, nq + 2, nq + 4, nq + 40, 700]
    c = Case8(lens, nq, hq, hkv, d, 0, 16, T[dtype], seed=nq + d)
    assert way(c, 0) == "few rows"
    o, _ = c.run(o_type=torch.float32)
    check_beside(c, o)
