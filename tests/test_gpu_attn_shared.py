"""Attention where the prefix is done apart for the whole batch, against the definition in f64 (tolerances and pages:
test_gpu_attn).  The library does so only where that pays, so each size here is checked to take that path: a call that
does not share needs the workspace of one without a prefix."""
import random

import pytest
import torch

import quant_packed_gemv_gb300 as q
from tests.test_gpu_attn import Case, T

pytestmark = pytest.mark.gpu


def apart(c, prefix=None, most=None):
    most = max(c.lens) if most is None else most
    size = lambda p: q.plm_attn_workspace_size(len(c.lens), c.nq, c.hq, c.hkv, c.d, p, most)  # noqa: E731
    return size(c.prefix if prefix is None else prefix) != size(0)


# query heads, key/value heads, head size, tokens: 5 to 96 rows per sequence and key/value head
FEW = [(14, 2, 64, 1), (14, 2, 64, 3), (14, 2, 64, 13), (16, 8, 128, 1), (32, 8, 128, 4), (32, 8, 128, 7), (5, 1, 128, 1), (5, 1, 128, 6),
       (8, 8, 64, 1), (8, 8, 64, 20), (8, 8, 64, 96), (12, 2, 128, 4), (32, 8, 128, 10), (16, 8, 128, 36)]


@pytest.mark.parametrize("hq,hkv,d,nq", FEW)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page,order", [(16, "heads first"), (32, "tokens first"), (64, "heads first"), (128, "tokens first"), (256, "heads first")])
def test_few_rows(hq, hkv, d, nq, dtype, page, order):
    # a first sequence too short to share, idle ones, one that ends with the prefix, one that shares no token of its last page
    prefix = -(-(5248 if nq * hq // hkv <= 16 else 2688) // page) * page
    lens = [40, prefix + nq, prefix + 333, 0, prefix + nq - 1, prefix + 17 + nq, prefix, 0, prefix + 129 + nq, max(1, nq - 3)]
    c = Case(lens, nq, hq, hkv, d, prefix, page, T[dtype], order=order, seed=nq + page)
    assert apart(c)
    c.check(*c.run(o_type=torch.float32 if page == 64 else None))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("batch,nq,hq,hkv,d,prefix", [(60, 1, 4, 2, 64, 2048), (200, 1, 8, 1, 128, 512), (33, 3, 16, 8, 128, 512)])
def test_few_rows_of_a_batch_behind_a_short_prefix(dtype, batch, nq, hq, hkv, d, prefix):
    r = random.Random(batch)
    lens = [r.choice((0, 9, prefix - 1, prefix + nq, prefix + r.randrange(nq, 300), prefix + r.randrange(nq, 300))) for _ in range(batch)]
    c = Case(lens, nq, hq, hkv, d, prefix, 32, T[dtype], seed=batch)
    assert apart(c)
    c.check(*c.run())


# more than 96 rows: the own keys in the tile kernel too.  A sequence's rows in one tile of 128, one of 256, two of 256
MANY = [(60, 14, 14, 2, 64, 10240), (23, 20, 10, 2, 128, 20480), (10, 129, 8, 8, 64, 8192), (24, 35, 32, 8, 64, 5632), (40, 26, 10, 2, 128, 10240),
        (10, 140, 16, 8, 128, 8192)]


@pytest.mark.parametrize("batch,nq,hq,hkv,d,prefix", MANY)
@pytest.mark.parametrize("dtype,page,order", [("f16", 16, "tokens first"), ("bf16", 64, "heads first"), ("bf16", 128, "tokens first"), ("f16", 256, "heads first")])
def test_many_rows(batch, nq, hq, hkv, d, prefix, dtype, page, order):
    r = random.Random(batch + page)
    lens = [prefix + r.randrange(nq, 400) for _ in range(batch)]
    # too short to share (the first of all), idle, fewer keys than queries, at the border of sharing
    lens[0], lens[3], lens[4], lens[6], lens[7], lens[9] = 77, 0, nq // 2, prefix + nq - 1, prefix + nq - 2, prefix
    c = Case(lens, nq, hq, hkv, d, prefix, page, T[dtype], order=order, seed=batch + page)
    assert apart(c)
    c.check(*c.run(o_type=torch.float32 if page == 64 else None))


@pytest.mark.parametrize("nq,batch,prefix", [(1, 5, 5248), (7, 5, 2688), (33, 24, 8192)])
def test_nobody_shares(nq, batch, prefix):
    # all too short or idle: the kernels of the prefix find no row to read it from
    r = random.Random(nq)
    c = Case([r.choice((0, 1, 100, 300)) for _ in range(batch - 1)] + [120], nq, 32, 8, 128, 0, 16, torch.bfloat16, seed=nq)
    assert apart(c, prefix, prefix + 400)
    c.check(*c.run(max_len=prefix + 400, prefix=prefix))


@pytest.mark.parametrize("hq,hkv,nq,d,most", [(40, 1, 1, 128, 5000), (10, 2, 7, 64, 9000), (64, 1, 1, 128, 4500), (8, 1, 8, 128, 4500), (3, 1, 21, 64, 8500),
                                              (96, 1, 1, 128, 2000), (5, 1, 19, 64, 7000), (24, 2, 8, 128, 1700)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_middling_rows_over_many_keys(hq, hkv, nq, d, most, dtype):
    # 33 to 96 rows a sequence and head whose keys are too many for the kernel of few rows
    c = Case([most, 0, most - 1, 3, most // 2 + 5, 130], nq, hq, hkv, d, 0, 32, T[dtype], order="tokens first", seed=nq + most)
    assert q.plm_attn_workspace_size(6, nq, hq, hkv, d, 0, most) > 0
    c.check(*c.run())


@pytest.mark.parametrize("nq", [18, 36, 48])
@pytest.mark.parametrize("prefix", [0, 512])
def test_a_bound_far_above_the_table(nq, prefix):
    # the kernels are chosen, and the workspace sized, by the bound; the rows of the table end long before it
    c = Case([prefix + nq + 9, prefix + 200, 0, 30, prefix + nq], nq, 8, 4, 128, prefix, 16, torch.bfloat16, seed=nq + prefix)
    assert q.plm_attn_workspace_size(5, nq, 8, 4, 128, prefix, 600) != q.plm_attn_workspace_size(5, nq, 8, 4, 128, prefix, 90000)
    c.check(*c.run())
    c.check(*c.run(max_len=90000))


@pytest.mark.parametrize("page", [128, 256, 1024])
@pytest.mark.parametrize("nq", [1, 5, 40, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_pages_alone(page, nq, dtype):
    # nothing shared; a unit of keys is a part of a page
    c = Case([page + nq, 2 * page - 1, 3 * page + 130, 0, 5], nq, 8, 2, 128 if page == 256 else 64, 0, page, T[dtype], seed=page + nq)
    c.check(*c.run())


@pytest.mark.parametrize("nq,batch,prefix", [(1, 6, 5248), (7, 6, 2688), (33, 24, 8192)])
def test_the_same_bits_every_time_apart(nq, batch, prefix):
    r = random.Random(nq)
    c = Case([prefix + r.randrange(nq, 300) for _ in range(batch)], nq, 32, 8, 128, prefix, 16, torch.bfloat16, seed=nq)
    assert apart(c)
    o, lse = c.run()
    for stream in (None, torch.cuda.Stream()):
        o2, l2 = c.run(stream=stream)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def grow(nq, batch, prefix, steps, seed=3):
    """Sequences behind one prompt take nq tokens a step, all calls of all steps queued at once: pages and lengths,
    keys and values, queries are each step's own and written right before they are read."""
    hq, hkv, d, page = 32, 8, 128, 16
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    most = prefix + nq * steps
    pages = prefix // page + batch * (-(-nq * steps // page) + 1) + 8
    pool = torch.full((pages, 2, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    table, lens, refs = torch.full((batch + 1, -(-most // page) + 1), -1, **i32), torch.zeros(batch + 1, **i32), torch.zeros(pages, **i32)
    kv, freqs = q.plm_kv_state(pool, table, lens, refs, page), q.plm_rope_freqs(d, 1e6, device="cuda")[0]
    ws = torch.empty(q.plm_kv_workspace_size(pages, batch), dtype=torch.uint8, device="cuda")
    aws = torch.full((q.plm_attn_workspace_size(batch, nq, hq, hkv, d, prefix, most),), 255, dtype=torch.uint8, device="cuda")
    assert aws.numel() != q.plm_attn_workspace_size(batch, nq, hq, hkv, d, 0, most)
    slots = torch.empty(1, prefix, dtype=torch.int64, device="cuda")
    q.plm_kv_reserve(kv, torch.tensor([0], **i32), torch.tensor([prefix], **i32), slots, ws)
    k, v = rand(prefix, hkv, d), rand(prefix, hkv, d)
    q.plm_rope([q.plm_rope_tensor(k, pool[:, 0], slots=slots[0]), q.plm_rope_tensor(v, pool[:, 1], slots=slots[0], rotate=False)],
               torch.arange(prefix, **i32), freqs, d)
    seqs = torch.arange(1, batch + 1, **i32)
    q.plm_kv_fork(kv, torch.zeros_like(seqs), seqs, ws)
    add, slots = torch.full((batch,), nq, **i32), torch.empty(batch, nq, dtype=torch.int64, device="cuda")
    qr = torch.empty(batch * nq, hq, d, dtype=torch.bfloat16, device="cuda")
    o = torch.empty(steps, batch * nq, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(steps, batch * nq, hq, device="cuda")
    x = rand(steps, batch * nq, hq + 2 * hkv, d)
    at = (prefix + torch.arange(nq * steps, **i32)).view(steps, 1, nq).expand(steps, batch, nq).reshape(steps, -1).contiguous()
    torch.cuda.synchronize()
    for t in range(steps):
        q.plm_kv_reserve(kv, seqs, add, slots, ws)
        s = slots.view(-1)
        q.plm_rope([q.plm_rope_tensor(x[t, :, :hq], qr), q.plm_rope_tensor(x[t, :, hq:hq + hkv], pool[:, 0], slots=s),
                    q.plm_rope_tensor(x[t, :, hq + hkv:], pool[:, 1], slots=s, rotate=False)], at[t], freqs, d)
        q.plm_attn_shared_prefix(qr, o[t], pool[:, 0], pool[:, 1], table, lens, nq, prefix, most, d ** -0.5, aws, lse=lse[t], seqs=seqs)
    torch.cuda.synchronize()
    assert q.plm_device_fault() == 0
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    return o, lse


@pytest.mark.parametrize("nq,batch,prefix,steps", [(1, 8, 5248, 40), (1, 90, 1024, 30), (7, 8, 2688, 20), (33, 24, 8192, 4)])
def test_the_same_bits_in_every_launch_mode_apart(nq, batch, prefix, steps):
    # with early launch the kernel of the own keys starts beside that of the prefix, and reads what earlier calls wrote
    runs, before = [], q.plm_set_overlap(q.PLM_OVERLAP_OFF)
    try:
        for mode in (q.PLM_OVERLAP_OFF, q.PLM_OVERLAP_LAUNCH, q.PLM_OVERLAP_PREFETCH, q.PLM_OVERLAP_LAUNCH):
            q.plm_set_overlap(mode)
            runs.append(grow(nq, batch, prefix, steps))
    finally:
        q.plm_set_overlap(before)
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
