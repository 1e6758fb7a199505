"""Host checks of the norm, the 8-bit cache, its attention and the sampler: refused arguments (nothing is launched), the
binding's blocks and its own checks."""
import ctypes
import struct

import pytest
import torch

import quant_packed_gemv_gb300 as q
from quant_packed_gemv_gb300 import plm as P

A = 1 << 20   # a 256-byte aligned fake address; never dereferenced: every call below is rejected
OK, BAD, MIS, UNS = P.PLM_OK, P.PLM_ERR_INVALID_ARG, P.PLM_ERR_MISALIGNED, P.PLM_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    p = dict(x=A, residual=A + (1 << 16), weight=A, sum=A + (1 << 17), xq=A, y=None, m=4, k=512, x_stride=512, residual_stride=512,
             sum_stride=512, y_stride=512, eps=1e-6, x_type=0, r_type=0, w_type=0, y_type=0)
    p.update(kw)
    return P._RmsnormProblem(**p)


def test_norm_refusals():
    st = lambda **kw: P.raw_status("plm_rmsnorm", ctypes.byref(norm(**kw)), None)  # noqa: E731
    assert P.raw_status("plm_rmsnorm", None, None) == BAD
    for bad in (dict(x=None), dict(xq=None), dict(residual=None), dict(m=-1), dict(m=1 << 31), dict(k=0), dict(k=1 << 31), dict(k=300, x_stride=512),
                dict(eps=-1.0), dict(eps=NAN), dict(x_type=3), dict(r_type=-1), dict(w_type=7), dict(y=A + 4096, y_type=5), dict(x_stride=511),
                dict(residual_stride=0), dict(sum_stride=100), dict(y=A + 4096, y_stride=-512), dict(y=A + (1 << 17)),
                # an output in the place of an input of another type or stride
                dict(sum=A, x_type=1), dict(sum=A, sum_stride=600), dict(sum=A + (1 << 16), sum_stride=600), dict(y=A, y_type=2),
                dict(y=A + (1 << 16), y_type=1), dict(y=A + (1 << 16), y_stride=1024)):
        assert st(**bad) == BAD, bad
    for bad in (dict(x=A + 2), dict(residual=A + 1), dict(weight=A + 2), dict(sum=A + 3), dict(xq=A + 2), dict(y=A + 4097, y_type=1)):
        assert st(**bad) == MIS, bad
    wide = dict(x_stride=1 << 31, residual_stride=1 << 31, sum_stride=1 << 31)
    assert st(m=0, k=1 << 30, **wide) == OK and st(m=0, k=(1 << 30) + 256, **wide) == BAD and st(m=1, k=(1 << 31) - 256, **wide) == BAD
    assert st(m=0) == OK
    assert st(m=0, sum=A) == OK and st(m=0, sum=A + (1 << 16)) == OK and st(m=0, y=A) == OK   # in place
    assert st(m=0, weight=None, w_type=9, residual=None, sum=None, r_type=9) == OK             # types of what is not there


def kv8(**kw):
    t = dict(rows=A, codes=A, exps=A, slots=A, heads=8, row_token_stride=1024, row_head_stride=128, page_tokens=16, pages=64,
             page_stride=1 << 16, head_stride=2048, token_stride=128, exp_page_stride=1 << 16, exp_head_stride=64, type=0, rotate=1)
    t.update(kw)
    return P._Kv8Tensor(**t)


def test_cache_refusals():
    def both(*tensors, count=None, tokens=4, d=128):
        arr, n = (P._Kv8Tensor * len(tensors))(*tensors), len(tensors) if count is None else count
        found = (P.raw_status("plm_kv8_write", arr, n, A, A, tokens, d, 32, 0, 1.0, None), P.raw_status("plm_kv8_read", arr, n, tokens, d, None))
        assert found[0] == found[1]
        return found[0]
    assert P.raw_status("plm_kv8_write", None, 1, A, A, 4, 128, 128, 0, 1.0, None) == BAD
    assert P.raw_status("plm_kv8_read", None, 1, 4, 128, None) == BAD
    for bad in (dict(count=0), dict(count=9), dict(tokens=-1), dict(tokens=1 << 31), dict(d=0), dict(d=48), dict(d=1056)):
        assert both(kv8(), **bad) == BAD, bad
    for bad in (dict(rows=None), dict(codes=None), dict(exps=None), dict(slots=None), dict(heads=0), dict(heads=65537), dict(type=3), dict(page_tokens=0),
                dict(pages=0), dict(page_tokens=1 << 31), dict(pages=1 << 31)):
        assert both(kv8(**bad)) == BAD, bad
    assert both(kv8(heads=65536), tokens=0) == OK and both(kv8(heads=65536), kv8(heads=1), tokens=0) == BAD
    for bad in (dict(rows=A + 2), dict(slots=A + 4), dict(codes=A + 2), dict(page_stride=6), dict(head_stride=2), dict(token_stride=130)):
        assert both(kv8(**bad)) == MIS, bad
    assert both(kv8(), tokens=0) == OK and both(kv8(exps=A + 1, exp_page_stride=3), tokens=0) == OK   # exponents are bytes

    def write(t=None, pos=A, freqs=A, rot=128, layout=0, tokens=4, d=128):
        return P.raw_status("plm_kv8_write", (P._Kv8Tensor * 1)(t or kv8()), 1, pos, freqs, tokens, d, rot, layout, 1.0, None)
    assert write(pos=None) == BAD and write(freqs=None) == BAD and write(rot=0) == BAD and write(rot=3) == BAD and write(rot=130) == BAD
    assert write(layout=2) == BAD and write(pos=A + 2) == MIS and write(freqs=A + 4) == MIS
    assert write(kv8(rotate=0), pos=None, freqs=None, rot=0, layout=7, tokens=0) == OK   # nothing turns: not looked at


def attn(**kw):
    p = dict(q=A, o=A, lse=None, k=A, v=A, k_exps=A, v_exps=A, table=A, lens=A, seqs=None, batch=4, tokens=1, heads=16, kv_heads=8,
             head_dim=128, q_token_stride=2048, q_head_stride=128, o_token_stride=2048, o_head_stride=128, page_tokens=16,
             pages=64, page_stride=1 << 15, kv_head_stride=2048, kv_token_stride=128, exp_page_stride=1 << 15, exp_head_stride=64,
             table_stride=8, rows=4, prefix_len=64, max_len=100, scale=0.1, type=2, o_type=2)
    p.update(kw)
    return P._AttnKv8Problem(**p)


def test_attention_refusals():
    ws = 1 << 40
    st = lambda w=A, b=ws, **kw: P.raw_status("plm_attn_kv8", ctypes.byref(attn(**kw)), w, b, None)  # noqa: E731
    assert P.raw_status("plm_attn_kv8", None, A, ws, None) == BAD
    for f in ("q", "o", "k", "v", "k_exps", "v_exps", "table", "lens"):
        assert st(**{f: None}) == BAD
    for bad in (dict(batch=-1), dict(batch=1 << 31), dict(tokens=0), dict(heads=0), dict(heads=12), dict(kv_heads=0),
                dict(kv_heads=32), dict(head_dim=0), dict(type=0), dict(type=5), dict(o_type=1), dict(pages=0), dict(rows=0),
                dict(page_tokens=0), dict(table_stride=0), dict(max_len=0), dict(prefix_len=-16), dict(prefix_len=112),
                dict(prefix_len=40), dict(page_stride=-16), dict(exp_page_stride=-16), dict(exp_head_stride=-16), dict(batch=1 << 20, tokens=1 << 10)):
        assert st(**bad) == BAD, bad
    for bad in (dict(head_dim=96), dict(page_tokens=8), dict(page_tokens=48, prefix_len=48)):
        assert st(**bad) == UNS, bad
    for bad in (dict(q=A + 8), dict(o=A + 8), dict(k=A + 8), dict(v=A + 8), dict(k_exps=A + 4), dict(v_exps=A + 8), dict(lse=A + 2), dict(table=A + 2),
                dict(lens=A + 1), dict(seqs=A + 2), dict(q_token_stride=2052), dict(q_head_stride=130), dict(o_token_stride=2052),
                dict(page_stride=8), dict(kv_head_stride=2056), dict(kv_token_stride=136), dict(exp_page_stride=8), dict(exp_head_stride=68),
                dict(o_type=0, o_head_stride=126)):
        assert st(**bad) == MIS, bad
    assert st(batch=0) == OK
    size = q.plm_attn_kv8_workspace_size
    for bad in ((0, 1, 16, 8, 128, 64, 100), (4, 0, 16, 8, 128, 64, 100), (4, 1, 12, 8, 128, 64, 100),
                (4, 1, 16, 8, 96, 64, 100), (4, 1, 16, 8, 128, 101, 100), (4, 1, 16, 8, 128, 64, 0)):
        assert size(*bad) == 0
    # which calls read back: by rows and keys, and a prefix that enough others would read
    assert [size(24, n, 32, 8, 128, 0, most) > 0 for n, most in ((12, 1 << 20), (13, 5120), (16, 5120), (16, 5121), (17, 2048), (24, 2048), (24, 2049),
                                                                 (25, 100))] == [False, False, False, True, False, False, True, True]
    assert [size(b, n, 32, 8, 128, p, p + 300) > 0 for b, n, p in ((1, 1, 32768), (2, 1, 16384), (16, 1, 1024), (64, 1, 512), (128, 1, 1024), (24, 1, 4096),
                                                                   (2, 7, 8192))] == [False, False, False, False, True, True, True]
    need = size(4, 100, 16, 8, 128, 64, 200)   # 200 rows a head: read back, 2 bytes a value
    assert need > 4 * 200 * 8 * 128 * 2 * 2
    assert st(tokens=100, max_len=200, b=need - 1) == BAD and st(tokens=100, max_len=200, w=None) == BAD
    assert st(tokens=100, max_len=200, w=A + 16) == MIS
    assert st(batch=1 << 16, tokens=100, heads=16, rows=1 << 16, max_len=1 << 30) == UNS   # more units than can be counted


def sample(**kw):
    p = dict(logits=A, u=A, temperature=A, top_k=A, top_p=A, min_p=A, tokens=A, prob=None, m=4, n=1000, stride=1000, type=0)
    p.update(kw)
    return P._SampleProblem(**p)


def test_sample_refusals():
    st = lambda **kw: P.raw_status("plm_sample", ctypes.byref(sample(**kw)), None)  # noqa: E731
    assert P.raw_status("plm_sample", None, None) == BAD
    for bad in (dict(logits=None), dict(tokens=None), dict(m=-1), dict(m=(1 << 24) + 1), dict(n=0), dict(n=(1 << 22) + 1, stride=1 << 23), dict(stride=999),
                dict(type=3)):
        assert st(**bad) == BAD, bad
    for f in ("u", "temperature", "top_k", "top_p", "min_p", "tokens", "prob"):
        assert st(**{f: A + 2}) == MIS
    assert st(logits=A + 2) == MIS and st(logits=A + 1, type=1) == MIS
    assert st(m=0) == OK and st(m=0, u=None, temperature=None, top_k=None, top_p=None, min_p=None) == OK


def test_packed_calls_are_the_same_calls():
    call = lambda entry, args: P.raw_status("plm_call", entry, args)  # noqa: E731
    q8 = lambda *v: struct.pack("@%dq" % len(v), *v)  # noqa: E731
    assert call(8, q8(0) + bytes(norm(k=300))) == BAD and call(8, q8(0) + bytes(norm(x=A + 2))) == MIS and call(8, q8(0) + bytes(norm(m=0))) == OK
    write = lambda count=1, pos=A, freqs=A, tokens=4, d=128, rot=128, layout=0, t=None: call(  # noqa: E731
        9, struct.pack("@7qdq", count, pos, freqs, tokens, d, rot, layout, 1.0, 0) + bytes(t or kv8()))
    assert write(count=0) == BAD and write(pos=0) == BAD and write(freqs=A + 4) == MIS and write(rot=3) == BAD and write(layout=2) == BAD
    assert write(d=48) == BAD and write(t=kv8(rows=A + 2)) == MIS and write(tokens=0) == OK
    assert call(10, q8(1, 4, 48, 0) + bytes(kv8())) == BAD and call(10, q8(1, 4, 128, 0) + bytes(kv8(slots=A + 4))) == MIS
    assert call(10, q8(1, 0, 128, 0) + bytes(kv8())) == OK
    assert call(11, q8(A, 1 << 40, 0) + bytes(attn(k_exps=A + 8))) == MIS and call(11, q8(A, 1 << 40, 0) + bytes(attn(head_dim=96))) == UNS
    assert call(11, q8(A, 1 << 40, 0) + bytes(attn(batch=0))) == OK
    assert call(12, q8(0) + bytes(sample(n=0))) == BAD and call(12, q8(0) + bytes(sample(u=A + 2))) == MIS and call(12, q8(0) + bytes(sample(m=0))) == OK
    assert call(13, q8(0) + bytes(attn())) == BAD


def test_the_bindings_blocks_have_the_structs_layout():
    for ctype, packed in ((P._RmsnormProblem, P._RMSNORM_PROBLEM), (P._Kv8Tensor, P._KV8_TENSOR), (P._AttnKv8Problem, P._ATTN_KV8_PROBLEM),
                          (P._SampleProblem, P._SAMPLE_PROBLEM)):
        values = list(range(1, len(ctype._fields_) + 1))
        assert ctypes.sizeof(ctype) == packed.size and bytes(ctype(*values)) == packed.pack(*values)


def test_a_pools_views_tile_its_pages():
    heads, page, d = 3, 16, 64
    size = q.plm_kv8_page_bytes(heads, page, d)
    assert size == 2 * heads * page * (d + 2) and size % 16 == 0
    pool = torch.zeros(5, size + 32, dtype=torch.uint8)
    views = q.plm_kv8_views(pool, heads, page, d)
    for i, x in enumerate(views):
        assert x.dtype == (torch.int8 if i < 2 else torch.uint8) and x.shape == (5, heads, page, d if i < 2 else d // 32)
        x.add_(i + 1)
    n = heads * page * d
    row = pool[2].tolist()
    assert row == [1] * n + [2] * n + [3] * (n // 32) + [4] * (n // 32) + [0] * 32   # each byte in one view
    part = pool[1:, 16:]   # a pool that is a part of another
    k = q.plm_kv8_views(part, heads, page, d)[0]
    assert k.data_ptr() == pool.data_ptr() + pool.shape[1] + 16 and k.stride(0) == pool.shape[1]
    for bad in (pool[:, :size - 1], pool.view(torch.int8), pool[0]):
        with pytest.raises(ValueError):
            q.plm_kv8_views(bad, heads, page, d)
    with pytest.raises(ValueError):
        q.plm_kv8_views(pool, heads, page, 48)


class OnDevice:
    """What the binding asks of a CUDA tensor, of one that is not."""

    def __init__(self, t):
        self.t = t
        self.is_cuda = True
        self.shape, self.dtype, self.nbytes = t.shape, t.dtype, t.nbytes

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_the_binding_checks_shapes_and_types():
    dev = lambda *shape, dtype=torch.float32: OnDevice(torch.zeros(*shape, dtype=dtype))  # noqa: E731
    x, i32 = dev(3, 512), torch.int32
    for kw in (dict(residual=dev(3, 500)), dict(sum=dev(3, 512)), dict(residual=dev(3, 512), sum=dev(3, 512, dtype=torch.float16)),
               dict(xq=dev(3, 584, dtype=torch.int16)), dict(y=dev(4, 512)), dict(y=dev(3, 512, dtype=i32)), dict(residual=torch.zeros(3, 512))):
        with pytest.raises(ValueError):
            q.plm_rmsnorm(x, None, 1e-6, **kw)
    with pytest.raises(ValueError):
        q.plm_rmsnorm(x, dev(511), 1e-6, y=dev(3, 512))
    with pytest.raises(ValueError):
        q.plm_rmsnorm(dev(3, 512, dtype=i32), None, 1e-6, y=dev(3, 512))
    codes, exps, slots = dev(9, 2, 16, 64, dtype=torch.int8), dev(9, 2, 16, 2, dtype=torch.uint8), dev(3, dtype=torch.int64)
    rows = dev(3, 2, 64)
    t = q.plm_kv8_tensor(rows, codes, exps, slots)
    for bad in ((dev(3, 3, 64), codes, exps, slots), (rows, exps, exps, slots), (rows, codes, dev(9, 2, 16, 3, dtype=torch.uint8), slots),
                (rows, codes, exps, dev(3, dtype=i32)), (rows, codes, exps, dev(4, dtype=torch.int64)), (dev(3, 2, 64, dtype=i32), codes, exps, slots)):
        with pytest.raises(ValueError):
            q.plm_kv8_tensor(*bad)
    other = q.plm_kv8_tensor(dev(4, 2, 64), codes, exps, dev(4, dtype=torch.int64), rotate=False)
    for call in (lambda: q.plm_kv8_write([t, other]), lambda: q.plm_kv8_read([t, other]), lambda: q.plm_kv8_read([]), lambda: q.plm_kv8_write([t]),
                 lambda: q.plm_kv8_write([t], dev(3, dtype=i32), dev(5, dtype=torch.int64), 64)):
        with pytest.raises(ValueError):
            call()
    logits, tokens = dev(3, 100), dev(3, dtype=i32)
    for kw in (dict(u=dev(4)), dict(u=dev(3, dtype=torch.float64)), dict(top_k=dev(3)), dict(top_p=dev(2)), dict(prob=dev(3, dtype=torch.float16))):
        with pytest.raises(ValueError):
            q.plm_sample(logits, tokens, **kw)
    with pytest.raises(ValueError):
        q.plm_sample(logits, dev(3, dtype=torch.int64))
