"""Host checks of rotary positions, cache pages and shared-prefix attention: the frequencies (host arithmetic) against
their definitions, and refused arguments (nothing is launched)."""
import ctypes
import math

import pytest
import torch

import quant_packed_gemv_gb300 as q
from quant_packed_gemv_gb300 import plm as P

A = 1 << 20   # a 256-byte aligned fake address; never dereferenced: every call below is rejected
BAD, MIS, UNS = P.PLM_ERR_INVALID_ARG, P.PLM_ERR_MISALIGNED, P.PLM_ERR_UNSUPPORTED


def radians(freqs):
    return [(int(f) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for f in freqs]


def close(got, want):
    # w = pow(..) in f64, rounded to 2^-64 of a turn
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert abs(g - w) <= 1e-14 * w + 2 * math.pi * 2.0 ** -63


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 250])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_frequencies(rot, base):
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    freqs, scale = q.plm_rope_freqs(rot, base)
    close(radians(freqs), plain)
    assert scale == 1.0
    close(radians(q.plm_rope_freqs(rot, base, "linear", factor=8.0)[0]), [w / 8.0 for w in plain])
    if rot > 2:
        freqs, scale = q.plm_rope_freqs(rot, base, "base", factor=4.0)
        close(radians(freqs), [(base * 4.0 ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)])
        if rot > 4:   # the slowest pair slows by the factor
            assert abs(radians(freqs)[-1] * 4.0 / plain[-1] - 1) < 1e-9
    got = radians(q.plm_rope_freqs(rot, base, "bands", factor=8.0, trained=8192, low=1.0, high=4.0)[0])
    want = []
    for w in plain:
        turns = 8192 * w / (2 * math.pi)
        r = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        want.append(w * (r + (1 - r) / 8.0))
    close(got, want)
    freqs, scale = q.plm_rope_freqs(rot, base, "ramp", factor=16.0, trained=4096, low=1.0, high=32.0)
    assert abs(scale - (0.1 * math.log(16.0) + 1.0)) < 1e-6
    got = radians(freqs)
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    first, last = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
    for i, w in enumerate(plain):
        r = 1.0 if i <= first else 0.0 if i >= last else 1 - (i - first) / (last - first)
        assert abs(got[i] - w * (r + (1 - r) / 16.0)) <= 1e-12 * w + 2 * math.pi * 2.0 ** -63


def test_frequency_refusals():
    held = torch.empty(64, dtype=torch.int64)
    f = held.data_ptr()
    st = lambda *a: P.raw_status("plm_rope_freqs", *a)  # noqa: E731
    none = None
    assert st(None, 64, 1e4, none, none) == BAD
    for rot in (0, -2, 3, 1 << 20):
        assert st(f, rot, 1e4, none, none) == BAD
    for base in (1.0, 0.0, -5.0, float("nan"), float("inf")):
        assert st(f, 64, base, none, none) == BAD
    for bad in ((7, 2.0, 0, 0, 0), (-1, 2.0, 0, 0, 0), (1, 0.5, 0, 0, 0), (1, float("nan"), 0, 0, 0),
                (3, 2.0, 0.0, 1.0, 4.0), (3, 2.0, 8192, 4.0, 1.0), (4, 2.0, 8192, 0.0, 4.0)):
        assert st(f, 64, 1e4, ctypes.byref(P._RopeScaling(*bad)), none) == BAD
    assert st(f, 2, 1e4, ctypes.byref(P._RopeScaling(2, 2.0, 0, 0, 0)), none) == BAD
    assert st(f, 64, 1e4, none, none) == P.PLM_OK


def rope_tensor(**kw):
    t = dict(x=A, y=A + 4096, slots=None, heads=8, x_token_stride=1024, x_head_stride=128, y_token_stride=1024,
             y_head_stride=128, page_tokens=0, page_stride=0, pages=0, x_type=0, y_type=2, rotate=1)
    t.update(kw)
    return P._RopeTensor(**t)


def test_rope_refusals():
    def st(t=None, count=1, pos=A, freqs=A, tokens=4, d=128, rot=128, layout=0):
        arr = (P._RopeTensor * 1)(t or rope_tensor())
        return P.raw_status("plm_rope", arr, count, pos, freqs, tokens, d, rot, layout, 1.0, 0, None)
    assert P.raw_status("plm_rope", None, 1, A, A, 4, 128, 128, 0, 1.0, 0, None) == BAD
    assert st(count=0) == BAD and st(count=9) == BAD
    assert st(pos=None) == BAD and st(freqs=None) == BAD and st(tokens=-1) == BAD and st(tokens=1 << 31) == BAD
    assert st(d=0) == BAD and st(d=127) == BAD and st(d=2048) == BAD
    assert st(rot=0) == BAD and st(rot=3) == BAD and st(rot=130) == BAD and st(layout=2) == BAD
    for kw in (dict(x=None), dict(y=None), dict(heads=0), dict(heads=1 << 20), dict(x_type=3), dict(y_type=-1),
               dict(slots=A, page_tokens=0, pages=4), dict(slots=A, page_tokens=16, pages=0),
               dict(y=A), dict(y=A, y_type=0, y_token_stride=2048), dict(y=A, y_type=0, slots=A, page_tokens=16, pages=4)):
        assert st(rope_tensor(**kw)) == BAD, kw
    for kw in (dict(x=A + 2), dict(y=A + 1), dict(slots=A + 4, page_tokens=16, pages=4)):
        assert st(rope_tensor(**kw)) == MIS, kw
    assert st(pos=A + 2) == MIS and st(freqs=A + 4) == MIS
    assert st(tokens=0) == P.PLM_OK   # nothing to do


def kv(**kw):
    s = dict(pool=A, page_bytes=4096, pages=64, table=A, lens=A, refs=A, status=None, max_seqs=4, max_pages=16,
             page_tokens=16)
    s.update(kw)
    return P._KvState(**s)


def test_page_refusals():
    ws = q.plm_kv_workspace_size(64, 4)
    assert ws >= 4 * 64 and q.plm_kv_workspace_size(0, 4) == 0 and q.plm_kv_workspace_size(64, -1) == 0
    calls = {
        "plm_kv_reserve": lambda s, n=4, w=A, b=ws: P.raw_status("plm_kv_reserve", s, A, A, n, None, 0, w, b, None),
        "plm_kv_fork": lambda s, n=4, w=A, b=ws: P.raw_status("plm_kv_fork", s, A, A, None, n, w, b, None),
        "plm_kv_free": lambda s, n=4, w=A, b=ws: P.raw_status("plm_kv_free", s, A, n, None),
        "plm_kv_compact": lambda s, n=4, w=A, b=ws: P.raw_status("plm_kv_compact", s, None, w, b, None),
        "plm_kv_copy_pages": lambda s, n=4, w=A, b=ws: P.raw_status("plm_kv_copy_pages", s, A, A, n, None),
    }
    for name, call in calls.items():
        st = lambda n=4, w=A, b=ws, **kw: call(ctypes.byref(kv(**kw)), n, w, b)  # noqa: E731
        assert call(None) == BAD
        for bad in (dict(table=None), dict(lens=None), dict(refs=None), dict(pages=0), dict(pages=1 << 31), dict(max_seqs=0),
                    dict(max_pages=0), dict(page_tokens=0)):
            assert st(**bad) == BAD, (name, bad)
        for bad in (dict(table=A + 2), dict(lens=A + 1), dict(refs=A + 2), dict(status=A + 2)):
            assert st(**bad) == MIS, (name, bad)
        if name != "plm_kv_compact":
            assert st(n=-1) == BAD
            assert st(n=0) == P.PLM_OK
        if name in ("plm_kv_reserve", "plm_kv_fork", "plm_kv_compact"):
            assert st(w=None) == BAD and st(b=15) == BAD and st(w=A + 16) == MIS
        if name in ("plm_kv_fork", "plm_kv_compact", "plm_kv_copy_pages"):
            assert st(pool=None) == BAD and st(page_bytes=24) == BAD and st(page_bytes=0) == BAD
            assert st(pool=A + 8) == MIS
    s = ctypes.byref(kv())
    assert P.raw_status("plm_kv_reserve", s, None, A, 4, None, 0, A, ws, None) == BAD
    assert P.raw_status("plm_kv_reserve", s, A, None, 4, None, 0, A, ws, None) == BAD
    assert P.raw_status("plm_kv_reserve", s, A, A, 4, A, 0, A, ws, None) == BAD
    assert P.raw_status("plm_kv_reserve", s, A, A, 4, A + 4, 2, A, ws, None) == MIS
    assert P.raw_status("plm_kv_fork", s, None, A, None, 4, A, ws, None) == BAD
    assert P.raw_status("plm_kv_fork", s, A, A, A + 1, 4, A, ws, None) == MIS


def attn(**kw):
    p = dict(q=A, o=A, lse=None, k=A, v=A, table=A, lens=A, seqs=None, batch=4, tokens=1, heads=16, kv_heads=8,
             head_dim=128, q_token_stride=2048, q_head_stride=128, o_token_stride=2048, o_head_stride=128, page_tokens=16,
             pages=64, page_stride=1 << 15, kv_head_stride=2048, kv_token_stride=128, table_stride=8, rows=4,
             prefix_len=64, max_len=100, scale=0.1, type=2, o_type=2)
    p.update(kw)
    return ctypes.byref(P._AttnProblem(**p))


def test_attention_refusals():
    ws = 1 << 40
    st = lambda w=A, b=ws, **kw: P.raw_status("plm_attn_shared_prefix", attn(**kw), w, b, None)  # noqa: E731
    assert P.raw_status("plm_attn_shared_prefix", None, A, ws, None) == BAD
    for f in ("q", "o", "k", "v", "table", "lens"):
        assert st(**{f: None}) == BAD
    for bad in (dict(batch=-1), dict(batch=1 << 31), dict(tokens=0), dict(heads=0), dict(heads=12), dict(kv_heads=0),
                dict(kv_heads=32), dict(head_dim=0), dict(type=0), dict(type=5), dict(o_type=1), dict(pages=0), dict(rows=0),
                dict(page_tokens=0), dict(table_stride=0), dict(max_len=0), dict(prefix_len=-16), dict(prefix_len=112),
                dict(prefix_len=40), dict(page_stride=-8), dict(batch=1 << 20, tokens=1 << 10)):
        assert st(**bad) == BAD, bad
    for bad in (dict(head_dim=96), dict(page_tokens=8), dict(page_tokens=48, prefix_len=48)):
        assert st(**bad) == UNS, bad
    for bad in (dict(q=A + 8), dict(o=A + 8), dict(k=A + 8), dict(v=A + 8), dict(lse=A + 2), dict(table=A + 2),
                dict(lens=A + 1), dict(seqs=A + 2), dict(q_token_stride=2052), dict(q_head_stride=130), dict(o_token_stride=2052),
                dict(page_stride=4), dict(kv_head_stride=2044), dict(kv_token_stride=129), dict(o_type=0, o_head_stride=126)):
        assert st(**bad) == MIS, bad
    assert st(batch=0) == P.PLM_OK
    size = q.plm_attn_workspace_size
    for bad in ((0, 1, 16, 8, 128, 64, 100), (4, 0, 16, 8, 128, 64, 100), (4, 1, 12, 8, 128, 64, 100),
                (4, 1, 16, 8, 96, 64, 100), (4, 1, 16, 8, 128, 101, 100), (4, 1, 16, 8, 128, 64, 0)):
        assert size(*bad) == 0
    need = size(4, 1, 16, 8, 128, 64, 100)
    if need:
        assert st(b=need - 1) == BAD and st(w=None) == BAD and st(w=A + 16) == MIS


def test_packed_calls_are_the_same_calls():
    # the block form refuses what the entry points refuse, with the same status (nothing is launched)
    import struct
    call = lambda entry, args: P.raw_status("plm_call", entry, args)  # noqa: E731
    assert call(7, b"\0" * 64) == BAD and call(-1, b"\0" * 64) == BAD and call(0, None) == BAD

    def q8(*v):
        return struct.pack("@%dq" % len(v), *v)

    def rope(count=1, pos=A, freqs=A, tokens=4, d=128, rot=128, layout=0, t=None):
        return call(0, struct.pack("@7qd2q", count, pos, freqs, tokens, d, rot, layout, 1.0, 0, 0) + bytes(t or rope_tensor()))
    assert rope(count=0) == BAD and rope(pos=0) == BAD and rope(rot=3) == BAD and rope(layout=2) == BAD
    assert rope(freqs=A + 4) == MIS and rope(t=rope_tensor(x=A + 2)) == MIS and rope(tokens=0) == P.PLM_OK
    ws, s = q.plm_kv_workspace_size(64, 4), bytes(kv())
    assert call(1, q8(A, A, 4, A + 4, 2, A, ws, 0) + s) == MIS and call(1, q8(0, A, 4, 0, 0, A, ws, 0) + s) == BAD
    assert call(1, q8(A, A, 0, 0, 0, A, ws, 0) + s) == P.PLM_OK
    assert call(2, q8(A, A, A + 1, 4, A, ws, 0) + s) == MIS and call(2, q8(A, A, 0, 4, A, 3, 0) + s) == BAD
    assert call(3, q8(A + 2, 4, 0) + s) == MIS and call(3, q8(A, 0, 0) + s) == P.PLM_OK
    assert call(4, q8(A + 2, A, ws, 0) + s) == MIS and call(4, q8(0, 0, ws, 0) + s) == BAD
    assert call(5, q8(A, 0, 4, 0) + s) == BAD and call(5, q8(A, A, 0, 0) + s) == P.PLM_OK
    a = lambda **kw: bytes(P._AttnProblem.from_address(ctypes.addressof(attn(**kw)._obj)))  # noqa: E731
    assert call(6, q8(A, 1 << 40, 0) + a(k=A + 8)) == MIS and call(6, q8(A, 1 << 40, 0) + a(head_dim=96)) == UNS
    assert call(6, q8(A, 1 << 40, 0) + a(batch=0)) == P.PLM_OK


def test_the_bindings_blocks_have_the_structs_layout():
    for ctype, packed in ((P._RopeTensor, P._ROPE_TENSOR), (P._KvState, P._KV_STATE), (P._AttnProblem, P._ATTN_PROBLEM)):
        values = list(range(1, len(ctype._fields_) + 1))
        assert ctypes.sizeof(ctype) == packed.size and bytes(ctype(*values)) == packed.pack(*values)


class Stub:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.nbytes = shape, dtype, math.prod(shape) * 4
        self.strides = [math.prod(shape[i + 1:]) for i in range(len(shape))]

    def stride(self):
        return self.strides

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


def test_arguments_made_ahead_hold_their_tensors():
    # else a temporary's memory may be the next temporary's before the call is made
    import gc
    import weakref
    made = {"x": Stub((4, 2, 64), torch.float32), "y": Stub((9, 2, 16, 64), torch.bfloat16), "slots": Stub((4,), torch.int64),
            "pool": Stub((8, 16), torch.int32), "table": Stub((2, 4), torch.int32), "lens": Stub((2,), torch.int32),
            "refs": Stub((8,), torch.int32), "status": Stub((1,), torch.int32)}
    part = q.plm_rope_tensor(made["x"], made["y"], slots=made["slots"])
    state = q.plm_kv_state(made["pool"], made["table"], made["lens"], made["refs"], 16, made["status"])
    seen = {k: weakref.ref(v) for k, v in made.items()}
    made.clear()
    gc.collect()
    assert [k for k, v in seen.items() if v() is None] == []
    del part, state
    gc.collect()
    assert [k for k, v in seen.items() if v() is not None] == []


def test_page_calls_without_items():
    # a step in which no sequence grows, splits or ends: torch gives an empty list's address as null
    ws, s = q.plm_kv_workspace_size(64, 0), ctypes.byref(kv())
    assert P.raw_status("plm_kv_reserve", s, None, None, 0, None, 0, A, ws, None) == P.PLM_OK
    assert P.raw_status("plm_kv_fork", s, None, None, None, 0, A, ws, None) == P.PLM_OK
    assert P.raw_status("plm_kv_free", s, None, 0, None) == P.PLM_OK
    assert P.raw_status("plm_kv_copy_pages", s, None, None, 0, None) == P.PLM_OK
    for n in (1, -1):   # else the lists are wanted
        assert P.raw_status("plm_kv_reserve", s, None, None, n, None, 0, A, 1 << 30, None) == BAD
        assert P.raw_status("plm_kv_fork", s, None, None, None, n, A, 1 << 30, None) == BAD
        assert P.raw_status("plm_kv_free", s, None, n, None) == BAD
        assert P.raw_status("plm_kv_copy_pages", s, None, A, n, None) == BAD


def test_rope_limits_as_stated():
    # more than 65536 heads together; an odd head size, whatever its rotary part
    def st(*tensors, d=128, rot=128):
        return P.raw_status("plm_rope", (P._RopeTensor * len(tensors))(*tensors), len(tensors), A, A, 0, d, rot, 0, 1.0, 0, None)
    many = lambda n: rope_tensor(heads=n)  # noqa: E731
    assert st(many(65536)) == P.PLM_OK and st(many(65537)) == BAD
    assert st(many(32768), many(32768)) == P.PLM_OK and st(many(32768), many(32769)) == BAD
    assert st(*[many(8192)] * 8) == P.PLM_OK and st(*[many(8193)] * 8) == BAD
    assert st(many(8), d=127, rot=64) == BAD and st(many(8), d=1024, rot=1024) == P.PLM_OK and st(many(8), d=1026, rot=64) == BAD


def test_when_the_prefix_of_many_rows_is_done_apart():
    # more than 96 rows; measured on both sides (csrc/attn.cu).  Done apart, a call needs more workspace than without
    def apart(batch, tokens, group, kv_heads, d, prefix):
        size = lambda p: q.plm_attn_workspace_size(batch, tokens, group * kv_heads, kv_heads, d, p, prefix + tokens + 100)  # noqa: E731
        return size(prefix) != size(0)
    assert not apart(60, 32, 4, 8, 128, 2048) and not apart(96, 70, 7, 8, 128, 15360) and not apart(96, 70, 7, 2, 128, 15360)
    assert not apart(24, 28, 4, 8, 128, 4096) and not apart(60, 28, 4, 8, 64, 2048) and not apart(8, 509, 4, 8, 128, 16384)
    assert apart(24, 35, 4, 8, 128, 8192) and apart(40, 26, 5, 2, 128, 10240) and apart(60, 35, 4, 8, 64, 8192) and apart(60, 25, 4, 2, 128, 32768)


def test_where_the_rows_kernel_ends():
    # 33 to 96 rows; measured on both sides (csrc/attn.cu).  Alone it needs no workspace, the tile kernel does
    size = lambda batch, tokens, d, keys: q.plm_attn_workspace_size(batch, tokens, 32, 8, d, 0, keys)  # noqa: E731
    assert size(24, 8, 128, 90000) == 0 and size(24, 10, 128, 4000) == 0 and size(24, 16, 128, 2000) == 0 and size(5, 20, 128, 500) == 0
    assert size(24, 10, 128, 16000) > 0 and size(24, 16, 128, 3000) > 0 and size(60, 20, 128, 4000) > 0 and size(60, 24, 128, 2000) > 0
    assert size(24, 16, 64, 4000) == 0 and size(24, 20, 64, 1000) == 0 and size(24, 20, 64, 4000) > 0 and size(8, 25, 128, 100) > 0


def test_few_rows_of_very_many_keys_are_not_refused():
    # 2^32 units of the tile kernel by the bound: up to 96 rows there is a kernel without them.  (k is misaligned, which
    # is checked after: nothing is launched)
    st = lambda tokens, **kw: P.raw_status("plm_attn_shared_prefix", attn(batch=1 << 16, rows=1 << 16, tokens=tokens, heads=16,  # noqa: E731
                                           kv_heads=8, prefix_len=0, max_len=1 << 20, k=A + 8, **kw), A, 1 << 50, None)
    for tokens in (1, 16, 20, 48):
        assert st(tokens) == MIS
    assert st(49) == UNS
