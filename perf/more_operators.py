"""What a decode step needs between this package's products, and behind the last, as measurable cases: the residual sum
and norm that make a product's q8_K activations, a cache in 8 bits (written, read back, attended over) and the choice of
the next token.  Inputs as a decoding program has them, the operators in plain torch, and through this package.

Shapes: hidden sizes, head counts and the vocabulary of the Qwen3 checkpoints the repository's matrices come from (1024,
2048 or 4096 wide, 16 or 32 query heads, 8 key/value heads of 128, 151936 tokens), plus generic ones."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 292  # bytes of 256 values as q8_K: f32 scale, 256 codes, 16 sums of 16 codes


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a single stream: a layer's residual sum and norm into the activations of its next product (latency)
        dict(name="norm_decode_1", op="norm", m=1, k=1024, xt="f32", rt="f32", wt="f32", q8=True, yt=""),
        # the same for a prompt of ragged length in a 4096 wide model
        dict(name="norm_prompt_8191", op="norm", m=8191, k=4096, xt="f32", rt="f32", wt="f32", q8=True, yt=""),
        # a decode step's keys and values of 61 streams go into the 8-bit cache and are read back (latency)
        dict(name="kv8_write_61", op="write", tokens=61, hkv=8, d=128, rot=128, half=True, xt="f32", yt="bf16", page=16, base=1e6),
        # a prompt's keys and values, half of each head turned, interleaved pairs, ragged length
        dict(name="kv8_write_8191", op="write", tokens=8191, hkv=8, d=128, rot=64, half=False, xt="f32", yt="f16", page=64, base=1e6),
        # a stored conversation of 333 tokens is read back in 32 bits
        dict(name="kv8_read_333", op="read", tokens=333, hkv=2, d=64, yt="f32", page=16, gone=0.0),
        # many streams' tokens at once, some of their slots gone
        dict(name="kv8_read_48000", op="read", tokens=48000, hkv=8, d=128, yt="bf16", page=64, gone=0.05),
        # four streams, one token each, behind a system prompt of 1024 tokens (latency)
        dict(name="attn8_decode_4", op="attn", batch=4, nq=1, hq=16, hkv=8, d=128, prefix=1024, tail=64, page=16, type="bf16", idle=0),
        # a serving batch of unequal lengths, nothing shared
        dict(name="attn8_decode_128", op="attn", batch=128, nq=1, hq=32, hkv=8, d=128, prefix=0, tail=6000, page=32, type="bf16", idle=2),
        # five drafted tokens of 47 streams are verified at once behind a shared document; heads of 64, seven to a key/value head
        dict(name="attn8_verify_47", op="attn", batch=47, nq=5, hq=14, hkv=2, d=64, prefix=8192, tail=1200, page=32, type="f16", idle=1),
        # eight users' questions of 509 tokens enter behind a shared document
        dict(name="attn8_prompt_8x509", op="attn", batch=8, nq=509, hq=32, hkv=8, d=128, prefix=16384, tail=1021, page=64, type="bf16", idle=0),
        # one stream's next token by temperature and top-p over the whole vocabulary (latency)
        dict(name="sample_1", op="sample", m=1, n=151936, type="f32", spread=3.0, mode="p"),
        # a serving batch whose requests ask for different things: greedy, top-k, top-p, min-p, all of them
        dict(name="sample_256", op="sample", m=256, n=151936, type="f32", spread=2.5, mode="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "write", "read", "attn", "attn", "sample"))
    if op == "norm":
        q8 = rng.random() < 0.6
        k = 256 * _log(rng, 1, 48) if q8 else _log(rng, 8, 12288)
        t = rng.choice(("f32", "f32", "f16", "bf16"))
        return dict(op=op, m=_log(rng, 1, max(1, 33000000 // k)), k=k, xt=t, rt=rng.choice(("", t, t, "f32")), wt=rng.choice(("", "f32", t)), q8=q8,
                    yt=rng.choice(("f32", "f16", "bf16")) if not q8 or rng.random() < 0.2 else "")
    if op in ("write", "read"):
        d, page = rng.choice((64, 128, 128, 32 * rng.randrange(1, 9))), rng.choice((16, 32, 64))
        if op == "read":
            return dict(op=op, tokens=_log(rng, 1, 40000), hkv=rng.choice((1, 2, 5, 8)), d=d, yt=rng.choice(("f32", "f16", "bf16")), page=page,
                        gone=rng.choice((0.0, 0.0, 0.1)))
        return dict(op=op, tokens=_log(rng, 1, 16000), hkv=rng.choice((1, 2, 5, 8)), d=d, rot=rng.choice((d, d, d // 2, 2 * rng.randrange(1, d // 2))),
                    half=rng.random() < 0.5, xt=rng.choice(("f32", "f32", "f16", "bf16")), yt=rng.choice(("f16", "bf16")), page=page, base=rng.choice((1e4, 1e6)))
    if op == "sample":
        return dict(op=op, m=_log(rng, 1, 256), n=_log(rng, 32, 151936), type=rng.choice(("f32", "f32", "f16", "bf16")),
                    spread=rng.uniform(0.5, 5.0), mode=rng.choice(("greedy", "plain", "k", "p", "min", "mixed", "mixed")))
    for _ in range(100):
        hkv = rng.choice((2, 8))
        c = dict(op="attn", batch=_log(rng, 1, 200), nq=rng.choice((1, 1, rng.randrange(2, 9), _log(rng, 9, 700))), hq=hkv * rng.choice((1, 2, 4, 7)),
                 hkv=hkv, d=rng.choice((64, 128)), prefix=0, tail=0, page=rng.choice((16, 32, 64)), type=rng.choice(("bf16", "f16")), idle=0)
        c["prefix"] = rng.choice((0, 0, 1, 1)) * _log(rng, 1, 16384 // c["page"]) * c["page"]
        c["tail"] = c["nq"] + _log(rng, 1, 4000)
        c["idle"] = rng.randrange(0, 1 + c["batch"] // 16)
        most = listed()[9]
        if work(c)["flops"] <= work(most)["flops"] and work(c)["bytes"] <= 1e9 and _scores(c) <= _scores(most):
            return c
    return dict(c, batch=7, nq=1)


def _scores(c):
    return c["batch"] * c["nq"] * c["hq"] * (c["prefix"] + c["tail"])


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["m"] * c["k"]
        moved = n * (SIZE[c["xt"]] + (2 * SIZE[c["rt"]] if c["rt"] else 0) + (SIZE[c["yt"]] if c["yt"] else 0)) + (n // 256 * BLOCK if c["q8"] else 0)
        return {"bytes": moved + (c["k"] * SIZE[c["wt"]] if c["wt"] else 0), "flops": n * (9 if c["q8"] else 6)}
    heads = 2 * c.get("hkv", 0)
    row = c.get("d", 0) * 33 // 32  # bytes of a head's codes and exponents
    if c["op"] == "write":  # written, then read back
        n = c["tokens"] * heads * c["d"]
        return {"bytes": n * (SIZE[c["xt"]] + SIZE[c["yt"]]) + 2 * c["tokens"] * heads * row + c["tokens"] * 12, "flops": n * 5}
    if c["op"] == "read":
        n = c["tokens"] * heads
        return {"bytes": n * (row * (1 - c["gone"]) + c["d"] * SIZE[c["yt"]]) + 8 * c["tokens"], "flops": n * c["d"]}
    if c["op"] == "sample":
        return {"bytes": c["m"] * (c["n"] * SIZE[c["type"]] + 28), "flops": c["m"] * c["n"] * (1 if c["mode"] == "greedy" else 8)}
    g = c["batch"] - c["idle"]
    mean = (c["nq"] + c["tail"]) / 2                 # own tokens of a stream, on average
    seen = c["prefix"] + mean - (c["nq"] - 1) / 2    # keys that a query sees
    return {"bytes": heads * row * (c["prefix"] + g * mean) + c["batch"] * c["nq"] * c["hq"] * (4 * c["d"] + 4) + 4 * g * mean / c["page"],
            "flops": 4 * c["d"] * c["hq"] * g * c["nq"] * seen}


# ------------------------------------------------------------------------------------------------- their inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_norm(c, seed):
    g, shape = _gen(seed), (c["m"], c["k"])
    wide = 1 + 2 * _rand(g, c["k"]).abs() ** 3  # some channels of the residual stream are far larger than most
    s = {"c": c, "x": (0.5 * _rand(g, *shape)).to(TYPES[c["xt"]]), "eps": 1e-6}
    s["weight"] = (1 + 0.2 * _rand(g, c["k"])).to(TYPES[c["wt"]]) if c["wt"] else None
    if c["rt"]:
        s["residual"] = (_rand(g, *shape) * wide).to(TYPES[c["rt"]])
        s["sum"] = torch.empty_like(s["residual"])
    if c["q8"]:
        s["xq"] = torch.empty(c["m"], c["k"] // 256 * BLOCK, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(c["m"], c["k"] // 256, 256, dtype=torch.float16, device="cuda")
    if c["yt"]:
        s["y"] = torch.empty(shape, dtype=TYPES[c["yt"]], device="cuda")
    return s


def _views(pool, hkv, page, d):
    """Codes of keys and values [pages][heads][page][d] and their exponents [pages][heads][page][d / 32] in a pool of bytes:
    a page is the keys' codes, the values' codes, the keys' exponents, the values' exponents."""
    n = hkv * page * d
    at = (0, n, 2 * n, 2 * n + n // 32, 2 * n + n // 16)
    part = [pool[:, a:b].view(-1, hkv, page, d if i < 2 else d // 32) for i, (a, b) in enumerate(zip(at, at[1:]))]
    return part[0].view(torch.int8), part[1].view(torch.int8), part[2], part[3]


def _fill(pool, c, g):
    """The pool as a decoded text leaves it: normal values in blocks of 32, each with its own power of two."""
    ck, cv, ek, ev = _views(pool, c["hkv"], c["page"], c["d"])
    for codes, exps in ((ck, ek), (cv, ev)):
        for i in range(0, codes.shape[0], 1024):
            x = _rand(g, *codes[i:i + 1024].shape)
            e, q = _encode(x)
            codes[i:i + 1024], exps[i:i + 1024] = q, e


def _prepare_cache(c, seed):
    g, t = _gen(seed), c["tokens"]
    n = -(-t // c["page"]) + 5
    s = {"c": c, "pool": torch.zeros(n, 2 * c["hkv"] * c["page"] * c["d"] * 33 // 32, dtype=torch.uint8, device="cuda")}
    pages = torch.randperm(n, generator=g, device="cuda")
    at = torch.arange(t, device="cuda") + c["page"] // 2  # the first page is already half full
    s["slots"] = pages[at // c["page"]] * c["page"] + at % c["page"]
    s["k"], s["v"] = torch.empty(2, t, c["hkv"], c["d"], dtype=TYPES[c["yt"]], device="cuda")
    if c["op"] == "read":
        _fill(s["pool"], c, g)
        if c["gone"]:
            s["slots"][torch.rand(t, generator=g, device="cuda") < c["gone"]] = -1
        return s
    x = _rand(g, t, 2 * c["hkv"] * c["d"]).to(TYPES[c["xt"]]).view(t, -1, c["d"])  # one product's rows
    s["xk"], s["xv"] = x[:, :c["hkv"]], x[:, c["hkv"]:]
    freqs = [int(round(c["base"] ** (-2.0 * i / c["rot"]) / (2 * math.pi) * 2.0 ** 64)) for i in range(c["rot"] // 2)]
    s["freqs"] = torch.tensor(freqs, dtype=torch.int64).cuda()  # 64-bit fractions of a turn
    start = torch.randint(0, 32768, (1,), generator=g, device="cuda")
    s["positions"] = (start + torch.arange(t, device="cuda") % 2048).to(torch.int32)  # several streams, one after the other
    return s


def _prepare_attn(c, seed):
    g, r = _gen(seed), random.Random(seed)
    b, ps, shared = c["batch"], c["page"], c["prefix"] // c["page"]
    mine = [r.randrange(c["nq"], c["tail"] + 1) for _ in range(b)]
    lens = [c["prefix"] + v for v in mine]
    for i in r.sample(range(1, b), c["idle"]) if c["idle"] else ():
        lens[i] = mine[i] = 0
    width = shared + -(-c["tail"] // ps)
    order = list(range(shared + sum(-(-v // ps) for v in mine) + 3))
    r.shuffle(order)
    pages = len(order)
    prefix, table = [order.pop() for _ in range(shared)], []
    for v, n in zip(mine, lens):
        k = -(-v // ps)
        table.append((prefix if n else [-1] * shared) + [order.pop() for _ in range(k)] + [-1] * (width - shared - k))
    pool = torch.empty(pages, 2 * c["hkv"] * ps * c["d"] * 33 // 32, dtype=torch.uint8, device="cuda")
    _fill(pool, c, g)
    q = (2.5 * _rand(g, b * c["nq"], c["hq"], c["d"])).to(TYPES[c["type"]])  # scores spread as a trained head's
    return {"c": c, "q": q, "pool": pool, "o": torch.empty_like(q), "lse": torch.empty(b * c["nq"], c["hq"], device="cuda"),
            "most": max(max(lens), 1), "scale": c["d"] ** -0.5, "table": torch.tensor(table, dtype=torch.int32).cuda(),
            "lens": torch.tensor(lens, dtype=torch.int32).cuda()}


def _prepare_sample(c, seed):
    g, r, m = _gen(seed), random.Random(seed), c["m"]
    x = c["spread"] * _rand(g, m, c["n"])
    some = torch.randint(0, c["n"], (m, 8), generator=g, device="cuda")
    x.scatter_add_(1, some, c["spread"] * _rand(g, m, 8).abs() * 2)  # what the text makes likely
    rows = []
    for i in range(m):
        mode = ("greedy", "plain", "k", "p", "min", "all")[r.randrange(6)] if c["mode"] == "mixed" else c["mode"]
        rows.append((0.0 if mode == "greedy" else r.choice((0.6, 0.7, 0.8, 1.0, 1.3)),
                     r.choice((1, 20, 40, 50, 200)) if mode in ("k", "all") else 0,
                     r.choice((0.5, 0.8, 0.9, 0.95)) if mode in ("p", "all") else 1.0,
                     r.choice((0.02, 0.05, 0.1)) if mode in ("min", "all") else 0.0))
    t, k, p, low = zip(*rows)
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).cuda()  # noqa: E731
    return {"c": c, "logits": x.to(TYPES[c["type"]]), "temperature": f32(t), "top_k": torch.tensor(k, dtype=torch.int32).cuda(), "top_p": f32(p),
            "min_p": f32(low), "u": torch.rand(m, generator=g, device="cuda"), "tokens": torch.empty(m, dtype=torch.int32, device="cuda"),
            "prob": torch.empty(m, device="cuda")}


PREPARE = {"norm": _prepare_norm, "write": _prepare_cache, "read": _prepare_cache, "attn": _prepare_attn, "sample": _prepare_sample}


def prepare(case, seed):
    return PREPARE[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------------- plain forms
def _q8k(y):
    """The values that y [m][k], in 32 bits, has as q8_K: per 256 values codes of -128 / (the first of the largest ones)."""
    y = y.view(y.shape[0], -1, 256)
    size = y.abs()
    top = size.amax(-1, keepdim=True)
    place = torch.where(size == top, torch.arange(256, device=y.device), 256).amin(-1, keepdim=True)
    first = torch.gather(y, -1, place)
    turn = -128.0 / torch.where(first == 0, 1.0, first)
    codes = torch.clamp(torch.round(turn * y), max=127.0)
    return torch.where(first == 0, 0.0, codes * (1.0 / turn))


def _plain_norm(s):
    c, out = s["c"], {}
    h = s["x"].float()
    if c["rt"]:
        s["sum"].copy_(h + s["residual"].float())
        h, out["sum"] = s["sum"].float(), s["sum"]
    y = h * (1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + s["eps"]))
    if c["wt"]:
        y = y * s["weight"].float()
    if c["q8"]:
        s["values"].copy_(_q8k(y))
        out["xq"] = s["values"]
    if c["yt"]:
        s["y"].copy_(y)
        out["y"] = s["y"]
    return out


def _encode(x):
    """Exponents and codes of x [..][d] in blocks of 32: value = code 2^(e - 127), 2^(e - 127) the smallest power of two
    with |code| <= 127 after rounding."""
    x = torch.clamp(torch.nan_to_num(x, nan=0.0, posinf=2.0 ** 120, neginf=-2.0 ** 120), -2.0 ** 120, 2.0 ** 120)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    e = torch.clamp((bits >> 23) - 6 + ((bits & 0x7FFFFF) >= 0x7F0000).int(), min=27)
    e = torch.where(bits == 0, 0, e)
    back = ((254 - e) << 23).view(torch.float32)  # 2^(127 - e)
    return e.to(torch.uint8), torch.round(b * torch.where(e == 0, 0.0, back)[..., None]).view(x.shape).to(torch.int8)


def _decode(codes, exps):
    size = (exps.int() << 23).view(torch.float32)  # 2^(e - 127), and 0 for 0
    return (codes.float().view(*exps.shape, 32) * size[..., None]).view(codes.shape)


def _turned(x, cos, sin, rot, half):
    """x [tokens][heads][d] in 32 bits, its first `rot` values turned by pairs."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_cache(s):
    c = s["c"]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    parts = _views(s["pool"], c["hkv"], c["page"], c["d"])
    if c["op"] == "write":
        part = s["positions"].long()[:, None] * s["freqs"]  # wraps at whole turns
        angle = (part >> 32).float() * (2 * math.pi / 2.0 ** 32)
        k = _turned(s["xk"].float(), angle.cos(), angle.sin(), c["rot"], c["half"])
        for x, codes, exps in ((k, parts[0], parts[2]), (s["xv"].float(), parts[1], parts[3])):
            e, q = _encode(x)
            codes[page, :, at], exps[page, :, at] = q, e
    there = (s["slots"] >= 0)[:, None, None]
    for y, codes, exps in ((s["k"], parts[0], parts[2]), (s["v"], parts[1], parts[3])):
        y.copy_(torch.where(there, _decode(codes[page, :, at], exps[page, :, at]), 0.0))
    return {"k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c, g, ps = s["c"], s["c"]["hq"] // s["c"]["hkv"], s["c"]["page"]
    b, nq, hkv, d, prefix = c["batch"], c["nq"], c["hkv"], c["d"], c["prefix"]
    ck, cv, ek, ev = _views(s["pool"], hkv, ps, d)
    q = s["q"].float().view(b, nq, hkv, g, d).permute(2, 0, 1, 3, 4).reshape(hkv, b, nq * g, d) * s["scale"]
    seen = (s["lens"].long()[:, None] - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0)  # keys that a query sees
    seen = seen.repeat_interleave(g, 1)                                                         # [b][nq g]

    def gather(codes, exps, pages):  # [n][pages] -> [hkv][n][tokens][d]
        return _decode(codes[pages], exps[pages]).permute(2, 0, 1, 3, 4).reshape(hkv, pages.shape[0], -1, d)

    shared, rest = s["table"][:1, :prefix // ps].long(), s["table"][:, prefix // ps:].long().clamp(min=0)
    token = torch.arange(prefix + rest.shape[1] * ps, device="cuda")
    hidden = token >= seen[..., None]                                                           # [b][nq g][tokens]
    scores = torch.matmul(q.reshape(hkv, b * nq * g, d), gather(ck, ek, shared)[:, 0].transpose(-1, -2)).view(hkv, b, nq * g, prefix)
    scores = torch.cat((scores, torch.matmul(q, gather(ck, ek, rest).transpose(-1, -2))), -1).masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores[..., prefix:], gather(cv, ev, rest))
    o += torch.matmul(scores[..., :prefix].reshape(hkv, b * nq * g, prefix), gather(cv, ev, shared)[:, 0]).view_as(o)
    o /= torch.where(total == 0, 1.0, total)
    lse = total.log() + top
    s["o"].copy_(o.view(hkv, b, nq, g, d).permute(1, 2, 0, 3, 4).reshape(b * nq, -1, d))
    s["lse"].copy_(lse.view(hkv, b, nq, g).permute(1, 2, 0, 3).reshape(b * nq, -1))
    return {"o": s["o"], "lse": s["lse"]}


def _plain_sample(s):
    """In 64 bits: which tokens are kept, and which one is met, turns on sums next to a border."""
    x = s["logits"].double()
    n, hot = x.shape[1], s["temperature"].double()[:, None]
    top = x.amax(-1, keepdim=True)
    w = torch.exp((x - top) / torch.where(hot > 0, hot, 1.0))
    sorted_w, order = torch.sort(s["logits"].float(), descending=True, stable=True, dim=-1)  # ties: lowest index first
    sorted_w = torch.gather(w, -1, order)
    most = s["top_k"].long()[:, None]
    sorted_w = torch.where((torch.arange(n, device="cuda") < most) | (most <= 0), sorted_w, 0.0)
    before = torch.cumsum(sorted_w, -1) - sorted_w
    p = s["top_p"].double()[:, None]
    keep = (before < p * sorted_w.sum(-1, keepdim=True)) | (p >= 1.0)
    keep[:, 0] = True
    keep &= (sorted_w > 0) & (sorted_w >= s["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(-1, order, torch.where(keep, sorted_w, 0.0))
    up = torch.cumsum(w, -1)
    met = torch.where(up > s["u"].double()[:, None] * up[:, -1:], torch.arange(n, device="cuda"), n).amin(-1)
    first = torch.where(x == top, torch.arange(n, device="cuda"), n).amin(-1)
    token = torch.where(hot[:, 0] > 0, met, first)
    s["tokens"].copy_(token)
    s["prob"].copy_(torch.where(hot[:, 0] > 0, torch.gather(w, -1, token[:, None])[:, 0] / up[:, -1], 1.0))
    return {"tokens": s["tokens"], "prob": s["prob"]}


PLAIN = {"norm": _plain_norm, "write": _plain_cache, "read": _plain_cache, "attn": _plain_attn, "sample": _plain_sample}


# ------------------------------------------------------------------------------------------- through the package
def _own(s):
    import quant_packed_gemv_gb300 as qp
    c = s["c"]
    if c["op"] == "norm":
        qp.plm_rmsnorm(s["x"], s["weight"], s["eps"], residual=s.get("residual"), sum=s.get("sum"), xq=s.get("xq"), y=s.get("y"))
        out = {n: s[n] for n in ("sum", "y") if n in s}
        if c["q8"]:  # the values that the blocks stand for
            blocks = s["xq"].view(c["m"], -1, BLOCK)
            torch.mul(blocks[..., 4:260].view(torch.int8), blocks.view(torch.float32)[..., :1], out=s["values"])
            out["xq"] = s["values"]
        return out
    if c["op"] == "sample":
        qp.plm_sample(s["logits"], s["tokens"], u=s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                      prob=s["prob"])
        return {"tokens": s["tokens"], "prob": s["prob"]}
    ck, cv, ek, ev = qp.plm_kv8_views(s["pool"], c["hkv"], c["page"], c["d"])
    if c["op"] == "attn":
        if "workspace" not in s:  # kept by the program for all its calls
            need = qp.plm_attn_kv8_workspace_size(c["batch"], c["nq"], c["hq"], c["hkv"], c["d"], c["prefix"], s["most"])
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        qp.plm_attn_kv8(s["q"], s["o"], ck, cv, ek, ev, s["table"], s["lens"], c["nq"], c["prefix"], s["most"], s["scale"], s["workspace"],
                        lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "write":
        qp.plm_kv8_write([qp.plm_kv8_tensor(s["xk"], ck, ek, s["slots"]), qp.plm_kv8_tensor(s["xv"], cv, ev, s["slots"], rotate=False)],
                         s["positions"], s["freqs"], c["rot"], "half" if c["half"] else "interleaved")
    qp.plm_kv8_read([qp.plm_kv8_tensor(s["k"], ck, ek, s["slots"]), qp.plm_kv8_tensor(s["v"], cv, ev, s["slots"])])
    return {"k": s["k"], "v": s["v"]}


def run(state):
    return _own(state) if own else PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------------- definitions in 64 bits
def _exact_norm(c, s):
    out, h = {}, s["x"].double()
    if c["rt"]:
        h = h + s["residual"].double()
        out["sum"] = h
        h = h.to(s["residual"].dtype).double()  # the norm is of the sum as it is stored
    y = h / (h.pow(2).sum(-1, keepdim=True) / c["k"] + s["eps"]).sqrt()
    if c["wt"]:
        y = y * s["weight"].double()
    if c["q8"]:
        b = y.reshape(-1, 256)
        big = b.gather(1, b.abs().argmax(1, keepdim=True))
        step = big / -128
        out["xq"] = torch.where(step == 0, 0.0, (b / step).round().clamp(max=127) * step).view(c["m"], -1, 256)
    if c["yt"]:
        out["y"] = y
    return out


def _exact_cache(c, s):
    out, there = {}, s["slots"] >= 0
    page, at = s["slots"][there] // c["page"], s["slots"][there] % c["page"]
    for name, i in (("k", 0), ("v", 1)):
        if c["op"] == "write":
            x = s["x" + name].double()
            if name == "k":
                w = torch.tensor([c["base"] ** (-2.0 * j / c["rot"]) for j in range(c["rot"] // 2)], dtype=torch.float64, device="cuda")
                turn = torch.polar(torch.ones_like(w), s["positions"].double()[:, None] * w)[:, None]
                one = slice(0, c["rot"] // 2) if c["half"] else slice(0, c["rot"], 2)
                two = slice(c["rot"] // 2, c["rot"]) if c["half"] else slice(1, c["rot"], 2)
                z, x = torch.complex(x[..., one], x[..., two]) * turn, x.clone()
                x[..., one], x[..., two] = z.real, z.imag
            b = x.view(*x.shape[:-1], -1, 32)
            top = b.abs().amax(-1, keepdim=True)
            step = 2.0 ** torch.floor(torch.log2(torch.where(top == 0, 1.0, top) / 127.5) + 1)
            out[name] = ((b / step).round() * step).view(x.shape)
        else:
            codes, exps = (t.permute(0, 2, 1, 3) for t in (_views(s["pool"], c["hkv"], c["page"], c["d"])[j] for j in (i, i + 2)))
            values = codes[page, at].double().view(-1, c["hkv"], c["d"] // 32, 32) * 2.0 ** (exps[page, at].double() - 127)[..., None]
            out[name] = torch.zeros(c["tokens"], c["hkv"], c["d"], dtype=torch.float64, device="cuda")
            out[name][there] = values.view(-1, c["hkv"], c["d"])
    return out


def _exact_attn(c, s):
    o = torch.zeros(c["batch"], c["nq"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["nq"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group, views = c["hq"] // c["hkv"], _views(s["pool"], c["hkv"], c["page"], c["d"])
    q = s["q"].view(c["batch"], c["nq"], c["hq"], c["d"])
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        late = torch.arange(n, device="cuda")[None] > torch.arange(n - c["nq"], n, device="cuda")[:, None]
        for h in range(c["hkv"]):
            k, v = ((views[i][pages, h].double().view(-1, c["d"] // 32, 32) * 2.0 ** (views[i + 2][pages, h].double().view(-1, c["d"] // 32, 1) - 127))
                    .view(-1, c["d"])[:n] for i in (0, 1))
            x = torch.einsum("thd,nd->htn", q[b, :, h * group:(h + 1) * group].double(), k) * s["scale"]
            x = x.masked_fill(late, -math.inf)
            total = torch.logsumexp(x, -1)
            lse[b, :, h * group:(h + 1) * group] = total.T
            o[b, :, h * group:(h + 1) * group] = torch.einsum("htn,nd->thd", (x - total[..., None]).exp(), v)
    return {"o": o.view(-1, c["hq"], c["d"]), "lse": lse.view(-1, c["hq"])}


def _exact_sample(c, s):
    tokens, probs = [], []
    params = [s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p", "u")]
    for i, (t, k, p, low, u) in enumerate(zip(*params)):
        x = s["logits"][i].double()
        if t <= 0:
            tokens.append(int((x == x.max()).nonzero()[0, 0]))
            probs.append(1.0)
            continue
        order = torch.argsort(x, descending=True, stable=True)[:k if k > 0 else c["n"]]
        w = ((x[order] - x[order[0]]) / t).exp()
        if p < 1:
            mass = w.cumsum(0)
            count = max(1, int((mass - w < p * w.sum()).sum()))
            order, w = order[:count], w[:count]
        order, w = order[w >= low], w[w >= low]
        order, back = order.sort()
        mass = w[back].cumsum(0)
        j = min(int((mass <= u * mass[-1]).sum()), order.numel() - 1)
        tokens.append(int(order[j]))
        probs.append(float(w[back][j] / mass[-1]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "prob": torch.tensor(probs, dtype=torch.float64)}


def exact(case, seed):
    how = {"norm": _exact_norm, "write": _exact_cache, "read": _exact_cache, "attn": _exact_attn, "sample": _exact_sample}
    return how[case["op"]](case, prepare(case, seed))
