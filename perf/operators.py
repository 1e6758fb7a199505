"""The attention-side operators (rotary positions, cache pages, attention over a shared prefix) as measurable
cases: inputs as a decoding program has them, the operators in plain torch, and through this package.

Shapes: head counts and sizes of the Qwen3 checkpoints the repository's matrices come from (16 or 32 query heads,
8 key/value heads, heads of 128, 28 or 36 layers), plus generic ones (heads of 64, 2 key/value heads)."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a single stream: q, k, v of a 16-head layer turned and put into the cache (latency)
        dict(name="rope_decode_1", op="rope", tokens=1, hq=16, hkv=8, d=128, rot=128, half=True, xt="f32", yt="bf16",
             cache=True, page=16, inverse=False, base=1e6, factor=1.0),
        # a prompt's q, k, v, stretched frequencies, half of each head turned, interleaved pairs, ragged length
        dict(name="rope_prompt_8191", op="rope", tokens=8191, hq=32, hkv=8, d=128, rot=64, half=False, xt="f32",
             yt="bf16", cache=True, page=64, inverse=False, base=1e6, factor=4.0),
        # the gradient of q and k of a training batch: the inverse rotation
        dict(name="rope_grad_16381", op="rope", tokens=16381, hq=32, hkv=8, d=128, rot=128, half=True, xt="bf16",
             yt="bf16", cache=False, page=0, inverse=True, base=1e4, factor=1.0),
        # a decode step's page bookkeeping: every one of 61 streams grows by one token
        dict(name="reserve_decode_61", op="reserve", pages=8192, words=4, page=16, seqs=64, items=61, longest=1500, grow=1),
        # 37 prompts, each forked into 8 samples; the page is all 28 layers of 8 heads of 128, keys and values, 16 tokens
        dict(name="fork_37x8", op="fork", pages=3000, words=458752, page=16, seqs=512, items=37, each=8, longest=1000),
        # 300 of 512 streams end and give their pages back
        dict(name="free_300", op="free", pages=65536, words=4, page=16, seqs=512, items=300, longest=2000),
        # a pool left half full by departed streams is packed so that its tail can be given back
        dict(name="compact_3000", op="compact", pages=3000, words=458752, page=16, seqs=256, live=0.55),
        # four streams, one token each, behind a system prompt of 1024 tokens (latency)
        dict(name="attn_decode_4", op="attn", batch=4, nq=1, hq=16, hkv=8, d=128, prefix=1024, tail=64, page=16,
             type="bf16", idle=0),
        # a middling batch: odd sizes, heads of 64, seven query heads to a key/value head, some streams idle
        dict(name="attn_decode_61", op="attn", batch=61, nq=1, hq=14, hkv=2, d=64, prefix=8176, tail=900, page=16,
             type="f16", idle=3),
        # five drafted tokens of 48 streams are verified at once
        dict(name="attn_verify_48", op="attn", batch=48, nq=5, hq=32, hkv=8, d=128, prefix=8192, tail=1200, page=32,
             type="bf16", idle=1),
        # a full serving batch behind a long shared document
        dict(name="attn_decode_256", op="attn", batch=256, nq=1, hq=32, hkv=8, d=128, prefix=32768, tail=2000, page=64,
             type="bf16", idle=2),
        # eight users' questions of 509 tokens enter behind a shared document
        dict(name="attn_prompt_8x509", op="attn", batch=8, nq=509, hq=32, hkv=8, d=128, prefix=16384, tail=1021, page=64,
             type="bf16", idle=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "pages", "pages", "attn", "attn", "attn"))
    if op == "rope":
        d = rng.choice((64, 128))
        cache = rng.random() < 0.6
        xt, yt = rng.choice((("f32", "bf16"), ("f32", "f16"), ("f32", "f32"), ("bf16", "bf16"), ("f16", "f16")))
        return dict(op="rope", tokens=_log(rng, 1, 16000), hq=rng.choice((8, 14, 16, 32)), hkv=rng.choice((2, 8)), d=d,
                    rot=rng.choice((d, d, d // 2, 2 * rng.randrange(1, d // 2))), half=rng.random() < 0.5, xt=xt, yt=yt,
                    cache=cache, page=rng.choice((16, 32, 64)) if cache else 0, inverse=not cache and rng.random() < 0.6,
                    base=rng.choice((1e4, 1e6)), factor=rng.choice((1.0, 1.0, 4.0, 8.0)))
    if op == "pages":
        op = rng.choice(("reserve", "fork", "free", "compact"))
        page = rng.choice((16, 32, 64))
        if op == "compact":
            return dict(op=op, pages=_log(rng, 64, 3000), words=1024 * rng.randrange(1, 449), page=page, seqs=rng.randrange(8, 257),
                        live=rng.uniform(0.2, 0.9))
        if op == "fork":
            return dict(op=op, pages=3000, words=4 * _log(rng, 64, 114688), page=page, seqs=512, items=_log(rng, 1, 40),
                        each=rng.randrange(1, 9), longest=_log(rng, 17, 1000))
        n = _log(rng, 1, 500)
        return dict(op=op, pages=_log(rng, 16000, 65536) if op == "reserve" else 65536, words=4, page=page, seqs=512, items=n,
                    longest=_log(rng, 17, 250 if op == "reserve" else 2000), **({"grow": _log(rng, 1, 200)} if op == "reserve" else {}))
    for _ in range(100):
        hkv = rng.choice((2, 8))
        c = dict(op="attn", batch=_log(rng, 1, 256), nq=rng.choice((1, 1, rng.randrange(2, 9), _log(rng, 9, 700))), hq=hkv * rng.choice((1, 2, 4, 7)),
                 hkv=hkv, d=rng.choice((64, 128)), prefix=0, tail=0, page=rng.choice((16, 32, 64)), type=rng.choice(("bf16", "f16")), idle=0)
        c["prefix"] = rng.choice((0, 1, 1, 1)) * _log(rng, 1, 32768 // c["page"]) * c["page"]
        c["tail"] = c["nq"] + _log(rng, 1, 2000)
        c["idle"] = rng.randrange(0, 1 + c["batch"] // 16)
        w, most = work(c), work(listed()[-1])
        if w["flops"] <= most["flops"] and w["bytes"] <= 1.5e9 and _scores(c) <= _scores(listed()[-1]):
            return c
    return dict(c, batch=7, nq=1)


def _scores(c):
    return c["batch"] * c["nq"] * c["hq"] * (c["prefix"] + c["tail"])


def work(case):
    c = case
    if c["op"] == "rope":
        heads = c["hq"] + (2 if c["cache"] else 1) * c["hkv"]
        turned = c["hq"] + c["hkv"]
        per = SIZE[c["xt"]] + SIZE[c["yt"]]
        return {"bytes": c["tokens"] * (heads * c["d"] * per + 12) + c["rot"] * 4, "flops": c["tokens"] * turned * c["rot"] * 3}
    if c["op"] == "attn":
        g = c["batch"] - c["idle"]
        mean = (c["nq"] + c["tail"]) / 2 + (c["nq"] == 1) * 0.5  # own tokens of a stream, on average
        seen = c["prefix"] + mean - (c["nq"] - 1) / 2            # keys that a query sees
        kv = 2 * c["hkv"] * c["d"] * 2
        return {"bytes": kv * (c["prefix"] + g * mean) + 4 * c["batch"] * c["nq"] * c["hq"] * (c["d"] + 1) + 4 * g * mean / c["page"],
                "flops": 4 * c["d"] * c["hq"] * g * c["nq"] * seen}
    meta = 4 * c["pages"]
    row = c.get("longest", 0) / 2 / c["page"]  # pages of a stream
    if c["op"] == "reserve":
        return {"bytes": meta + c["items"] * (16 + 8 * c["grow"]), "flops": c["items"]}
    if c["op"] == "free":
        return {"bytes": c["items"] * (8 + row * 16), "flops": c["items"] * row}
    if c["op"] == "fork":
        n = c["items"] * c["each"]
        return {"bytes": meta + n * (16 + row * 12) + n * (1 - 1 / c["page"]) * 2 * 4 * c["words"], "flops": n * row}
    moved = c["pages"] * c["live"] * (1 - c["live"])
    return {"bytes": 8 * moved * c["words"] + 3 * meta + 8 * c["pages"] * c["live"], "flops": c["pages"]}


# ------------------------------------------------------------------------------------------------- their inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _frequencies(rot, base, factor):
    """Radians per position of each pair. factor > 1: trained on 4096 positions, stretched `factor` times; pairs that
    turn often keep their frequency, slow ones are divided by the factor, those between are blended."""
    found = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        turns = 4096 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0))) if factor > 1 else 1.0
        found.append(f * keep + f / factor * (1 - keep))
    return found, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _fraction(f):
    """f radians as a 64-bit fraction of a turn (as a signed number of the same bits)."""
    v = int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64
    return v - 2 ** 64 if v >= 2 ** 63 else v


def _prepare_rope(c, seed):
    g, t, d = _gen(seed), c["tokens"], c["d"]
    freqs, mscale = _frequencies(c["rot"], c["base"], c["factor"])
    hv = c["hkv"] if c["cache"] else 0
    x = torch.randn(t, (c["hq"] + c["hkv"] + hv) * d, generator=g, device="cuda").to(TYPES[c["xt"]])  # one product's rows
    x = x.view(t, -1, d)
    s = {"c": c, "mscale": mscale, "q": x[:, :c["hq"]], "k": x[:, c["hq"]:c["hq"] + c["hkv"]], "v": x[:, c["hq"] + c["hkv"]:],
         "freqs": torch.tensor([_fraction(f) for f in freqs], device="cuda"),
         "yq": torch.empty(t, c["hq"], d, dtype=TYPES[c["yt"]], device="cuda")}
    if t == 1:
        s["positions"] = torch.randint(0, 40000, (1,), generator=g, device="cuda", dtype=torch.int32)
    else:  # several streams' tokens, one after the other
        start = torch.randint(0, 32768, (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(t, device="cuda") % 2048).to(torch.int32)
    if c["cache"]:
        n = -(-t // c["page"]) + 5
        s["pool"] = torch.zeros(n, 2, c["hkv"], c["page"], d, dtype=TYPES[c["yt"]], device="cuda")
        pages = torch.randperm(n, generator=g, device="cuda")
        at = torch.arange(t, device="cuda") + c["page"] // 2  # the first page is already half full
        s["slots"] = pages[at // c["page"]] * c["page"] + at % c["page"]
    else:
        s["yk"] = torch.empty(t, c["hkv"], d, dtype=TYPES[c["yt"]], device="cuda")
    return s


def _prepare_pages(c, seed):
    r, g = random.Random(seed), _gen(seed)
    n, ps = c["pages"], c["page"]
    lens, free = [0] * c["seqs"], list(range(n))
    r.shuffle(free)
    s = {"c": c}
    if c["op"] == "compact":
        mean, left, items = n * c["live"] / c["seqs"], int(n * c["live"]), []
        width = int(2 * mean) + 2
        for i in range(c["seqs"]):
            k = min(left, r.randrange(width))
            lens[i], left = k * ps - r.randrange(ps) if k else 0, left - k
    else:
        width = -(-c["longest"] // ps) + -(-c.get("grow", 0) // ps) + 1
        items = r.sample(range(c["seqs"] if c["op"] != "fork" else 64), c["items"])
        for i in items if c["op"] != "free" else range(c["seqs"]):
            lens[i] = r.randrange(c["longest"] // 2, c["longest"] + 1)
    table = [[-1] * width for _ in lens]
    for i, v in enumerate(lens):
        k = -(-v // ps)
        shared = table[i - 1][:k // 2] if c["op"] == "free" and i % 2 else []  # every other stream is a fork of the one before
        shared = [p for p in shared if p >= 0]
        table[i][:k] = shared + [free.pop() for _ in range(k - len(shared))]
    refs = [0] * n
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    meta = [p for row in table for p in row] + lens + refs + [0, 0]
    s["start"] = torch.tensor(meta, dtype=torch.int32).cuda()
    s["meta"] = s["start"].clone()
    a, b = c["seqs"] * width, c["seqs"] * (width + 1)
    s["table"], s["lens"], s["refs"] = s["meta"][:a].view(c["seqs"], width), s["meta"][a:b], s["meta"][b:b + n]
    s["status"], s["live"] = s["meta"][b + n:b + n + 1], s["meta"][b + n + 1:]
    s["pool"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, c["words"]), generator=g, device="cuda", dtype=torch.int32)
    if c["op"] == "fork":
        parents = [i for i in items for _ in range(c["each"])]
        children = r.sample(range(64, c["seqs"]), len(parents))
        s["parents"], s["children"] = (torch.tensor(v, dtype=torch.int32).cuda() for v in (parents, children))
    elif items:
        s["items"] = torch.tensor(items, dtype=torch.int32).cuda()
    if c["op"] == "reserve":
        add = [r.randrange(1, c["grow"] + 1) for _ in items]
        s["add"] = torch.tensor(add, dtype=torch.int32).cuda()
        s["slots"] = torch.empty(len(items), c["grow"], dtype=torch.int64, device="cuda")
    return s


def _prepare_attn(c, seed):
    g, r = _gen(seed), random.Random(seed)
    b, ps, shared = c["batch"], c["page"], c["prefix"] // c["page"]
    own = [r.randrange(c["nq"], c["tail"] + 1) for _ in range(b)]
    lens = [c["prefix"] + v for v in own]
    for i in r.sample(range(1, b), c["idle"]) if c["idle"] else ():
        lens[i] = own[i] = 0
    width = shared + -(-c["tail"] // ps)
    order = list(range(shared + sum(-(-v // ps) for v in own) + 3))
    r.shuffle(order)
    pages = len(order)
    prefix, table = [order.pop() for _ in range(shared)], []
    for v, n in zip(own, lens):
        k = -(-v // ps)
        table.append((prefix if n else [-1] * shared) + [order.pop() for _ in range(k)] + [-1] * (width - shared - k))
    t = TYPES[c["type"]]
    pool = torch.empty(pages, 2, c["hkv"], ps, c["d"], dtype=t, device="cuda")
    pool.normal_(generator=g)
    q = (2.5 * torch.randn(b * c["nq"], c["hq"], c["d"], generator=g, device="cuda")).to(t)  # scores spread as a trained head's
    return {"c": c, "q": q, "pool": pool, "k": pool[:, 0], "v": pool[:, 1], "o": torch.empty_like(q),
            "lse": torch.empty(b * c["nq"], c["hq"], device="cuda"), "most": max(lens), "scale": c["d"] ** -0.5,
            "table": torch.tensor(table, dtype=torch.int32).cuda(), "lens": torch.tensor(lens, dtype=torch.int32).cuda()}


def prepare(case, seed):
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    return _prepare_attn(case, seed) if case["op"] == "attn" else _prepare_pages(case, seed)


# --------------------------------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, half):
    """x [tokens][heads][d] in 32 bits, its first `rot` values turned by pairs."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["c"]
    part = s["positions"].long()[:, None] * s["freqs"]              # wraps at whole turns
    angle = (part >> 32).float() * (2 * math.pi / 2.0 ** 32)
    cos, sin = angle.cos() * s["mscale"], angle.sin() * (-s["mscale"] if c["inverse"] else s["mscale"])
    s["yq"].copy_(_turn(s["q"].float(), cos, sin, c["rot"], c["half"]))
    k = _turn(s["k"].float(), cos, sin, c["rot"], c["half"])
    if not c["cache"]:
        s["yk"].copy_(k)
        return {"q": s["yq"], "k": s["yk"]}
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    s["pool"][page, 0, :, at] = k.to(s["pool"].dtype)
    s["pool"][page, 1, :, at] = s["v"].to(s["pool"].dtype)
    return {"q": s["yq"], "pool": s["pool"]}


def _first_free(refs):
    """The free pages in ascending order, then padding."""
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    found = torch.zeros(refs.numel() + 1, dtype=torch.int64, device="cuda")
    found[torch.where(free, rank, refs.numel())] = torch.arange(refs.numel(), device="cuda")
    return found


def _plain_reserve(s):
    c, table, refs = s["c"], s["table"], s["refs"]
    seqs, add, ps, width = s["items"].long(), s["add"].long(), c["page"], table.shape[1]
    old = s["lens"].long()[seqs]
    have = (old + ps - 1) // ps
    need = (old + add + ps - 1) // ps - have
    first = torch.cumsum(need, 0) - need
    k = torch.arange(-(-c["grow"] // ps) + 1, device="cuda")
    wanted = k < need[:, None]
    page = _first_free(refs)[torch.where(wanted, first[:, None] + k, refs.numel())]
    at = (seqs * width + have)[:, None] + k
    padded = torch.cat((table.flatten(), table.new_zeros(1)))
    padded[torch.where(wanted, at, table.numel())] = page.int()
    table.copy_(padded[:-1].view_as(table))
    counts = torch.cat((refs, refs.new_zeros(1)))
    counts[torch.where(wanted, page, refs.numel())] = 1
    refs.copy_(counts[:-1])
    s["lens"][seqs] = (old + add).int()
    j = torch.arange(c["grow"], device="cuda")
    pos = old[:, None] + j
    slot = table[seqs[:, None], torch.clamp(pos // ps, max=width - 1)].long() * ps + pos % ps
    s["slots"].copy_(torch.where(j < add[:, None], slot, -1))
    return {"meta": s["meta"], "slots": s["slots"]}


def _plain_fork(s):
    c, table, refs, pool = s["c"], s["table"], s["refs"], s["pool"]
    parents, children, ps = s["parents"].long(), s["children"].long(), c["page"]
    length = s["lens"].long()[parents]
    full, part = length // ps, (length % ps) > 0
    fresh = _first_free(refs)[torch.cumsum(part, 0) - 1]
    col = torch.arange(table.shape[1], device="cuda")
    rows = table[parents]
    shared = col < full[:, None]
    last = torch.gather(rows, 1, torch.clamp(full, max=table.shape[1] - 1)[:, None])[:, 0].long()
    refs += torch.bincount(torch.where(shared, rows, refs.numel()).flatten(), minlength=refs.numel() + 1)[:-1].int()
    new = torch.where(shared, rows, -1)
    table[children] = torch.where((col == full[:, None]) & part[:, None], fresh[:, None].int(), new)
    s["lens"][children] = length.int()
    copied = part.nonzero()[:, 0]
    refs[fresh[copied]] = 1
    pool[fresh[copied]] = pool[last[copied]]
    return {"meta": s["meta"], "pool": pool}


def _plain_free(s):
    table, refs, seqs = s["table"], s["refs"], s["items"].long()
    rows = table[seqs]
    refs -= torch.bincount(torch.where(rows >= 0, rows, refs.numel()).flatten(), minlength=refs.numel() + 1)[:-1].int()
    table[seqs] = -1
    s["lens"][seqs] = 0
    return {"meta": s["meta"]}


def _plain_compact(s):
    table, refs, pool = s["table"], s["refs"], s["pool"]
    alive = refs > 0
    live = alive.sum()
    index = torch.arange(refs.numel(), device="cuda")
    hole, high = (~alive & (index < live)).nonzero()[:, 0], (alive & (index >= live)).nonzero()[:, 0]
    pool[hole] = pool[high]
    place = index.clone()
    place[high] = hole
    table.copy_(torch.where(table >= 0, place[table.long().clamp(min=0)].int(), table))
    refs[hole] = refs[high]
    refs[high] = 0
    s["live"].copy_(live)
    return {"meta": s["meta"], "pool": pool}


def _plain_attn(s):
    c, g, ps = s["c"], s["c"]["hq"] // s["c"]["hkv"], s["c"]["page"]
    b, nq, hkv, d, prefix = c["batch"], c["nq"], c["hkv"], c["d"], c["prefix"]
    q = s["q"].float().view(b, nq, hkv, g, d).permute(2, 0, 1, 3, 4).reshape(hkv, b, nq * g, d) * s["scale"]
    seen = (s["lens"].long()[:, None] - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0)  # keys that a query sees
    seen = seen.repeat_interleave(g, 1)                                                         # [b][nq g]

    def gather(pool, pages):  # [n][pages] -> [hkv][n][tokens][d]
        return pool[pages].float().permute(2, 0, 1, 3, 4).reshape(hkv, pages.shape[0], -1, d)

    shared, rest = s["table"][:1, :prefix // ps].long(), s["table"][:, prefix // ps:].long().clamp(min=0)
    token = torch.arange(prefix + rest.shape[1] * ps, device="cuda")
    hidden = token >= seen[..., None]                                                           # [b][nq g][tokens]
    kt = gather(s["k"], rest)
    own_scores = torch.matmul(q, kt.transpose(-1, -2))
    scores = torch.matmul(q.reshape(hkv, b * nq * g, d), gather(s["k"], shared)[:, 0].transpose(-1, -2)).view(hkv, b, nq * g, prefix)
    scores = torch.cat((scores, own_scores), -1).masked_fill_(hidden, -math.inf)
    del own_scores, kt
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    v = torch.where((token[prefix:] < s["lens"][:, None])[..., None], gather(s["v"], rest), 0.0)
    o = torch.matmul(scores[..., prefix:], v)
    o += torch.matmul(scores[..., :prefix].reshape(hkv, b * nq * g, prefix), gather(s["v"], shared)[:, 0]).view_as(o)
    o /= torch.where(total == 0, 1.0, total)
    lse = total.log() + top
    s["o"].copy_(o.view(hkv, b, nq, g, d).permute(1, 2, 0, 3, 4).reshape(b * nq, -1, d))
    s["lse"].copy_(lse.view(hkv, b, nq, g).permute(1, 2, 0, 3).reshape(b * nq, -1))
    return {"o": s["o"], "lse": s["lse"]}


PLAIN = {"rope": _plain_rope, "reserve": _plain_reserve, "fork": _plain_fork, "free": _plain_free,
         "compact": _plain_compact, "attn": _plain_attn}


# ------------------------------------------------------------------------------------------- through the package
def _workspace(s, size):
    if "workspace" not in s:  # kept by the program for all its calls
        s["workspace"] = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import quant_packed_gemv_gb300 as qp
    c = s["c"]
    if c["op"] == "rope":
        parts = [qp.plm_rope_tensor(s["q"], s["yq"])]
        if c["cache"]:
            parts += [qp.plm_rope_tensor(s["k"], s["pool"][:, 0], slots=s["slots"]),
                      qp.plm_rope_tensor(s["v"], s["pool"][:, 1], slots=s["slots"], rotate=False)]
        else:
            parts.append(qp.plm_rope_tensor(s["k"], s["yk"]))
        qp.plm_rope(parts, s["positions"], s["freqs"], c["rot"], "half" if c["half"] else "interleaved",
                    scale=s["mscale"], inverse=c["inverse"])
        return {"q": s["yq"], "pool": s["pool"]} if c["cache"] else {"q": s["yq"], "k": s["yk"]}
    if c["op"] == "attn":
        ws = _workspace(s, 0) if "workspace" in s else _workspace(s, qp.plm_attn_workspace_size(
            c["batch"], c["nq"], c["hq"], c["hkv"], c["d"], c["prefix"], s["most"]))
        qp.plm_attn_shared_prefix(s["q"], s["o"], s["k"], s["v"], s["table"], s["lens"], c["nq"], c["prefix"], s["most"],
                                  s["scale"], ws, lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    kv = qp.plm_kv_state(s["pool"], s["table"], s["lens"], s["refs"], c["page"], s["status"])
    if c["op"] == "free":
        qp.plm_kv_free(kv, s["items"])
        return {"meta": s["meta"]}
    n = s["children"].numel() if c["op"] == "fork" else c.get("items", 0)
    ws = _workspace(s, qp.plm_kv_workspace_size(c["pages"], n))
    if c["op"] == "reserve":
        qp.plm_kv_reserve(kv, s["items"], s["add"], s["slots"], ws)
        return {"meta": s["meta"], "slots": s["slots"]}
    if c["op"] == "fork":
        qp.plm_kv_fork(kv, s["parents"], s["children"], ws)
    else:
        qp.plm_kv_compact(kv, s["live"], ws)
    return {"meta": s["meta"], "pool": s["pool"]}


def run(state):
    if "start" in state:  # tables, lengths and counts as they were before the call
        state["meta"].copy_(state["start"])
    return _own(state) if own else PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    c = case
    if c["op"] not in ("rope", "attn"):
        return None  # pages are moved and counted, not computed
    s = prepare(case, seed)
    if c["op"] == "rope":
        freqs, mscale = _frequencies(c["rot"], c["base"], c["factor"])
        angle = s["positions"].double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full_like(angle, mscale), -angle if c["inverse"] else angle)[:, None]

        def turned(x):
            x, out = x.double(), x.double().clone()
            h = c["rot"] // 2
            first = slice(0, h) if c["half"] else slice(0, c["rot"], 2)
            second = slice(h, c["rot"]) if c["half"] else slice(1, c["rot"], 2)
            z = torch.complex(x[..., first], x[..., second]) * turn
            out[..., first], out[..., second] = z.real, z.imag
            return out

        if not c["cache"]:
            return {"q": turned(s["q"]), "k": turned(s["k"])}
        pool = s["pool"].double()
        flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, c["hkv"], c["d"])  # [slot][k, v][head][d]
        flat[s["slots"], 0], flat[s["slots"], 1] = turned(s["k"]), s["v"].double()
        return {"q": turned(s["q"]), "pool": flat.view(-1, c["page"], 2, c["hkv"], c["d"]).permute(0, 2, 3, 1, 4).contiguous()}
    o = torch.zeros(c["batch"], c["nq"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["nq"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        k, v = (s["pool"][pages, i].transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:n].double() for i in (0, 1))
        q = s["q"].view(c["batch"], c["nq"], c["hq"], c["d"])[b].double()
        late = torch.arange(n, device="cuda")[None] > torch.arange(n - c["nq"], n, device="cuda")[:, None]
        for h in range(c["hkv"]):
            x = torch.einsum("thd,nd->htn", q[:, h * group:(h + 1) * group], k[:, h]) * s["scale"]
            x = x.masked_fill(late, -math.inf)
            total = torch.logsumexp(x, -1)
            lse[b, :, h * group:(h + 1) * group] = total.T
            o[b, :, h * group:(h + 1) * group] = torch.einsum("htn,nd->thd", (x - total[..., None]).exp(), v[:, h])
    return {"o": o.view(-1, c["hq"], c["d"]), "lse": lse.view(-1, c["hq"])}
