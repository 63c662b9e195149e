"""Cases of the operators around rotated positions and a key/value cache held in 8 bits: the rotation of
queries and keys, the append that rotates on the way into a paged cache, the append into 8-bit pages, the
read of 8-bit pages, and decode attention over them.

``listed()`` names the measured cases, ``draw()`` gives more of the same ranges.  With ``own`` false,
``run`` computes the operators in elementary torch operations in 32 bits (angles in 64); with ``own`` true it
makes the framework's calls.  ``exact`` computes them from their definitions in 64 bits.

An 8-bit cache is k_cache, v_cache [pages, heads, page, d] of e4m3 and k_scale, v_scale [pages, heads,
page / block] in fp32: a value is its code times the scale of its block of keys.  A block that receives rows
takes the smallest scale 2^e, -54 <= e <= 54, with 448 * 2^e no less than the reach of these rows, or the one
it had if that is larger and it holds earlier rows; these are rescaled then.  The reach is the largest length
of a pair that is turned (lengths do not change under a rotation, so a scale does not depend on positions),
and the largest magnitude of the elements that are not.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token's queries and keys in one layer of a long conversation: latency
        dict(name="rope_one", op="rope", packed=True, batch=1, n=1, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, inverse=False, method="yarn", far=100000),
        # packed prompts
        dict(name="rope_prompts", op="rope", packed=True, batch=1, n=8192, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, inverse=False, method="linear", far=30000),
        # gradient of a training batch, pairs side by side, half of the head turned, odd length
        dict(name="rope_gradient", op="rope", packed=False, batch=4, n=2047, hq=16, hkv=16, d=96, rot=48,
             interleaved=True, inverse=True, method="", far=2047),
        # a serving step: the next token of every sequence, its queries turned in the same call
        dict(name="append_step", op="append", batch=64, n=1, ragged=False, lo=1000, hi=30000, hq=64, hkv=8,
             d=128, rot=128, interleaved=False, method="ntk", page=16),
        # chunks of prompts of different lengths, a quarter of a large head turned
        dict(name="append_chunks", op="append", batch=8, n=777, ragged=True, lo=0, hi=2000, hq=16, hkv=4,
             d=256, rot=64, interleaved=True, method="", page=64),
        # next tokens of a batch into 8-bit pages, a scale for every 16 keys
        dict(name="q8_append", op="append8", batch=128, n=1, ragged=False, lo=20, hi=1000, hq=32, hkv=8, d=128,
             rot=128, interleaved=False, method="", page=64, block=16),
        # chunks of prompts appended, and the sequences read back for the chunks' attention
        dict(name="q8_chunks", op="prompt8", batch=8, n=1024, ragged=True, lo=0, hi=4000, hkv=8, d=128, rot=128,
             interleaved=False, method="", page=64, block=64),
        # one sequence's next token: latency
        dict(name="q8_decode_one", op="decode8", batch=1, hq=32, hkv=8, sq=1, lo=2000, hi=2000, d=128, page=64,
             block=64, window=0, first=0, causal=False, sinks=False),
        # next tokens of a batch over long caches
        dict(name="q8_decode_batch", op="decode8", batch=64, hq=64, hkv=8, sq=1, lo=1024, hi=16384, d=128,
             page=64, block=64, window=0, first=0, causal=False, sinks=False),
        # a few drafted tokens with a window, first keys and sink logits, small pages of an odd size
        dict(name="q8_decode_drafts", op="decode8", batch=24, hq=24, hkv=4, sq=5, lo=500, hi=9000, d=64, page=48,
             block=16, window=2048, first=4, causal=True, sinks=True),
        # one very long sequence, large head
        dict(name="q8_decode_long", op="decode8", batch=1, hq=16, hkv=2, sq=1, lo=130000, hi=130000, d=256,
             page=128, block=128, window=0, first=0, causal=False, sinks=False),
        # a serving step as it is used: queries and keys turned, keys and values appended, attended
        dict(name="q8_step", op="step8", batch=32, n=1, ragged=False, hq=32, hkv=8, sq=1, lo=200, hi=6000, d=128,
             rot=128, interleaved=False, method="yarn", page=32, block=32, window=0, first=0, causal=True,
             sinks=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.6e12 + w["flops"] / 2e14


def draw(rng):
    op = rng.choice(["rope", "append", "append8", "prompt8", "decode8", "decode8", "step8"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    d = rng.choice([64, 128, 128, 256])
    turned = dict(interleaved=rng.random() < 0.5, method=rng.choice(["", "linear", "ntk", "yarn"]))
    if op == "rope":
        d = rng.choice([64, 96, 128, 256, 512])
        n, packed = _log(rng, 1, 8192), rng.random() < 0.5
        c = dict(op=op, packed=packed, batch=1 if packed else _log(rng, 1, 8), n=n, hq=hkv * group, hkv=hkv, d=d,
                 rot=16 * rng.randint(1, d // 16), inverse=rng.random() < 0.3, far=max(n, _log(rng, 1, 1000000)),
                 **turned)
    elif op in ("append", "append8", "prompt8"):
        n = _log(rng, 1, 1024) if op != "append8" else rng.choice([1, 1, 2, 5, 16])
        hi = _log(rng, 1, 30000 if op == "append" else 4000)
        c = dict(op=op, batch=_log(rng, 1, 128 if n < 16 else 8), n=n, ragged=rng.random() < 0.5,
                 lo=rng.randint(0, hi), hi=hi, hkv=hkv, d=d, rot=16 * rng.randint(1, d // 16), **turned)
        if op != "prompt8":
            c["hq"] = rng.choice([0, hkv * group])
    else:
        hi = _log(rng, 64, 30000)
        sq = 1 if op == "step8" else rng.choice([1, 1, 1, 2, 5, 8])
        c = dict(op=op, batch=_log(rng, 1, 64), hq=hkv * group, hkv=hkv, sq=sq, lo=rng.randint(sq, hi), hi=hi,
                 d=d, window=0, first=0, causal=rng.random() < 0.7, sinks=rng.random() < 0.3)
        if rng.random() < 0.4:
            c.update(window=_log(rng, 16, 4096), first=rng.choice([0, 1, 4, 130]))
        if op == "step8":
            c.update(n=1, ragged=False, rot=16 * rng.randint(1, d // 16), **turned)
    if op != "rope":
        c["page"] = rng.choice([16, 32, 48, 64, 100, 128, 256])
    if "8" in op:
        c["block"] = c["page"] // rng.choice([1, 1, 2, 4])
    most = max(_cost(x) for x in listed() if x["op"] == op)
    while _cost(c) > most:   # smaller, but of the same kind
        if c["batch"] > 1:
            c["batch"] = (c["batch"] + 1) // 2
        else:
            for key in ("hi", "lo", "n"):
                if key in c:
                    c[key] = (c[key] + 1) // 2
    return c


def work(case):
    """Bytes and operations of one pass with lengths at the middle of their range."""
    c, d = case, case["d"]
    if c["op"] == "rope":
        tokens = c["batch"] * c["n"]
        return {"bytes": tokens * ((c["hq"] + c["hkv"]) * d * 4.0 + 4),
                "flops": tokens * (c["hq"] + c["hkv"]) * c["rot"] * 3.0}
    byt = flops = 0.0
    new = 0
    if c["op"] != "decode8":
        new = (1 + c["n"]) / 2 if c["ragged"] else c["n"]
        rows = c["batch"] * new
        byt += rows * (2 * c["hkv"] * d * (4 if c["op"] == "append" else 3) + 4 * c.get("hq", 0) * d)
        flops += rows * (c["hkv"] + c.get("hq", 0)) * c["rot"] * 3.0
    if c["op"] == "prompt8":
        byt += c["batch"] * ((c["lo"] + c["hi"]) / 2 + new) * 2 * c["hkv"] * d * 3
    if c["op"] in ("decode8", "step8"):
        keys = (c["lo"] + c["hi"]) / 2 + new
        if c["window"] > 0:
            keys = min(keys, c["window"] + c["sq"] - 1 + c["first"])
        byt += c["batch"] * c["hkv"] * keys * (2 * d + 8 / c["block"])
        if c["op"] == "decode8":
            byt += c["batch"] * c["hq"] * c["sq"] * (4 * d + 4)
        flops += 4.0 * c["batch"] * c["hq"] * c["sq"] * keys * d
    return {"bytes": byt, "flops": flops}


# ----------------------------------------------------------------- inputs ----

def _spread(g, lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], in an order of the seed's (their sum, and with it the
    shapes of packed tensors, is the case's)."""
    even = [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]
    return [even[i] for i in torch.randperm(n, generator=g).tolist()]


def _randn(gd, *shape):
    return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _inv_freq(rot, method):
    """Radians a position of each pair, 64 bits, and the factor of the turned pairs; contexts stretched by 8."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    base, stretch, original = 10000.0, 8.0, 4096
    if method == "ntk":
        base *= stretch ** (rot / max(1, rot - 2))
    inv = base ** (-2.0 * i / rot)
    if method == "linear":
        return inv / stretch, 1.0
    if method == "yarn":   # pairs that turn often in the original context stay, slow ones are stretched
        turns = original * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return inv * (keep + (1.0 - keep) / stretch), 0.1 * math.log(stretch) + 1.0
    return inv, 1.0


def _scale_of(square):
    """The smallest 2^e, -54 <= e <= 54, with (448 * 2^e)^2 = 49/64 * 2^(18 + 2 e) no less than `square`."""
    part, power = torch.frexp(square.clamp(max=1e38))
    y = power - 18
    e = torch.div(y + 1, 2, rounding_mode="floor") + ((y % 2 == 0) & (part > 0.765625)).to(y.dtype)
    e = torch.where(square > 0, e, -54).clamp(-54, 54)
    return torch.ldexp(torch.ones_like(square), e)


def _codes(gd, pages, heads, page, block, d):
    """Codes and scales of random rows, whose magnitudes differ from head to head and page to page."""
    x = torch.randn(pages, heads, page, d, generator=gd, device=DEV)
    x *= torch.exp(0.7 * torch.randn(pages, heads, 1, 1, generator=gd, device=DEV))
    x = x.view(pages, heads, page // block, block * d)
    scale = _scale_of(x.abs().amax(-1) ** 2)
    return (x / scale[..., None]).to(F8).view(pages, heads, page, d), scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator().manual_seed(seed * 2 + 1)
    gd = torch.Generator(device=DEV).manual_seed(seed * 2)
    s = {"case": c}
    d, batch = c["d"], c["batch"]
    if "rot" in c:
        inv, s["factor"] = _inv_freq(c["rot"], c["method"])
        s["inv_freq"] = inv.to(DEV)
        # radians in units of 2^-64 of a turn
        s["freqs"] = torch.tensor([int(round(f / (2 * math.pi) * 2 ** 64)) for f in inv.tolist()],
                                  dtype=torch.int64, device=DEV)
    if c["op"] == "rope":
        n = c["n"]
        start = int(torch.randint(0, c["far"] - n + 1, (1,), generator=g))
        s["positions"] = torch.arange(start, start + n, device=DEV, dtype=torch.int32)
        if c["packed"]:   # tokens of a projection, heads side by side
            s["q"], s["k"] = _randn(gd, n, c["hq"], d), _randn(gd, n, c["hkv"], d)
        else:
            s["q"], s["k"] = _randn(gd, batch, c["hq"], n, d), _randn(gd, batch, c["hkv"], n, d)
        return s
    lens = _spread(g, c["lo"], c["hi"], batch)
    hkv, page, more = c["hkv"], c["page"], c.get("n", 0)
    need = [-(-(n + more) // page) for n in lens]
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    table = torch.full((batch, max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):   # pages in a random order, the last one of the caches spare
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["lens"] = table.to(DEV), _i32(lens)
    if "8" in c["op"]:
        s["k"], s["k_scale"] = _codes(gd, at + 1, hkv, page, c["block"], d)
        s["v"], s["v_scale"] = _codes(gd, at + 1, hkv, page, c["block"], d)
    else:
        s["k"], s["v"] = _randn(gd, at + 1, hkv, page, d), _randn(gd, at + 1, hkv, page, d)
    if "rot" in c:
        new = _spread(g, 1, c["n"], batch) if c["ragged"] else [c["n"]] * batch
        s["n_new"] = _i32(new)
        # rows as a projection leaves them: token by token, heads side by side
        s["k_new"], s["v_new"] = (_randn(gd, batch, c["n"], hkv, d).transpose(1, 2) for _ in range(2))
        if c.get("hq"):
            s["q_new"] = _randn(gd, batch, c["n"], c["hq"], d).transpose(1, 2)
            s["q_out"] = torch.zeros(batch, c["hq"], c["n"], d, dtype=torch.bfloat16, device=DEV)
        total = [a + b for a, b in zip(lens, new)]
        s["ends"] = _i32(total)
        s["cu"] = _i32([0] + torch.tensor(total).cumsum(0).tolist())
        s["total"], s["longest"] = sum(total), max(total)
    if c["op"] == "decode8":
        s["q"] = _randn(gd, batch, c["hq"], c["sq"], d)
    if c.get("sinks"):
        s["sinks"] = torch.randn(c["hq"], generator=gd, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----

def _turn(x, positions, s, inverse=False):
    """x [..., n, d] in 32 bits, positions [..., n] that broadcast over it: the turned rows in 32 bits."""
    rot, x = s["case"]["rot"], x.float()
    angle = positions.double()[..., None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["factor"]).float() for f in (torch.cos, torch.sin))
    sin = -sin if inverse else sin
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    c, at = s["case"], s["positions"]
    if c["packed"]:
        q, k = (_turn(s[x].transpose(0, 1), at, s, c["inverse"]).transpose(0, 1) for x in "qk")
    else:
        q, k = (_turn(s[x], at, s, c["inverse"]) for x in "qk")
    return {"q": q.to(torch.bfloat16).contiguous(), "k": k.to(torch.bfloat16).contiguous()}


def _page_of(table, place, page):
    return torch.gather(table, 1, (place // page).clamp(0, table.shape[1] - 1).long())


def _plain_q(s):
    """Queries of the new rows, turned; rows behind a sequence's last stay as they were."""
    i = torch.arange(s["case"]["n"], device=DEV)
    q = _turn(s["q_new"], (s["lens"][:, None] + i)[:, None], s).to(torch.bfloat16)
    s["q_out"].copy_(torch.where((i < s["n_new"][:, None])[:, None, :, None], q, s["q_out"]))
    return s["q_out"]


def _put(cache, page, slot, rows, real):
    """cache[page, :, slot] = rows where real; the others go to the spare page as it is."""
    spare = cache.shape[0] - 1
    rows = torch.where(real[..., None, None], rows, cache[spare, :, 0])
    cache[torch.where(real, page, spare).long(), :, torch.where(real, slot, 0).long()] = rows


def _plain_append(s):
    c = s["case"]
    i = torch.arange(c["n"], device=DEV)
    place = s["lens"][:, None] + i
    k = _turn(s["k_new"], place[:, None], s).to(torch.bfloat16)
    at, real = (_page_of(s["table"], place, c["page"]), place % c["page"]), i < s["n_new"][:, None]
    _put(s["k"], *at, k.transpose(1, 2), real)
    _put(s["v"], *at, s["v_new"].transpose(1, 2), real)
    out = {"k": s["k"], "v": s["v"]}
    if c["hq"]:
        out["q"] = _plain_q(s)
    return out


def _reach(x, rot, interleaved, factor):
    """Square of the reach of each row [..., d] in 32 bits."""
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    one = torch.tensor(factor, device=DEV)
    pairs = (a * a + b * b).amax(-1) * (one * one) if rot else torch.zeros(x.shape[:-1], device=DEV)
    rest = x[..., rot:]
    return torch.maximum(pairs, (rest * rest).amax(-1)) if rest.shape[-1] else pairs


def _plain_append8(s, name, rows, square):
    """rows [b, h, n, d] in 32 bits to the blocks of keys lens[b] + i; square [b, h, n] their reaches."""
    c, codes, scale = s["case"], s[name], s[name + "_scale"]
    page, block, n = c["page"], c["block"], c["n"]
    batch, heads, _, d = rows.shape
    lens, end = s["lens"][:, None], s["lens"][:, None] + s["n_new"][:, None]
    # the blocks that new rows lie in, [b, blocks], and the keys of each, [b, blocks * block]
    at = lens // block + torch.arange((n + block - 2) // block + 1, device=DEV)
    key = (at[..., None] * block + torch.arange(block, device=DEV)).flatten(1)
    touched = (at * block < end) & (lens < end)
    spare = codes.shape[0] - 1
    home = torch.where(touched, _page_of(s["table"], at * block, page), spare).long()
    slot = torch.where(touched, at * block % page // block, 0).long()
    fresh = ((key >= lens) & (key < end))[:, None]                  # [b, 1, keys]
    source = (key - lens).clamp(0, n - 1).long()[:, None].expand(-1, heads, -1)
    x = torch.gather(rows, 2, source[..., None].expand(-1, -1, -1, d))
    need = torch.where(fresh, torch.gather(square, 2, source), 0.0)
    need = _scale_of(need.unflatten(2, (-1, block)).amax(-1))       # [b, h, blocks]
    before = torch.where((at * block < lens)[:, None], scale[home, :, slot].transpose(1, 2), 0.0)
    now = torch.maximum(before, need)
    ratio = (before / now)[..., None, None]
    old = codes.view(torch.uint8).unflatten(2, (-1, block))[home, :, slot].transpose(1, 2).contiguous()
    old = old.view(F8).float()                                      # [b, h, blocks, block, d]
    x = x.unflatten(2, (-1, block))
    fresh, key = fresh.unflatten(2, (-1, block))[..., None], key.unflatten(1, (-1, block))
    got = torch.where(fresh, x / now[..., None, None], old * ratio).to(F8).view(torch.uint8)
    kept = (key < end[..., None]) & touched[..., None]              # rows behind the last stay
    raw = codes.view(torch.uint8).unflatten(2, (-1, block))
    was = raw[home, :, slot].transpose(1, 2)
    got = torch.where(kept[:, None, ..., None], got, was)
    raw[home, :, slot] = got.transpose(1, 2)
    scale[home, :, slot] = torch.where(touched[:, None], now, scale[home, :, slot].transpose(1, 2)).transpose(1, 2)


def _plain_rows8(s):
    c = s["case"]
    place = (s["lens"][:, None] + torch.arange(c["n"], device=DEV))[:, None]
    square = _reach(s["k_new"], c["rot"], c["interleaved"], s["factor"])
    _plain_append8(s, "k", _turn(s["k_new"], place, s), square)
    _plain_append8(s, "v", s["v_new"].float(), _reach(s["v_new"], 0, False, 1.0))
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _values(s, name):
    """Values [b, heads, keys, d] in 32 bits of an 8-bit cache."""
    c, table = s["case"], s["table"].clamp(min=0).long()
    x = s[name].view(torch.uint8)[table].view(F8).float()           # [b, pages, heads, page, d]
    scale = s[name + "_scale"][table]                               # [b, pages, heads, page / block]
    x = x.unflatten(3, (-1, c["block"])) * scale[..., None, None]
    return x.flatten(3, 4).transpose(1, 2).flatten(2, 3)


def _plain_read(s):
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    at = row - s["cu"].long()[seq]
    return {"k_read": _values(s, "k")[seq, :, at].to(torch.bfloat16),
            "v_read": _values(s, "v")[seq, :, at].to(torch.bfloat16)}


def _plain_decode(s, q, lens):
    c = s["case"]
    batch, hq, n, d = q.shape
    k, v, lens = _values(s, "k"), _values(s, "v"), lens[:, None, None]
    place = torch.arange(n, device=DEV)[:, None] + lens - n
    key = torch.arange(k.shape[2], device=DEV)
    seen = key < lens
    if c["causal"]:
        seen = seen & (key <= place)
    if c["window"]:
        seen = seen & ((key > place - c["window"]) | (key < c["first"]))
    seen = seen.expand(batch, n, -1)
    v = torch.where(key[:, None] < lens[:, None], v, 0.0)
    score = torch.matmul(q.float().reshape(batch, c["hkv"], -1, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = torch.where(seen[:, None], score.reshape(batch, hq, n, -1), -math.inf)
    top = score.amax(-1, keepdim=True)
    sinks = s["sinks"].reshape(1, -1, 1, 1) if c["sinks"] else None
    top = torch.maximum(top, sinks) if c["sinks"] else top
    base = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - base)
    total = p.sum(-1, keepdim=True)
    total = total + torch.exp(sinks - base) if c["sinks"] else total
    o = torch.matmul(p.reshape(batch, c["hkv"], -1, k.shape[2]), v).reshape(batch, hq, n, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, base + torch.log(total), -math.inf)
    return {"o": o.to(torch.bfloat16), "lse": lse[..., 0]}


# ------------------------------------------------------- the framework's calls ----

def _own(s):
    from attention_forward_blackwell_gb300 import binding as fa
    c = s["case"]
    turned = dict(interleaved=c.get("interleaved", False), factor=s.get("factor", 1.0))
    if c["op"] == "rope":
        q, k = fa.rope(s["q"], s["k"], s["positions"], s["freqs"], inverse=c["inverse"], **turned)
        return {"q": q, "k": k}
    out = {}
    q, lens = s.get("q"), s["lens"]
    if "rot" in c:
        rows = dict(n_new=s["n_new"] if c["ragged"] else None, q=s.get("q_new"), q_out=s.get("q_out"), **turned)
        if c["op"] == "append":
            fa.cache_append_rope(s["k"], s["v"], s["table"], lens, s["k_new"], s["v_new"], s["freqs"], **rows)
            out = {"k": s["k"], "v": s["v"]}
        else:
            fa.cache_append_q8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], lens, s["k_new"],
                               s["v_new"], s["freqs"], **rows)
            out = {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if c.get("hq"):
            out["q"] = s["q_out"]
        q, lens = s.get("q_out"), s["ends"]
    if c["op"] == "prompt8":
        out["k_read"], out["v_read"] = fa.cache_read_q8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"],
                                                        s["cu"], s["total"], s["longest"])
    if c["op"] in ("decode8", "step8"):
        out["o"], out["lse"] = fa.decode_paged_q8(q, s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], lens,
                                                  causal=c["causal"], window=c["window"], first=c["first"],
                                                  sinks=s.get("sinks"))
    return out


def run(state):
    if own:
        return _own(state)
    s, op = state, state["case"]["op"]
    if op == "rope":
        return _plain_rope(s)
    if op == "append":
        return _plain_append(s)
    if op == "decode8":
        return _plain_decode(s, s["q"], s["lens"])
    out = _plain_rows8(s)
    if s["case"].get("hq"):
        out["q"] = _plain_q(s)
    if op == "prompt8":
        out.update(_plain_read(s))
    if op == "step8":
        out.update(_plain_decode(s, s["q_out"], s["ends"]))
    return out


# --------------------------------------------------------------- 64 bits ----

def _exact_turn(x, positions, inv, factor, interleaved, inverse=False):
    """Rows x [n, ..., d] at positions [n], as complex numbers times e^(i angle)."""
    x, rot = x.double(), 2 * inv.numel()
    angle = torch.outer(positions.double(), inv) * (-1.0 if inverse else 1.0)
    by = torch.polar(torch.full_like(angle, factor), angle)
    by = by.reshape(by.shape[0], *([1] * (x.dim() - 2)), -1)
    out = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * by
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * by
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _exact_reach(x, rot, interleaved, factor):
    """Largest length of a turned pair and magnitude of the other elements of rows [..., d]."""
    x = x.double()
    pairs = x[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1)) if rot else None
    most = x[..., rot:].abs().amax() if x.shape[-1] > rot else torch.zeros((), device=DEV, dtype=torch.float64)
    if rot:
        most = torch.maximum(most, factor * pairs.square().sum(-1 if interleaved else -2).amax().sqrt())
    return float(most)


def _round8(x):
    """e4m3 values next to x (|x| <= 448), ties to even, in 64 bits."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4       # steps of 2^(exponent - 3), subnormal ones 2^-9
    step = torch.ldexp(torch.ones_like(x), e)
    return torch.round(x / step) * step


def _exact_append8(s, values, scales, rows, reach_of):
    """values [pages, h, page, d] in 64 bits (codes), scales in 64 bits, both changed; rows [b][n, h, d]."""
    page, block = s["case"]["page"], s["case"]["block"]
    lens = s["lens"].tolist()
    for b, x in enumerate(rows):
        for first in range(lens[b] // block * block, lens[b] + x.shape[0], block):
            p, at = int(s["table"][b, first // page]), first % page
            lo, hi = max(first, lens[b]), min(first + block, lens[b] + x.shape[0])
            for h in range(x.shape[1]):
                most = reach_of(b, h, lo - lens[b], hi - lens[b])
                e = max(-54, min(54, math.ceil(math.log2(most / 448.0)))) if most > 0 else -54
                new, old = 2.0 ** e, float(scales[p, h, at // block])
                if lo > first and old > new:
                    new = old
                if lo > first:
                    part = values[p, h, at:at + lo - first]
                    values[p, h, at:at + lo - first] = _round8(part * (old / new))
                values[p, h, at + lo - first:at + hi - first] = _round8(x[lo - lens[b]:hi - lens[b], h] / new)
                scales[p, h, at // block] = new


def _exact_decode(s, q, k, v, lens):
    """q [b, hq, n, d] and values k, v [pages, h, page, d] in 64 bits."""
    c = s["case"]
    out, lses = [], []
    for b, length in enumerate(lens):
        token = torch.arange(length, device=DEV)
        home = s["table"][b].long()[token // c["page"]]
        kb, vb = (x[home, :, token % c["page"]].double().transpose(0, 1) for x in (k, v))
        n = q.shape[2]
        far = torch.arange(length - n, length, device=DEV)[:, None] - token     # how far back a key lies
        hidden = (far < 0) if c["causal"] else torch.zeros_like(far, dtype=torch.bool)
        if c["window"]:
            hidden = hidden | ((far >= c["window"]) & (token >= c["first"]))
        x = torch.einsum("hgnd,hmd->hgnm", q[b].double().unflatten(0, (c["hkv"], -1)), kb) / math.sqrt(c["d"])
        x = x.masked_fill(hidden, -math.inf).flatten(0, 1)
        if c["sinks"]:
            x = torch.cat([x, s["sinks"].double()[:, None, None].expand(-1, n, 1)], -1)
        lse = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])[..., :length]
        out.append(torch.einsum("hgnm,hmd->hgnd", w.unflatten(0, (c["hkv"], -1)), vb).flatten(0, 1))
        lses.append(lse)
    return {"o": torch.stack(out), "lse": torch.stack(lses)}


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if "rot" in c:
        how = (s["inv_freq"], s["factor"], c["interleaved"])
    if c["op"] == "rope":
        if c["packed"]:
            return {x: _exact_turn(s[x], s["positions"], *how, c["inverse"]) for x in "qk"}
        return {x: _exact_turn(s[x].permute(2, 0, 1, 3), s["positions"], *how, c["inverse"]).permute(1, 2, 0, 3)
                .contiguous() for x in "qk"}
    if "rot" in c:
        lens, new = s["lens"].tolist(), s["n_new"].tolist()
        place = [torch.arange(a, a + n, device=DEV) for a, n in zip(lens, new)]
        turned = lambda name: [_exact_turn(s[name][b, :, :n].transpose(0, 1), place[b], *how)  # noqa: E731
                               for b, n in enumerate(new)]
        plain = [s["v_new"][b, :, :n].transpose(0, 1).double() for b, n in enumerate(new)]
        out = {}
        if c.get("hq"):
            out["q"] = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
            for b, x in enumerate(turned("q_new")):
                out["q"][b, :, :new[b]] = x.transpose(0, 1)
    if c["op"] == "append":
        for name, rows in (("k", turned("k_new")), ("v", plain)):
            out[name] = s[name].double()
            for b, x in enumerate(rows):
                out[name][s["table"][b].long()[place[b] // c["page"]], :, place[b] % c["page"]] = x
        return out
    values = {x: s[x].to(torch.float64) for x in "kv"}
    scales = {x: s[x + "_scale"].double() for x in "kv"}
    by_value = lambda x: (values[x].unflatten(2, (-1, c["block"])) * scales[x][..., None, None]).flatten(2, 3)  # noqa: E731
    if c["op"] == "decode8":
        return _exact_decode(s, s["q"], by_value("k"), by_value("v"), s["lens"].tolist())
    if c["batch"] * c["hkv"] * (c["n"] / c["block"] + 1) > 6000:   # (a block at a time)
        return None
    for name, rows, rot in (("k", turned("k_new"), c["rot"]), ("v", plain, 0)):
        _exact_append8(s, values[name], scales[name], rows, lambda b, h, lo, hi: _exact_reach(
            s[name + "_new"][b, h, lo:hi], rot, c["interleaved"], s["factor"]))
        out[name], out[name + "_scale"] = values[name], scales[name]
    if c["op"] == "prompt8":
        for name in "kv":
            x = by_value(name)
            rows = [x[s["table"][b].long()[t // c["page"]], :, t % c["page"]] for b, t in
                    enumerate(torch.arange(e, device=DEV) for e in s["ends"].tolist())]
            out[name + "_read"] = torch.cat(rows)
    if c["op"] == "step8":   # (the queries that the attention takes are those in bf16)
        out.update(_exact_decode(s, out["q"].to(torch.bfloat16), by_value("k"), by_value("v"), s["ends"].tolist()))
    return out
