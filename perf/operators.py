"""Cases of the serving operators around a key/value cache: attention of drafted token trees, attention
with a sliding window and visible first tokens, and the page operators of a paged cache.

``listed()`` names the measured cases, ``draw()`` gives more of the same ranges.  With ``own`` false,
``run`` computes the operators in elementary torch operations in 32 bits; with ``own`` true it makes the
framework's calls.  ``exact`` computes the attentions from their definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one sequence, a short draft, every head with its own keys: latency of one layer's call
        dict(name="tree_one", op="tree", batch=1, hq=16, hkv=16, nodes=7, ragged=False, lo=900, hi=1100,
             d=64, page=0, sinks=False, fresh=False),
        # a serving step: small ragged trees over a paged cache, the mask built from the drafts' parents
        dict(name="tree_step", op="tree", batch=16, hq=64, hkv=8, nodes=16, ragged=True, lo=1024, hi=16384,
             d=128, page=64, sinks=False, fresh=True),
        # wide trees, 512 query rows per key/value head: the tensor cores count as much as the memory
        dict(name="tree_wide", op="tree", batch=8, hq=64, hkv=8, nodes=64, ragged=False, lo=4096, hi=8192,
             d=128, page=128, sinks=False, fresh=False),
        # large head dimension, an odd number of nodes, contiguous caches, a sink logit per head
        dict(name="tree_d256", op="tree", batch=4, hq=32, hkv=4, nodes=25, ragged=True, lo=2048, hi=8192,
             d=256, page=0, sinks=True, fresh=False),
        # one sequence's next token with a short window: latency
        dict(name="window_decode_one", op="window_decode", batch=1, hq=32, hkv=8, sq=1, lo=8000, hi=8192,
             d=128, page=0, window=1024, first=4, sinks=False),
        # next tokens of a batch over a cache of small pages
        dict(name="window_decode_batch", op="window_decode", batch=64, hq=64, hkv=8, sq=1, lo=1024, hi=16384,
             d=128, page=16, window=4096, first=64, sinks=False),
        # prompts of one length, four first tokens kept
        dict(name="window_prefill", op="window_prefill", batch=2, hq=16, hkv=16, qlo=4096, qhi=4096, plo=0,
             phi=0, d=128, page=0, packed=False, window=1024, first=4, sinks=False),
        # chunks of prompts, packed, over a paged cache, first tokens past one key block, sink logits
        dict(name="window_chunks", op="window_prefill", batch=8, hq=32, hkv=4, qlo=200, qhi=1024, plo=0,
             phi=3000, d=256, page=128, packed=True, window=512, first=130, sinks=True),
        # one sequence: the drafted nodes' rows appended, the accepted path moved together
        dict(name="accept_one", op="accept", batch=1, hkv=8, nodes=8, lo=500, hi=1000, d=128, page=16),
        # the same for a batch of wide trees
        dict(name="accept_batch", op="accept", batch=128, hkv=8, nodes=64, lo=256, hi=2048, d=128, page=16),
        # one prompt continued by four samples: pages shared, the last one copied, one token appended
        dict(name="fork_one", op="fork", groups=1, samples=4, hkv=8, lo=300, hi=500, d=128, page=16, extra=1),
        # a batch of prompts, eight samples each
        dict(name="fork_batch", op="fork", groups=32, samples=8, hkv=8, lo=512, hi=4096, d=128, page=64,
             extra=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.8e15


def draw(rng):
    op = rng.choice(["tree", "tree", "window_decode", "window_prefill", "accept", "fork"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "tree":
        hi = _log(rng, 64, 16384)
        c = dict(op=op, batch=_log(rng, 1, 48), hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), hkv=hkv,
                 nodes=_log(rng, 1, 100), ragged=rng.random() < 0.5, lo=rng.randint(0, hi), hi=hi,
                 d=rng.choice([64, 128, 128, 256]), page=rng.choice([0, 0, 16, 32, 48, 64, 100, 128, 256]),
                 sinks=rng.random() < 0.3, fresh=rng.random() < 0.3)
    elif op == "window_decode":
        hi = _log(rng, 64, 16384)
        c = dict(op=op, batch=_log(rng, 1, 64), hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv,
                 sq=rng.choice([1, 1, 1, 2, 5]), lo=rng.randint(5, hi), hi=hi, d=rng.choice([64, 128, 256]),
                 page=rng.choice([0, 0, 16, 64, 100, 128]), window=_log(rng, 16, 4096),
                 first=_log(rng, 1, 300), sinks=rng.random() < 0.3)
    elif op == "window_prefill":
        hi = _log(rng, 64, 4096)
        packed = rng.random() < 0.6
        c = dict(op=op, batch=_log(rng, 1, 8), hq=hkv * rng.choice([1, 2, 4]), hkv=hkv,
                 qlo=rng.randint(1, hi) if packed else hi, qhi=hi, plo=0,
                 phi=_log(rng, 1, 3000) if packed else 0, d=rng.choice([64, 96, 128, 256, 512]),
                 page=rng.choice([0, 128, 256]) if packed else 0, packed=packed, window=_log(rng, 16, 2048),
                 first=_log(rng, 1, 300), sinks=rng.random() < 0.3)
    elif op == "accept":
        hi = _log(rng, 16, 2048)
        c = dict(op=op, batch=_log(rng, 1, 128), hkv=hkv, nodes=_log(rng, 1, 100), lo=rng.randint(0, hi),
                 hi=hi, d=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 100, 128]))
    else:
        hi = _log(rng, 16, 4096)
        c = dict(op=op, groups=_log(rng, 1, 32), samples=rng.randint(1, 8), hkv=hkv, lo=rng.randint(1, hi),
                 hi=hi, d=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 100, 128]),
                 extra=rng.choice([1, 1, 3, 40]))
    most = max(_cost(x) for x in listed() if x["op"] == op)
    while _cost(c) > most:   # smaller, but of the same kind
        for key in ("batch", "groups"):
            if c.get(key, 1) > 1:
                c[key] = (c[key] + 1) // 2
                break
        else:
            for key in ("hi", "qhi", "lo", "qlo", "phi"):
                if key in c:
                    c[key] = (c[key] + 1) // 2
    return c


def work(case):
    """Bytes and operations of one pass with lengths at the middle of their range."""
    c, d = case, case["d"]
    if c["op"] == "tree":
        t = (1 + c["nodes"]) / 2 if c["ragged"] else c["nodes"]
        ctx = (c["lo"] + c["hi"]) / 2
        words = (c["nodes"] + 31) // 32
        byt = c["batch"] * (c["hkv"] * (ctx + t) * d * 4 + c["hq"] * t * (d * 4 + 4) + c["nodes"] * words * 4)
        return {"bytes": byt, "flops": 4.0 * c["batch"] * c["hq"] * t * (ctx + t / 2) * d}
    if c["op"] == "window_decode":
        keys = min((c["lo"] + c["hi"]) / 2, c["window"] + c["sq"] - 1 + c["first"])
        byt = c["batch"] * (c["hkv"] * keys * d * 4 + c["hq"] * c["sq"] * (d * 4 + 4))
        return {"bytes": byt, "flops": 4.0 * c["batch"] * c["hq"] * c["sq"] * keys * d}
    if c["op"] == "window_prefill":
        q, past = (c["qlo"] + c["qhi"]) / 2, (c["plo"] + c["phi"]) / 2
        w = c["window"] + c["first"]
        full = max(0.0, min(q, w - past))              # rows that see every key up to their own
        pairs = full * (past + full / 2) + (q - full) * w
        byt = c["batch"] * (c["hkv"] * (q + past) * d * 4 + c["hq"] * q * (d * 4 + 4))
        return {"bytes": byt, "flops": 4.0 * c["batch"] * c["hq"] * pairs * d}
    if c["op"] == "accept":
        t = (1 + c["nodes"]) / 2
        rows = t + max(1.0, t / 4)                     # appended, and moved
        return {"bytes": 8.0 * c["batch"] * rows * c["hkv"] * d, "flops": 0.0}
    forks = c["groups"] * c["samples"]
    rows = c["page"] / 2 + c["extra"]                  # copied, and appended
    pages = (c["lo"] + c["hi"]) / 2 / c["page"]
    return {"bytes": forks * (8.0 * rows * c["hkv"] * d + 12.0 * pages), "flops": 0.0}


# ----------------------------------------------------------------- inputs ----

def _ints(g, lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], in an order of the seed's (their sum, and with it the
    shapes of packed tensors, is the case's)."""
    even = [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]
    return [even[i] for i in torch.randperm(n, generator=g).tolist()]


def _randn(gd, *shape):
    return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _paged(gd, g, lens, hkv, page, d, more=0):
    """Caches whose sequences' pages lie in a random order: (k, v, table), the last page spare."""
    need = [-(-(n + more) // page) for n in lens]
    width = max(1, max(need))
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (at + 1, hkv, page, d)
    return _randn(gd, *shape), _randn(gd, *shape), table.to(DEV)


def _tree(g, batch, nodes):
    """Parents of random trees [batch, nodes] (a node hangs on one of the eight before it)."""
    back = torch.randint(1, 9, (batch, nodes), generator=g)
    at = torch.arange(nodes)
    parents = torch.clamp(at - back, min=0)
    parents[:, 0] = -1
    return parents.to(torch.int32)


def _ancestors(parents):
    """Visibility [batch, nodes, nodes] of each node's ancestors and itself."""
    p = parents.numpy()
    batch, nodes = p.shape
    seen = np.zeros((batch, nodes, nodes), dtype=bool)
    rows = np.arange(batch)
    for i in range(nodes):
        up = p[:, i]
        seen[:, i] = np.where(up[:, None] >= 0, seen[rows, np.maximum(up, 0)], False)
        seen[:, i, i] = True
    return seen


def _words(seen):
    """Bits of [..., n] truth values in 32-bit words [..., ceil(n / 32)], bit j % 32 of word j / 32."""
    n = seen.shape[-1]
    words = (n + 31) // 32
    bits = torch.nn.functional.pad(seen.to(torch.int64), (0, words * 32 - n))
    bits = bits.reshape(*seen.shape[:-1], words, 32) << torch.arange(32, device=seen.device)
    return bits.sum(-1).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator().manual_seed(seed * 2 + 1)
    gd = torch.Generator(device=DEV).manual_seed(seed * 2)
    s = {"case": c}
    d, hkv = c["d"], c["hkv"]
    if c["op"] in ("tree", "window_decode"):
        batch, hq = c["batch"], c["hq"]
        rows = c["nodes"] if c["op"] == "tree" else c["sq"]
        ctx = _ints(g, c["lo"], c["hi"], batch)
        if c["op"] == "tree":
            nodes = _ints(g, 1, rows, batch) if c["ragged"] else [rows] * batch
            lens = [n + t for n, t in zip(ctx, nodes)]
            parents = _tree(g, batch, rows)
            s["parents"] = parents.to(DEV)
            s["mask"] = _words(torch.from_numpy(_ancestors(parents)).to(DEV))
            s["tree_lens"] = _i32(nodes) if c["ragged"] else None
        else:
            lens = ctx
        s["q"] = _randn(gd, batch, hq, rows, d)
        if c["page"]:
            s["k"], s["v"], s["table"] = _paged(gd, g, lens, hkv, c["page"], d)
        else:
            s["k"], s["v"] = (_randn(gd, batch, hkv, max(lens), d) for _ in range(2))
        s["lens"] = _i32(lens)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(batch, hq, rows, device=DEV)
    elif c["op"] == "window_prefill":
        batch, hq = c["batch"], c["hq"]
        q_lens = _ints(g, c["qlo"], c["qhi"], batch)
        past = _ints(g, c["plo"], c["phi"], batch)
        lens = [a + b for a, b in zip(q_lens, past)]
        s["lens"] = _i32(lens)
        if not c["packed"]:
            s["q"] = _randn(gd, batch, hq, c["qhi"], d)
            s["k"], s["v"] = (_randn(gd, batch, hkv, c["qhi"], d) for _ in range(2))
        else:
            s["cu_q"] = _i32([0] + np.cumsum(q_lens).tolist())
            s["max_q"], s["max_k"] = max(q_lens), max(lens)
            s["q"] = _randn(gd, sum(q_lens), hq, d)
            if c["page"]:
                s["k"], s["v"], s["table"] = _paged(gd, g, lens, hkv, c["page"], d)
            else:
                s["cu_k"] = _i32([0] + np.cumsum(lens).tolist())
                s["k"], s["v"] = (_randn(gd, sum(lens), hkv, d) for _ in range(2))
    elif c["op"] == "accept":
        batch, nodes = c["batch"], c["nodes"]
        ctx = _ints(g, c["lo"], c["hi"], batch)
        new = _ints(g, 1, nodes, batch)
        s["k"], s["v"], s["table"] = _paged(gd, g, ctx, hkv, c["page"], d, more=nodes)
        s["lens"], s["n_new"] = _i32(ctx), _i32(new)
        # rows as a projection leaves them: token by token, heads side by side
        s["k_new"], s["v_new"] = (_randn(gd, batch, nodes, hkv, d).transpose(1, 2) for _ in range(2))
        keep = torch.zeros(batch, nodes, dtype=torch.int32)
        kept = []
        for b, t in enumerate(new):   # an accepted path: ascending nodes
            n = int(torch.randint(1, max(1, t // 2) + 1, (1,), generator=g))
            keep[b, :n] = torch.randperm(t, generator=g)[:n].sort().values.to(torch.int32)
            kept.append(n)
        s["keep"], s["n_keep"] = keep.to(DEV), _i32(kept)
    else:
        groups, samples, page = c["groups"], c["samples"], c["page"]
        lens = _ints(g, c["lo"], c["hi"], groups)
        need = [-(-n // page) for n in lens]
        width = -(-(max(lens) + c["extra"]) // page)
        forks = groups * samples
        spare = forks * (2 + c["extra"] // page)
        pages = sum(need) + spare + 1          # the last page stays out of the pool
        order = torch.randperm(pages - 1, generator=g).to(torch.int32)
        table = torch.full((groups + forks, width), -1, dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            refs[order[at:at + n].long()] = 1
            at += n
        refs[pages - 1] = 1
        s["k"], s["v"] = (_randn(gd, pages, hkv, page, d) for _ in range(2))
        s["table"], s["refs"] = table.to(DEV), refs.to(DEV)
        s["lens"] = _i32(lens + [0] * forks)
        s["src"] = _i32([i // samples for i in range(forks)])
        s["dst"] = _i32([groups + i for i in range(forks)])
        s["extra"] = _i32([0] * groups + [c["extra"]] * forks)
        s["k_new"], s["v_new"] = (_randn(gd, groups + forks, c["extra"], hkv, d).transpose(1, 2)
                                  for _ in range(2))
    if c.get("sinks"):
        s["sinks"] = torch.randn(c["hq"], generator=gd, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----

def _from_pages(cache, table):
    """[batch, heads, keys, d] of a paged cache."""
    x = cache[table.clamp(min=0).long()]                # [batch, pages, heads, page, d]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend(q, k, v, seen, sinks):
    """Masked softmax attention in 32 bits: q [b, hq, n, d], k, v [b, hkv, m, d], seen [b, n, m]."""
    batch, hq, n, d = q.shape
    hkv = k.shape[1]
    qg = q.float().reshape(batch, hkv, hq // hkv * n, d)
    score = torch.matmul(qg, k.float().transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = score.reshape(batch, hq, n, -1)
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks.reshape(1, -1, 1, 1))
    base = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - base)
    total = p.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks.reshape(1, -1, 1, 1) - base)
    o = torch.matmul(p.reshape(batch, hkv, hq // hkv * n, -1), v.float()).reshape(batch, hq, n, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, base + torch.log(total), -math.inf)
    return o.to(torch.bfloat16), lse[..., 0]


def _unpack(mask, nodes):
    bits = (mask[..., None] >> torch.arange(32, device=mask.device)) & 1
    return bits.reshape(*mask.shape[:-1], -1)[..., :nodes].bool()


def _mask_of_parents(parents):
    batch, n = parents.shape
    at = torch.arange(n, device=parents.device)
    seen = (parents[..., None] == at) | (at[:, None] == at)
    for _ in range((n - 1).bit_length()):               # paths of twice the length
        seen = torch.matmul(seen.float(), seen.float()) > 0
    return _words(seen)


def _plain_tree(s):
    c = s["case"]
    n = c["nodes"]
    mask = _mask_of_parents(s["parents"]) if c["fresh"] else s["mask"]
    k, v = (_from_pages(s[x], s["table"]) if c["page"] else s[x] for x in "kv")
    lens = s["lens"][:, None, None]
    t = s["tree_lens"][:, None, None] if c["ragged"] else n
    key = torch.arange(k.shape[2], device=DEV)
    node = (key - (lens - t)).expand(c["batch"], n, -1)   # node of each key
    bits = torch.gather(_unpack(mask, n), 2, node.clamp(0, n - 1))
    seen = ((node < 0) | bits) & (key < lens)
    o, lse = _attend(s["q"], k, v, seen, s.get("sinks"))
    if c["ragged"]:   # rows past a tree's nodes stay as they were
        real = torch.arange(n, device=DEV) < t[:, 0]
        o = torch.where(real[:, None, :, None], o, s["out"])
        lse = torch.where(real[:, None, :], lse, s["lse"])
    return {"o": o, "lse": lse, "mask": mask} if c["fresh"] else {"o": o, "lse": lse}


def _seen_in_window(c, place, key, lens):
    """place: the queries' key positions [b, n, 1]; key [m]; lens [b, 1, 1]."""
    return (key < lens) & (key <= place) & ((key > place - c["window"]) | (key < c["first"]))


def _plain_window(s):
    c = s["case"]
    lens = s["lens"][:, None, None]
    if c["op"] == "window_decode" or not c["packed"]:
        k, v = (_from_pages(s[x], s["table"]) if c["page"] else s[x] for x in "kv")
        n = s["q"].shape[2]
        place = torch.arange(n, device=DEV)[:, None] + lens - n
        key = torch.arange(k.shape[2], device=DEV)
        o, lse = _attend(s["q"], k, v, _seen_in_window(c, place, key, lens), s.get("sinks"))
        return {"o": o, "lse": lse}
    q, cu = s["q"], s["cu_q"].long()
    at = torch.arange(s["max_q"], device=DEV)
    n_q = (cu[1:] - cu[:-1])[:, None]
    padded = q[(cu[:-1, None] + at).clamp(max=q.shape[0] - 1)].transpose(1, 2)
    if c["page"]:
        k, v = (_from_pages(s[x], s["table"]) for x in "kv")
    else:
        token = s["cu_k"][:-1, None].long() + torch.arange(s["max_k"], device=DEV)
        token = token.clamp(max=s["k"].shape[0] - 1)
        k, v = (s[x][token].transpose(1, 2) for x in "kv")
    place = (at + s["lens"][:, None] - n_q)[..., None]
    key = torch.arange(k.shape[2], device=DEV)
    o, lse = _attend(padded, k, v, _seen_in_window(c, place, key, lens), s.get("sinks"))
    row = torch.arange(q.shape[0], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return {"o": o[seq, :, row - cu[seq]], "lse": lse[seq, :, row - cu[seq]].transpose(0, 1).contiguous()}


def _put(cache, page, slot, rows, real):
    """cache[page, :, slot] = rows where real; the others go to the spare page as it is."""
    spare = cache.shape[0] - 1
    rows = torch.where(real[..., None, None], rows, cache[spare, :, 0])
    cache[torch.where(real, page, spare).long(), :, torch.where(real, slot, 0).long()] = rows


def _page_of(table, place, page):
    at = (place // page).clamp(0, table.shape[1] - 1)
    return torch.gather(table, 1, at.long())


def _plain_append(s, count):
    page, table = s["case"]["page"], s["table"]
    n = s["k_new"].shape[2]
    i = torch.arange(n, device=DEV)
    place = s["lens"][:, None] + i
    for cache, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
        _put(cache, _page_of(table, place, page), place % page, new.transpose(1, 2), i < count[:, None])


def _plain_accept(s):
    page, table = s["case"]["page"], s["table"]
    _plain_append(s, s["n_new"])
    a = torch.arange(s["keep"].shape[1], device=DEV)
    old, new = s["lens"][:, None] + s["keep"], s["lens"][:, None] + a
    for cache in (s["k"], s["v"]):
        rows = cache[_page_of(table, old, page).clamp(min=0).long(), :, (old % page).long()]
        _put(cache, _page_of(table, new, page), new % page, rows, a < s["n_keep"][:, None])
    return {"k": s["k"], "v": s["v"]}


def _plain_fork(s):
    page, table, refs, lens = s["case"]["page"], s["table"], s["refs"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    # free what an earlier pass left in the rows
    held = table[dst].reshape(-1)
    refs.index_add_(0, held.clamp(min=0).long(), -(held >= 0).to(torch.int32))
    # fork: share every page
    pages = table[src]
    table[dst] = pages
    lens[dst] = lens[src]
    held = pages.reshape(-1)
    refs.index_add_(0, held.clamp(min=0).long(), (held >= 0).to(torch.int32))
    # reserve: pages that are missing or shared where rows will be written
    at = torch.arange(table.shape[1], device=DEV)
    first, last = lens[:, None] // page, (lens[:, None] + s["extra"][:, None] + page - 1) // page
    shared = (table >= 0) & (refs[table.clamp(min=0).long()] > 1)
    need = (at >= first) & (at < last) & ((table < 0) | shared)
    rank = torch.cumsum(need.reshape(-1), 0).reshape(need.shape) - 1
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)
    lack = (need.sum() - (refs == 0).sum()).clamp(min=0)
    need = need & (lack == 0)
    new = free[rank.clamp(0, free.numel() - 1)]
    old = table.clone()
    gone, come = (need & shared).reshape(-1), need.reshape(-1)
    refs.index_add_(0, old.reshape(-1).clamp(min=0).long(), -gone.to(torch.int32))
    refs.index_add_(0, new.reshape(-1).long(), come.to(torch.int32))
    table.copy_(torch.where(need, new, table))
    # copies: the page that holds a row's last keys, where it was shared
    at_first = first.clamp(max=table.shape[1] - 1).long()
    moved = torch.gather(need & shared, 1, at_first)[:, 0] & (lens % page > 0)
    copies = torch.stack([torch.gather(old, 1, at_first)[:, 0], torch.gather(table, 1, at_first)[:, 0],
                          lens % page], 1)
    copies = torch.where(moved[:, None], copies, _NO_COPY.to(DEV))
    slot = torch.arange(page, device=DEV)
    for cache in (s["k"], s["v"]):
        rows = cache[copies[:, 0].clamp(min=0).long()].transpose(1, 2)
        _put(cache, copies[:, 1:2].expand(-1, page), slot.expand(copies.shape[0], -1), rows,
             slot < copies[:, 2:3])
    _plain_append(s, s["extra"])
    return {"k": s["k"], "v": s["v"], "table": table, "refs": refs, "lens": lens, "copies": copies,
            "status": lack.to(torch.int32).reshape(1)}


_NO_COPY = torch.tensor([-1, -1, 0], dtype=torch.int32)


# ------------------------------------------------------- the framework's calls ----

def _own(s):
    from attention_forward_blackwell_gb300 import binding as fa
    c = s["case"]
    if c["op"] == "tree":
        mask = fa.tree_mask(s["parents"]) if c["fresh"] else s["mask"]
        more = dict(tree_lens=s["tree_lens"], sinks=s.get("sinks"), out=s["out"], lse=s["lse"])
        if c["page"]:
            o, lse = fa.decode_tree_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], mask, **more)
        else:
            o, lse = fa.decode_tree(s["q"], s["k"], s["v"], mask, seqlens_k=s["lens"], **more)
        return {"o": o, "lse": lse, "mask": mask} if c["fresh"] else {"o": o, "lse": lse}
    if c["op"] == "accept":
        fa.cache_append(s["k"], s["v"], s["table"], s["lens"], s["k_new"], s["v_new"], n_new=s["n_new"])
        fa.cache_compact(s["k"], s["v"], s["table"], s["lens"], s["keep"], s["n_keep"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "fork":
        fa.cache_free(s["refs"], s["table"], s["lens"], s["dst"])
        fa.cache_fork(s["refs"], s["table"], s["lens"], s["src"], s["dst"])
        copies, status = fa.cache_reserve(s["refs"], s["table"], s["lens"], s["extra"], c["page"])
        fa.cache_append(s["k"], s["v"], s["table"], s["lens"], s["k_new"], s["v_new"], n_new=s["extra"],
                        copies=copies)
        return {"k": s["k"], "v": s["v"], "table": s["table"], "refs": s["refs"], "lens": s["lens"],
                "copies": copies, "status": status}
    more = dict(causal=True, window=c["window"], first=c["first"], sinks=s.get("sinks"))
    if c["op"] == "window_decode":
        more.update(out=s["out"], lse=s["lse"])
        if c["page"]:
            o, lse = fa.decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], **more)
        else:
            o, lse = fa.decode(s["q"], s["k"], s["v"], seqlens_k=s["lens"], **more)
    elif not c["packed"]:
        o, lse = fa.prefill(s["q"], s["k"], s["v"], **more)
    elif c["page"]:
        o, lse = fa.prefill_varlen_paged(s["q"], s["k"], s["v"], s["cu_q"], s["max_q"], s["table"],
                                         s["lens"], **more)
    else:
        o, lse = fa.prefill_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                                   **more)
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tree":
        return _plain_tree(state)
    if op == "accept":
        return _plain_accept(state)
    if op == "fork":
        return _plain_fork(state)
    return _plain_window(state)


# --------------------------------------------------------------- 64 bits ----

def _exact_rows(q, k, v, seen, sinks):
    """Definition of one sequence: q [hq, n, d], k, v [hkv, m, d], seen [n, m]; O and LSE in 64 bits."""
    hq, n, d = q.shape
    hkv = k.shape[0]
    o = torch.zeros(hq, n, d, dtype=torch.float64, device=DEV)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=DEV)
    for h in range(hq):
        x = q[h].double() @ k[h * hkv // hq].double().T / math.sqrt(d)
        x.masked_fill_(~seen, -math.inf)
        if sinks is not None:
            x = torch.cat([x, sinks[h].double().expand(n, 1)], 1)
        if x.shape[1] == 0:
            continue
        lse[h] = torch.logsumexp(x, 1)
        p = torch.exp(x - torch.where(lse[h] == -math.inf, 0.0, lse[h])[:, None])
        o[h] = p[:, :k.shape[1]] @ v[h * hkv // hq].double()
    return o, lse


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("accept", "fork"):
        return None
    s = prepare(c, seed)
    packed = c.get("packed", False)
    out, lses = [], []
    for b in range(c["batch"]):
        length = int(s["lens"][b])
        if packed:
            lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
            q = s["q"][lo:hi].transpose(0, 1)
        else:
            q = s["q"][b]
        n = q.shape[1]
        if c["page"]:
            token = torch.arange(length, device=DEV)
            page = s["table"][b].long()[token // c["page"]]
            k, v = (s[x][page, :, token % c["page"]].transpose(0, 1) for x in "kv")
        elif packed:
            at = int(s["cu_k"][b])
            k, v = (s[x][at:at + length].transpose(0, 1) for x in "kv")
        else:
            k, v = (s[x][b, :, :length] for x in "kv")
        if c["op"] == "tree":
            t = int(s["tree_lens"][b]) if c["ragged"] else n
            parents = s["parents"][b].tolist()
            seen = torch.zeros(n, length, dtype=torch.bool)
            seen[:, :length - t] = True
            for i in range(t):
                node = i
                while node >= 0:
                    seen[i, length - t + node] = True
                    node = parents[node]
            o, lse = _exact_rows(q, k, v, seen.to(DEV), s.get("sinks"))
            o[:, t:], lse[:, t:] = 0.0, 0.0             # left as the buffers were
        else:
            place = torch.arange(length - n, length, device=DEV)[:, None]
            key = torch.arange(length, device=DEV)[None]
            seen = (place - key >= 0) & ((place - key < c["window"]) | (key < c["first"]))
            o, lse = _exact_rows(q, k, v, seen, s.get("sinks"))
        out.append(o)
        lses.append(lse)
    if packed:
        return {"o": torch.cat(out, 1).transpose(0, 1).contiguous(), "lse": torch.cat(lses, 1)}
    got = {"o": torch.stack(out), "lse": torch.stack(lses)}
    if c.get("fresh"):
        got["mask"] = None
    return got
