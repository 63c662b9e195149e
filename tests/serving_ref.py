"""Plain 64-bit forms of the serving operators (token trees, a window with
visible first tokens, cache pages) and the error bounds of the kernels' outputs."""
from __future__ import annotations

import math

import numpy as np
import torch


def attention64(q, k, v, seen, scale, sinks=None):
    """q [B, Hq, n, d], k, v [B, Hkv, m, d] (any float type), seen bool
    [B, n, m]: masked softmax attention in 64 bits on the CPU.  Returns
    (o, lse, bound_o, bound_lse).

    Bounds.  A score is a sum of d products of bf16 values (exact in fp32)
    accumulated and scaled in fp32: off by at most e = (d + 3) 2^-24 scale
    sum |q k|.  A probability then is off by a relative e (and the softmax's
    denominator too), 2^-8 more when it is rounded to bf16 for the value
    product, and o is rounded to bf16 at the end: with a = sum p |v| / l,
    |do| <= 2^-8 (|o| + a) + (2 e + s) a, the denominator and LSE without the
    2^-8.  s = m 2^-24 + 2^-18 covers the sums over m keys, the approximate
    exp2 and log2 (relative 2^-22 each) and the rescalings.
    """
    q, k, v = (t.detach().double().cpu() for t in (q, k, v))
    seen = seen.cpu()
    B, Hq, n, d = q.shape
    G = Hq // k.shape[1]
    m = k.shape[2]
    o = torch.zeros(B, Hq, n, d, dtype=torch.float64)
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for h in range(Hq):
            kk, vv = k[b, h // G], v[b, h // G]
            x = torch.where(seen[b], q[b, h] @ kk.T * scale, -math.inf)
            e = torch.where(seen[b], (q[b, h].abs() @ kk.abs().T) * scale, 0.0)
            e = (e.amax(1) if m else torch.zeros(n)) * (d + 3) * 2.0 ** -24
            if sinks is not None:
                x = torch.cat([x, sinks[h].double().cpu().expand(n, 1)], 1)
            if x.shape[1] == 0:
                continue
            l = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None])[:, :m]
            p = torch.where(seen[b], p, 0.0)
            vv = torch.where(seen[b].any(0)[:, None], vv, 0.0)
            o[b, h], lse[b, h] = p @ vv, l
            a = p @ vv.abs()
            s = m * 2.0 ** -24 + 2.0 ** -18
            bo[b, h] = 2.0 ** -8 * (o[b, h].abs() + a) + (2 * e[:, None] + s) * a
            bl[b, h] = e + s * (1 + torch.where(l == -math.inf, 0.0, l).abs())
    return o, lse, bo, bl


def check(o, lse, ref, what="", rows=None):
    """Compares with attention64's result; rows bool [B, n]: the rows that count."""
    ro, rl, bo, bl = ref
    o, lse = o.detach().double().cpu(), lse.detach().double().cpu()
    if rows is None:
        rows = torch.ones(ro.shape[0], ro.shape[2], dtype=torch.bool)
    rows = rows[:, None].expand(-1, ro.shape[1], -1)
    o, lse, ro, rl, bo, bl = (t[rows] for t in (o, lse, ro, rl, bo, bl))
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty), f"{what}: rows without keys differ"
    assert torch.all(o[empty] == 0), f"{what}: a row without keys is not zero"
    do, dl = (o - ro).abs(), (lse - rl).abs()[~empty]
    print(f"{what}: max|dO|={do.max().item() if do.numel() else 0:.2e} "
          f"max|dLSE|={dl.max().item() if dl.numel() else 0:.2e}")
    assert torch.all(do <= bo), f"{what}: O off by {(do - bo).max().item():.2e} over its bound"
    assert torch.all(dl <= bl[~empty]), f"{what}: LSE off"


def window_seen(n, lens, m, window, first, causal):
    """seen [B, n, m] of a window whose first keys stay visible."""
    i, j = torch.arange(n)[:, None], torch.arange(m)[None]
    out = []
    for L in lens:
        p = i + L - n
        s = (j < L).expand(n, m).clone()
        if causal:
            s &= j <= p
        if window > 0:
            s &= (j > p - window) | (j < first)
        out.append(s)
    return torch.stack(out)


def tree_seen(bits, lens, nodes, m):
    """seen [B, T, m] of tree bits [B, T, T] over lens keys, the last nodes[b] the trees'."""
    B, T, _ = bits.shape
    seen = torch.zeros(B, T, m, dtype=torch.bool)
    for b in range(B):
        base = lens[b] - nodes[b]
        for j in range(lens[b]):
            seen[b, :, j] = True if j < base else bits[b, :, j - base]
    return seen


def pack_bits(bits):
    """int32 words [..., ceil(T / 32)] of truth values [..., T]."""
    T = bits.shape[-1]
    W = (T + 31) // 32
    x = np.zeros(bits.shape[:-1] + (W * 32,), dtype=np.uint8)
    x[..., :T] = bits.cpu().numpy()
    words = np.packbits(x, axis=-1, bitorder="little").view(np.uint32)
    return torch.from_numpy(words.astype(np.int64)).to(torch.int64).where(
        torch.from_numpy(words < 2 ** 31), torch.from_numpy(words.astype(np.int64)) - 2 ** 32
    ).to(torch.int32)


def ancestors(parents):
    """bits [B, T, T] of trees: each node sees itself and its way up."""
    B, T = parents.shape
    bits = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            x = i
            while x >= 0:
                bits[b, i, x] = True
                up = int(parents[b, x])
                x = up if up < x else -1
    return bits


class Pool:
    """The page operators' definition, on lists of whole numbers."""

    def __init__(self, refs, table, lens):
        self.refs, self.table, self.lens = refs.tolist(), table.tolist(), lens.tolist()

    def page(self, e):
        return 0 <= e < len(self.refs)

    def fork(self, src, dst):
        B = len(self.table)
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B) or self.lens[d] > 0 or d in dst[:i] or d in src \
                    or any(self.page(e) for e in self.table[d]):
                return 1 + i
        for s, d in zip(src, dst):
            self.table[d] = [e if self.page(e) else -1 for e in self.table[s]]
            for e in self.table[d]:
                if self.page(e):
                    self.refs[e] += 1
            self.lens[d] = self.lens[s]
        return 0

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for j, e in enumerate(self.table[r]):
                    if self.page(e):
                        self.refs[e] -= 1
                    self.table[r][j] = -1
                self.lens[r] = 0

    def reserve(self, extra, P):
        none = [[-1, -1, 0] for _ in self.table]
        need = []
        for r, x in enumerate(extra):
            if x < 0:
                continue
            first, last = self.lens[r] // P, -(-(self.lens[r] + x) // P)
            if last > len(self.table[r]):
                return none, -1 - r
            for j in range(first, last):
                e = self.table[r][j]
                if not self.page(e) or self.refs[e] > 1:
                    need.append((r, j))
        free = [p for p, n in enumerate(self.refs) if n == 0]
        if len(free) < len(need):
            return none, len(need) - len(free)
        for (r, j), p in zip(need, free):
            e = self.table[r][j]
            if self.page(e):
                self.refs[e] -= 1
                if j == self.lens[r] // P and self.lens[r] % P:
                    none[r] = [e, p, self.lens[r] % P]
            self.table[r][j] = p
            self.refs[p] = 1
        return none, 0


def append_rows(cache, table, lens, new, counts, copies=None):
    """In place, on the CPU: cache [pages, H, P, d], new [B, H, n, d]."""
    pages, _, P, _ = cache.shape
    before = cache.clone()
    if copies is not None:
        for s, d, r in copies:
            if 0 <= s < pages and 0 <= d < pages:
                cache[d, :, :r] = before[s, :, :r]
    for b, n in enumerate(counts):
        for i in range(n):
            pos = lens[b] + i
            if pos // P < len(table[b]) and 0 <= table[b][pos // P] < pages:
                cache[table[b][pos // P], :, pos % P] = new[b, :, i]


def compact_rows(cache, table, start, keep):
    """In place, on the CPU: key start[b] + a takes key start[b] + keep[b][a]."""
    P = cache.shape[2]
    before = cache.clone()
    for b, ks in enumerate(keep):
        for a, x in enumerate(ks):
            s, d = start[b] + x, start[b] + a
            cache[table[b][d // P], :, d % P] = before[table[b][s // P], :, s % P]
