"""Plain 64-bit forms of rotated positions and of a key/value cache held in 8 bits, and the error
bounds of the kernels' outputs."""
from __future__ import annotations

import math

import torch

F8 = torch.float8_e4m3fn


def turn64(x, positions, inv_freq, factor=1.0, interleaved=False, inverse=False):
    """Rows x [..., n, d] at positions that broadcast over [..., n], turned in 64 bits."""
    x, w = x.double(), torch.as_tensor(inv_freq, dtype=torch.float64)
    rot = 2 * w.numel()
    angle = positions.double()[..., None] * w * (-1.0 if inverse else 1.0)
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    out = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                             slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    return out


def turn_bound(x, y, positions, rot, factor, interleaved):
    """Bound of a turned row y of x in bf16: 2^-8 of the value for its rounding.  Before it, in fp32, a
    sine or cosine is off by 2^-22: 2^-24 pi / 2 of a rounding of the fraction of half a turn to 24 bits,
    2^-29 of its cut to 2^-32 of a turn, 1.6e-7 of the polynomials and their roundings, 2^-24 of the
    factor's product.  A turned element is then off by sqrt(2) 2^-22 of its pair's length, and by three
    roundings of 2^-24: 5.2e-7 of it in all, below 2^-20.  Zero for elements that are not turned."""
    x = x.double().abs()
    size = torch.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    length = factor * torch.hypot(a, b) * 2.0 ** -20
    if interleaved:
        size[..., 0:rot:2] = size[..., 1:rot:2] = length
    else:
        size[..., :rot // 2] = size[..., rot // 2:rot] = length
    turned = torch.zeros_like(x)
    turned[..., :rot] = 1
    return turned * 2.0 ** -8 * y.abs() + size * (1 + 2.0 ** -8)


def round8(x):
    """e4m3 values next to x, ties to even, 448 at most, in 64 bits."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(x), e)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def half_step(x):
    """Half a step of e4m3 at x."""
    e = torch.frexp(x.abs())[1].clamp(min=-5) - 5
    return torch.ldexp(torch.ones_like(x), e)


def scale_for(reach):
    if reach <= 0:
        return 2.0 ** -54
    e = math.ceil(math.log2(reach / 448.0))
    while 448.0 * 2.0 ** e < reach:
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= reach:
        e -= 1
    return 2.0 ** max(-54, min(54, e))


def reach64(x, rot, factor, interleaved):
    """Reach of rows x [..., d]."""
    x = x.double()
    most = x[..., rot:].abs().max().item() if x.shape[-1] > rot else 0.0
    if rot:
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        most = max(most, factor * (a * a + b * b).max().sqrt().item())
    return most


class Cache8:
    """The 8-bit cache's definition on the CPU: codes' values and scales in 64 bits, and how far the
    kernels' values may be off (in codes)."""

    def __init__(self, k, v, k_scale, v_scale):
        self.codes = [k.cpu().double(), v.cpu().double()]
        self.scales = [k_scale.cpu().double(), v_scale.cpu().double()]
        self.slack = [torch.zeros_like(c) for c in self.codes]
        self.page = k.shape[2]
        self.block = self.page // k_scale.shape[2]

    def copy(self, copies):
        for i in range(2):
            codes, scales, slack = self.codes[i].clone(), self.scales[i].clone(), self.slack[i].clone()
            pages = codes.shape[0]
            for s, d, r in copies:
                if not (0 <= s < pages and 0 <= d < pages and s != d):
                    continue
                self.codes[i][d, :, :r] = codes[s, :, :r]
                self.slack[i][d, :, :r] = slack[s, :, :r]
                nb = -(-r // self.block)
                self.scales[i][d, :, :nb] = scales[s, :, :nb]

    def append(self, table, lens, k_new, v_new, counts, turn=None, positions=None):
        """k_new, v_new [B, H, n, d]; turn: (inv_freq, factor, interleaved) or None."""
        for i, new in enumerate((k_new, v_new)):
            new = new.cpu()
            turned = turn if i == 0 else None
            for b, count in enumerate(counts):
                for p0 in range(lens[b] // self.block * self.block, lens[b] + max(count, 0), self.block):
                    lo, hi = max(p0, lens[b]), min(p0 + self.block, lens[b] + count)
                    if lo >= hi or p0 // self.page >= len(table[b]):
                        continue
                    page = table[b][p0 // self.page]
                    if not 0 <= page < self.codes[i].shape[0]:
                        continue
                    row, blk = p0 % self.page, p0 % self.page // self.block
                    x = new[b, :, lo - lens[b]:hi - lens[b]]
                    at = torch.arange(lo, hi) if positions is None else positions[b, lo - lens[b]:hi - lens[b]]
                    y = turn64(x, at, *turned) if turned else x.double()
                    for h in range(x.shape[0]):
                        rot, f, il = (2 * len(turned[0]), turned[1], turned[2]) if turned else (0, 1.0, False)
                        s = scale_for(reach64(x[h], rot, f, il))
                        old = self.scales[i][page, h, blk].item()
                        if lo > p0:
                            s = max(s, old)
                            part = self.codes[i][page, h, row:row + lo - p0]
                            slack = self.slack[i][page, h, row:row + lo - p0]
                            new_part = round8(part * (old / s))
                            if s != old:   # what a code was off, and a rounding that may fall otherwise
                                slack = torch.where(slack > 0, slack * (old / s) + 2 * half_step(new_part), slack)
                            self.codes[i][page, h, row:row + lo - p0] = new_part
                            self.slack[i][page, h, row:row + lo - p0] = slack
                        z = y[h] / s
                        r0 = row + lo - p0
                        self.codes[i][page, h, r0:r0 + hi - lo] = z = round8(z)
                        # a turned element is off by 2^-20 of its pair: the code may be the other of two
                        near = torch.zeros_like(z)
                        if rot:
                            near[..., :rot] = 2 * half_step(z)[..., :rot]
                        self.slack[i][page, h, r0:r0 + hi - lo] = near
                        self.scales[i][page, h, blk] = s

    def values(self, i):
        c = self.codes[i]
        return (c.unflatten(2, (-1, self.block)) * self.scales[i][..., None, None]).flatten(2, 3)


def codes8(gen, pages, heads, page, block, d, spread=0.7, device="cuda"):
    """Random codes and power-of-two scales, magnitudes of their own for every block and head."""
    x = torch.randn(pages, heads, page // block, block * d, generator=gen)
    x = x * torch.exp(spread * torch.randn(pages, heads, page // block, 1, generator=gen))
    s = torch.tensor([scale_for(v) for v in x.abs().amax(-1).flatten().tolist()]).reshape(x.shape[:-1])
    return (x / s[..., None]).to(F8).reshape(pages, heads, page, d).to(device), s.float().to(device)


def attention8(q, k, v, vs, seen, scale, sinks=None):
    """q [B, Hq, n, d] bf16, values k, v [B, Hkv, m, d] in 64 bits, scales vs [B, Hkv, m] of the values,
    seen bool [B, n, m].  Returns (o, lse, bound_o, bound_lse).

    Bounds.  Products of fp16 queries and codes are exact and summed in fp32, the sum is multiplied by two
    factors: off by (d + 8) 2^-24 scale sum |q k|.  A query element below 2^-14 of its row's largest is off
    by 2^-25 of that: 2^-25 max|q| scale sum |k| more.  e is their sum.  A probability is off by a relative
    e, s = m 2^-24 + 2^-16 covers sums over m keys, approximate exp2 and log2 (2^-22 each), the
    roundings of exponents up to 64 (2^-18) and the rescalings; times its value's scale it is rounded to fp16:
    2^-11, or 2^-31 of the largest such product where it is small (fp16's smallest step 2^-24, halved, and
    2^6 of headroom), times a code of at most 448.  With a = sum p |v|: |do| <= 2^-8 |o| + (2^-11 +
    2 e + s)(1 + 2^-8) a + 448 m 2^-31 max(p s_v).
    """
    q, k, v, vs = (t.detach().double().cpu() for t in (q, k, v, vs))
    B, Hq, n, d = q.shape
    G, m = Hq // k.shape[1], k.shape[2]
    o = torch.zeros(B, Hq, n, d, dtype=torch.float64)
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for h in range(Hq):
            kk = torch.where(seen[b].any(0)[:, None], k[b, h // G], 0.0)
            vv = torch.where(seen[b].any(0)[:, None], v[b, h // G], 0.0)
            ss = torch.where(seen[b].any(0), vs[b, h // G], 0.0)
            x = torch.where(seen[b], q[b, h] @ kk.T * scale, -math.inf)
            e = q[b, h].abs() @ kk.abs().T * (d + 8) * 2.0 ** -24
            e = e + q[b, h].abs().amax(1, keepdim=True) * kk.abs().sum(1) * 2.0 ** -25
            e = (torch.where(seen[b], e, 0.0).amax(1) if m else torch.zeros(n, dtype=torch.float64)) * scale
            if sinks is not None:
                x = torch.cat([x, sinks[h].double().cpu().expand(n, 1)], 1)
            if x.shape[1] == 0:
                continue
            l = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None])[:, :m]
            p = torch.where(seen[b], p, 0.0)
            o[b, h], lse[b, h] = p @ vv, l
            a = p @ vv.abs()
            s = m * 2.0 ** -24 + 2.0 ** -16
            low = 448 * m * 2.0 ** -31 * ((p * ss).amax(1) if m else torch.zeros(n, dtype=torch.float64))
            bo[b, h] = (2.0 ** -8 * o[b, h].abs()
                        + (2.0 ** -11 + 2 * e[:, None] + s) * (1 + 2.0 ** -8) * a + low[:, None])
            bl[b, h] = e + s * (1 + torch.where(l == -math.inf, 0.0, l).abs())
    return o, lse, bo, bl
