"""Decode attention over a paged cache held in 8 bits against 64 bits (GPU)."""
import math

import pytest
import torch

import q8_ref as ref
import serving_ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
NAN8 = 0x7f


@pytest.fixture(scope="module")
def fa():
    from attention_forward_blackwell_gb300 import binding
    binding.lib()
    return binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(seed, lens, hkv, d, page, block, width=None, spread=0.7):
    """Caches of sequences whose pages lie in a random order; all that no key fills is NaN, scales too."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=g).tolist()
    width = width or max(1, max(need))
    table = []
    for n in need:
        table.append(order[:n] + [-1] * (width - n))
        order = order[n:]
    pages = sum(need) + 1
    out = []
    for _ in range(2):
        c, s = ref.codes8(g, pages, hkv, page, block, d, spread=spread, device="cpu")
        filled = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                filled[table[b][j // page], j % page] = True
        c.view(torch.uint8)[~filled[:, None].expand(-1, hkv, -1)] = NAN8
        s[~filled.unflatten(1, (-1, block)).any(2)[:, None].expand(-1, hkv, -1)] = math.nan
        out.append((c, s))
    return g, table, out


def gathered(table, lens, codes, scale):
    """Values and scales [B, Hkv, m, (d)] in 64 bits (zeros where no key is)."""
    pages, H, page, d = codes.shape
    block, m = page // scale.shape[2], max(lens, default=0)
    x = torch.zeros(len(lens), H, m, d, dtype=torch.float64)
    s = torch.zeros(len(lens), H, m, dtype=torch.float64)
    for b, n in enumerate(lens):
        for j in range(n):
            p = table[b][j // page]
            if 0 <= p < pages:
                s[b, :, j] = scale[p, :, j % page // block].double()
                x[b, :, j] = codes[p, :, j % page].double() * s[b, :, j, None]
    return x, s


def run(fa, seed, lens, hq, hkv, n, d, page, block, causal=False, window=0, first=0, sinks=False, width=None,
        spread=0.7, scale=None, q_spread=0.0):
    g, table, ((kc, ks), (vc, vs)) = case(seed, lens, hkv, d, page, block, width, spread)
    q = torch.randn(len(lens), hq, n, d, generator=g)
    q = (q * torch.exp(q_spread * torch.randn(q.shape, generator=g))).bfloat16()
    sink = torch.randn(hq, generator=g) if sinks else None
    k, _ = gathered(table, lens, kc, ks)
    v, s = gathered(table, lens, vc, vs)
    seen = serving_ref.window_seen(n, lens, max(lens), window, first, causal)
    if window > 0:   # keys that no row of the sequence sees may hold anything
        for b, L in enumerate(lens):
            for j in range(L):
                if not seen[b, :, j].any():
                    at = (table[b][j // page], slice(None), j % page)
                    kc.view(torch.uint8)[at] = vc.view(torch.uint8)[at] = NAN8
    want = ref.attention8(q, k, v, s, seen, scale or d ** -0.5, sink)
    o, lse = fa.decode_paged_q8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), i32(table), i32(lens),
                                scale=scale, causal=causal, window=window, first=first,
                                sinks=sink.cuda() if sinks else None)
    serving_ref.check(o, lse, want, f"d {d} rows {hq // hkv * n}")


SHAPES = [  # lens, hq, hkv, n, d, page, block
    ([1], 1, 1, 1, 64, 16, 16), ([0, 1, 2], 2, 1, 1, 128, 16, 4), ([17, 300, 64], 8, 2, 1, 128, 64, 64),
    ([1000, 3], 4, 4, 1, 64, 48, 16), ([513, 511, 512], 16, 2, 1, 256, 128, 32), ([77, 2000], 16, 1, 1, 128, 100, 25),
    ([250, 31], 24, 1, 1, 64, 32, 32), ([1500], 32, 1, 1, 256, 256, 256), ([900, 128], 40, 2, 2, 128, 64, 16),
    ([129, 640], 8, 1, 16, 64, 16, 16), ([70, 3], 7, 7, 5, 128, 1, 1), ([333], 5, 1, 3, 256, 7, 7),
    ([2100, 90], 33, 1, 1, 128, 64, 64), ([77, 300], 4, 2, 1, 64, 7, 7), ([130, 5], 2, 1, 2, 64, 1, 1),
    ([400], 8, 1, 1, 64, 6, 3), ([90, 33], 4, 1, 1, 128, 10, 5), ([1300, 0, 7], 20, 1, 1, 64, 20, 10)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,n,d,page,block", SHAPES)
def test_plain(fa, lens, hq, hkv, n, d, page, block, causal):
    run(fa, d + hq, lens, hq, hkv, n, d, page, block, causal=causal, sinks=causal)


@pytest.mark.parametrize("lens,hq,hkv,n,d,page,block", SHAPES)
def test_wide_tables(fa, lens, hq, hkv, n, d, page, block):
    """Tables of many more pages than are filled: more splits than one cluster, most of them empty."""
    run(fa, d + hq + 1, lens, hq, hkv, n, d, page, block, causal=True, width=-(-6000 // page))


MANY = [  # lens, hq, hkv, n, d, page, block: several units to a piece, empty and long ones among them
    ([7 * i % 45 for i in range(300)], 4, 2, 1, 64, 16, 16), ([1500 if i % 23 == 5 else i % 40 for i in range(70)], 15, 3, 2, 128, 16, 8),
    ([0] * 40 + [700, 1, 64, 0, 65], 16, 8, 1, 256, 32, 32), ([200 + 13 * i for i in range(50)], 20, 4, 5, 64, 48, 12),
    ([130] * 257, 2, 2, 1, 128, 26, 13)]


@pytest.mark.parametrize("width", [None, 300])
@pytest.mark.parametrize("lens,hq,hkv,n,d,page,block", MANY)
def test_many_sequences(fa, lens, hq, hkv, n, d, page, block, width):
    run(fa, d + hq + 2, lens, hq, hkv, n, d, page, block, causal=True, width=width, sinks=width is None)


WINDOWS = [  # lens, hq, hkv, n, d, page, block, window, first, width
    ([300, 40, 0], 4, 1, 1, 128, 16, 16, 64, 0, None), ([300, 40, 5], 4, 2, 3, 64, 48, 12, 50, 4, None),
    ([3000, 900], 8, 1, 1, 128, 64, 64, 256, 130, 200), ([3000, 64], 16, 2, 4, 256, 128, 64, 1, 1, None),
    ([700], 2, 2, 16, 64, 32, 32, 33, 300, 300), ([2500, 2499], 8, 8, 1, 128, 100, 50, 2 ** 31 - 1, 3, None),
    ([1200], 6, 1, 2, 128, 16, 16, 500, 2 ** 31 - 1, None), ([990, 300], 4, 2, 2, 64, 15, 5, 100, 3, 400),
    ([400, 5000], 12, 2, 1, 64, 16, 4, 200, 70, None)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,n,d,page,block,window,first,width", WINDOWS)
def test_window(fa, lens, hq, hkv, n, d, page, block, window, first, width, causal):
    run(fa, d + window % 1000, lens, hq, hkv, n, d, page, block, causal=causal, window=window, first=first,
        sinks=True, width=width)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_far_apart(fa, d):
    """Blocks whose scales differ by many binades, keys' and values': the largest terms decide."""
    run(fa, d, [400, 150], 8, 1, 1, d, 32, 8, causal=True, spread=6.0, scale=0.01 * d ** -0.5)


def test_queries_of_many_binades(fa):
    run(fa, 3, [200, 333], 8, 1, 2, 128, 64, 16, causal=True, q_spread=3.0, scale=2e-3)


def test_scores_that_grow(fa):
    """Every slice with a larger maximum than the one before, and scores of hundreds of binades."""
    g = torch.Generator().manual_seed(1)
    n, d, page = 640, 64, 16
    k = torch.zeros(n // page, 1, page, d)
    k[..., 0] = torch.arange(n).reshape(n // page, 1, page) // 16 * 8.0
    scale_k = torch.ones(n // page, 1, 1)
    v, sv = ref.codes8(g, n // page, 1, page, page, d, device="cpu")
    kc = k.to(F8)
    for sign in (1.0, -1.0):
        q = torch.zeros(1, 3, 1, d)
        q[0, :, 0, 0] = sign * torch.tensor([1.0, 8.0, 0.125])
        q = q.bfloat16()
        table = [list(range(n // page))]
        kk, _ = gathered(table, [n], kc, scale_k)
        vv, s = gathered(table, [n], v, sv)
        want = ref.attention8(q, kk, vv, s, torch.ones(1, 1, n, dtype=torch.bool), 1.0)
        got = fa.decode_paged_q8(q.cuda(), kc.cuda(), v.cuda(), scale_k.cuda(), sv.cuda(), i32(table), i32([n]), scale=1.0)
        serving_ref.check(*got, want, "growing")


def test_values_of_scale_zero_and_no_pages(fa):
    """Values of scale 0 add nothing but their probabilities; entries that are no page read as zeros."""
    g, table, ((kc, ks), (vc, vs)) = case(5, [200, 90], 2, 128, 16, 16)
    q = torch.randn(2, 4, 1, 128, generator=g).bfloat16()
    for b, e in ((0, 3), (1, 0)):
        vs[table[b][e]] = 0.0
    table[0][5], table[1][2] = 10 ** 6, -4
    k, _ = gathered(table, [200, 90], kc, ks)
    v, s = gathered(table, [200, 90], vc, vs)
    want = ref.attention8(q, k, v, s, serving_ref.window_seen(1, [200, 90], 200, 0, 0, False), 128 ** -0.5)
    got = fa.decode_paged_q8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), i32(table), i32([200, 90]))
    serving_ref.check(*got, want, "zeros")


def test_long_cache_past_32_bits(fa):
    """Codes whose offsets pass 2^32 bytes, read by pages at both ends."""
    pages, hkv, page, d = 70000, 8, 64, 128      # 4.6 GB each
    kc = torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda").view(F8)
    vc = torch.zeros_like(kc.view(torch.uint8)).view(F8)
    ks, vs = (torch.ones(pages, hkv, 1, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    table = [[69999, 3, 68000, 69998, 0]]
    x = torch.randn(1, hkv, 300, d, generator=g).bfloat16().cuda()
    y = torch.randn(1, hkv, 300, d, generator=g).bfloat16().cuda()
    fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32([0]), x, y)
    sub = torch.tensor(table[0])
    k, _ = gathered([[0, 1, 2, 3, 4]], [300], kc.view(torch.uint8)[sub.cuda()].view(F8).cpu(), ks[sub.cuda()].cpu())
    v, s = gathered([[0, 1, 2, 3, 4]], [300], vc.view(torch.uint8)[sub.cuda()].view(F8).cpu(), vs[sub.cuda()].cpu())
    # (codes of values of about 4 / 448: within half a step)
    assert ((k - x.cpu().double()).abs() <= 2.0 ** -4 * x.cpu().double().abs() + 2.0 ** -16).all()
    q = torch.randn(1, 16, 1, d, generator=g).bfloat16()
    want = ref.attention8(q, k, v, s, torch.ones(1, 1, 300, dtype=torch.bool), d ** -0.5)
    got = fa.decode_paged_q8(q.cuda(), kc, vc, ks, vs, i32(table), i32([300]))
    serving_ref.check(*got, want, "long")
    kr, vr = fa.cache_read_q8(kc, vc, ks, vs, i32(table), i32([0, 300]), 300, 300)
    assert torch.equal(kr.cpu().double(), k[0].transpose(0, 1)) and torch.equal(vr.cpu().double(), v[0].transpose(0, 1))


def test_layouts_outputs_and_empty(fa):
    g, table, ((kc, ks), (vc, vs)) = case(5, [60, 90], 2, 64, 16, 16)
    kc, ks, vc, vs = (t.cuda() for t in (kc, ks, vc, vs))
    lens = i32([60, 90])
    q = torch.randn(2, 3, 4, 64, generator=g).bfloat16().cuda().transpose(1, 2)   # heads and rows swapped
    o, lse = fa.decode_paged_q8(q, kc, vc, ks, vs, i32(table), lens, causal=True)
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    r = fa.decode_paged_q8(q.contiguous(), kc, vc, ks, vs, i32(table).t().contiguous().t(), lens, causal=True, out=out, lse=l2)
    assert r[0] is out and torch.equal(out, o) and torch.equal(l2, lse)
    o, lse = fa.decode_paged_q8(q[:0], kc, vc, ks, vs, i32(table)[:0], lens[:0])
    assert o.shape == (0, 4, 3, 64)
    o, lse = fa.decode_paged_q8(q, kc, vc, ks, vs, i32(table), i32([0, -4]))
    assert torch.all(o == 0) and torch.all(lse == -math.inf)


def test_refusals(fa):
    g, table, ((kc, ks), (vc, vs)) = case(5, [60, 90], 2, 64, 16, 16)
    kc, ks, vc, vs, t, lens = kc.cuda(), ks.cuda(), vc.cuda(), vs.cuda(), i32(table), i32([60, 90])
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    call = fa.decode_paged_q8
    for bad in (lambda: call(q.float(), kc, vc, ks, vs, t, lens), lambda: call(q, kc.float(), vc.float(), ks, vs, t, lens),
                lambda: call(q, kc, vc, ks.double(), vs, t, lens), lambda: call(q, kc, vc, ks, vs[:, :1], t, lens),
                lambda: call(q, kc, vc, ks, vs, t[:1], lens), lambda: call(q, kc, vc, ks, vs, t, lens.long()),
                lambda: call(q[..., :32], kc, vc, ks, vs, t, lens), lambda: call(q[:, :3], kc, vc, ks, vs, t, lens),
                lambda: call(q.expand(2, 4, 17, 64), kc, vc, ks, vs, t, lens),
                lambda: call(q, kc, vc, ks, vs, t, lens, first=-1), lambda: call(q, kc, vc, ks, vs, t, lens, scale=0.0),
                lambda: call(q, kc, vc, ks, vs, t, lens, sinks=torch.zeros(3, device="cuda")),
                lambda: call(q, kc, vc.cpu(), ks, vs, t, lens)):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            bad()
