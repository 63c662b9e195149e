"""Appending turned rows to paged caches in bf16 and in 8 bits, and reading the latter (GPU)."""
import pytest
import torch

import q8_ref as ref
import serving_ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def fa():
    from attention_forward_blackwell_gb300 import binding
    binding.lib()
    return binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(gen, *shape, spread=0.0):
    x = torch.randn(*shape, generator=gen)
    return (x * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=gen))).bfloat16()


def tables(gen, lens, more, page):
    """Pages in a random order for lens[b] + more keys; the number of pages, one of them spare."""
    need = [-(-(n + more) // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen).tolist()
    width = max(1, max(need, default=1)) + 1
    out = []
    for n in need:
        out.append(order[:n] + [-1] * (width - n))
        order = order[n:]
    return out, sum(need) + 1


def same_cache(got, want, what):
    """got: (k, v, k_scale, v_scale) on the device, want: ref.Cache8."""
    for i, name in enumerate(("k", "v")):
        assert torch.equal(got[2 + i].cpu().double(), want.scales[i]), f"{what}: {name} scales"
        off = (got[i].cpu().double() - want.codes[i]).abs()
        assert not off.isnan().any(), f"{what}: {name} codes"
        assert torch.all(off <= want.slack[i]), f"{what}: {name} codes off by {off.max().item()}"
        # a code may be the next one only where its element lies next to the middle
        assert (off > 0).double().mean().item() < 2e-3 or off.numel() < 20000, f"{what}: {name}"


APPENDS = [  # lens, n, counts, hkv, d, page, block, rot, interleaved, hq
    ([5], 1, None, 1, 64, 16, 16, 64, False, 1),
    ([0, 1, 15, 16, 17, 300], 1, None, 2, 128, 64, 16, 128, False, 8),
    ([0, 63, 64, 7], 70, [70, 1, 0, 33], 3, 128, 64, 64, 96, True, 0),
    ([10, 100, 3], 200, [200, 120, 5], 2, 256, 100, 25, 64, False, 4),
    ([31, 0], 40, None, 2, 64, 48, 12, 32, True, 2),
    ([3, 500], 300, [300, 299], 1, 128, 256, 256, 0, False, 2),
    ([2, 9], 9, None, 2, 80, 16, 4, 80, False, 2),
    ([129, 77], 600, [600, 513], 2, 256, 256, 128, 256, False, 0),
    ([4, 4], 5, [-3, 9], 1, 64, 1, 1, 16, False, 1),
    # many units: of 128 threads with two tasks kept or more, of a warp
    ([7 * i % 50 for i in range(30)], 40, [41 - i for i in range(30)], 8, 128, 64, 32, 128, False, 0),
    (list(range(26)), 50, None, 8, 64, 64, 64, 32, True, 1), ([13 * i for i in range(40)], 2, None, 16, 96, 32, 4, 48, False, 3),
    ([3, 0], 30, None, 1, 1024, 16, 16, 512, False, 2)]


@pytest.mark.parametrize("lens,n,counts,hkv,d,page,block,rot,interleaved,hq", APPENDS)
def test_append(fa, lens, n, counts, hkv, d, page, block, rot, interleaved, hq):
    g = torch.Generator().manual_seed(n + d)
    B = len(lens)
    table, pages = tables(g, lens, n, page)
    table_d, lens_d = i32(table), i32(lens)
    real = [max(0, min(c, n)) for c in counts] if counts else [n] * B
    k_new, v_new = (rows(g, B, n, hkv, d, spread=1.0).cuda().transpose(1, 2) for _ in range(2))
    inv, factor = fa.rope_inv_freq(rot, method="yarn", stretch=4.0, original=128) if rot else ([], 1.0)
    turn = (inv, factor, interleaved) if rot else None
    more = dict(n_new=i32(counts) if counts else None, interleaved=interleaved, factor=factor)
    freqs = fa.rope_freqs(inv) if rot else None
    if hq:
        more["q"] = rows(g, B, n, hq, d).cuda().transpose(1, 2)
        more["q_out"] = torch.full((B, hq, n, d), 7.0, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor(lens)[:, None] + torch.arange(n)

    def check_q(got):
        if not hq:
            assert got is None
            return
        q = more["q"].cpu()
        want = ref.turn64(q, at[:, None], inv, factor, interleaved) if rot else q.double()
        bound = ref.turn_bound(q, want, at[:, None], rot, factor, interleaved)
        for b in range(B):
            off = (got[b].cpu().double() - want[b]).abs()
            assert torch.all(off[:, :real[b]] <= bound[b][:, :real[b]])
            assert torch.all(got[b][:, real[b]:] == 7.0)   # rows behind the last stay

    # 8 bits
    kc, ks = ref.codes8(g, pages, hkv, page, block, d)
    vc, vs = ref.codes8(g, pages, hkv, page, block, d)
    want = ref.Cache8(kc, vc, ks, vs)
    want.append(table, lens, k_new, v_new, real, turn)
    check_q(fa.cache_append_q8(kc, vc, ks, vs, table_d, lens_d, k_new, v_new, freqs, **more))
    same_cache((kc, vc, ks, vs), want, "append")
    before = [t.clone() for t in (kc, vc, ks, vs)]
    fa.cache_append_q8(kc, vc, ks, vs, table_d, lens_d, k_new, v_new, freqs, **more)   # once more: no change
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, (kc, vc, ks, vs)))
    # bf16
    if not rot:
        return
    k16, v16 = (rows(g, pages, hkv, page, d).cuda() for _ in range(2))
    want_k, want_v = k16.cpu().double(), v16.cpu()
    bound = torch.zeros_like(want_k)
    turned = ref.turn64(k_new.cpu(), at[:, None], *turn)
    serving_ref.append_rows(want_k, table, lens, turned, real)
    serving_ref.append_rows(want_v, table, lens, v_new.cpu(), real)
    serving_ref.append_rows(bound, table, lens, ref.turn_bound(k_new.cpu(), turned, at[:, None], rot, factor,
                                                              interleaved), real)
    if hq:
        more["q_out"].fill_(7.0)
    check_q(fa.cache_append_rope(k16, v16, table_d, lens_d, k_new, v_new, freqs, **more))
    assert torch.equal(v16.cpu(), want_v)
    assert torch.all((k16.cpu().double() - want_k).abs() <= bound)


@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (32, 32)])
def test_token_by_token_is_as_at_once(fa, page, block):
    """Scales that grow with their block: rows appended one by one leave the codes of rows appended
    together, but for those that the larger scale takes below its smallest normal code."""
    g = torch.Generator().manual_seed(page)
    n, hkv, d = 70, 2, 128
    table, pages = tables(g, [0], n, page)
    k_new, v_new = (rows(g, 1, hkv, n, d, spread=1.5).cuda() for _ in range(2))
    inv, _ = fa.rope_inv_freq(d)
    freqs = fa.rope_freqs(inv)
    state = []
    for steps in ([n], [1] * n, [3, 1, 40, 1, 1, 24]):
        kc, vc = (torch.zeros(pages, hkv, page, d, device="cuda").to(F8) for _ in range(2))
        ks, vs = (torch.zeros(pages, hkv, page // block, device="cuda") for _ in range(2))
        want, at = ref.Cache8(kc, vc, ks, vs), 0
        for c in steps:
            part = (k_new[:, :, at:at + c], v_new[:, :, at:at + c])
            fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32([at]), *part, freqs)
            want.append(table, [at], *part, [c], (inv, 1.0, False))
            at += c
        same_cache((kc, vc, ks, vs), want, f"steps of {steps[0]}")
        state.append([(t.float().unflatten(2, (-1, block)) * s[..., None, None]) for t, s in ((kc, ks), (vc, vs))])
        state[-1] += [ks, vs]
    for other in state[1:]:
        assert torch.equal(other[2], state[0][2]) and torch.equal(other[3], state[0][3])
        for i in range(2):
            low = state[0][2 + i][..., None, None] * 2.0 ** -6
            differ = (other[i] != state[0][i]) & (torch.maximum(other[i].abs(), state[0][i].abs()) > low)
            assert not differ.any()


def test_copies(fa):
    """Pages that reserve replaced come along with their scales, the open block among them."""
    g = torch.Generator().manual_seed(4)
    page, block, hkv, d = 32, 8, 2, 64
    lens, counts = [20, 16, 13, 31, 8], [1, 3, 0, 5, 2]
    B, n = len(lens), 5
    table = [[3, -1], [4, -1], [5, -1], [6, 7], [8, -1]]
    copies = [[0, 3, 20], [1, 4, 16], [2, 5, 13], [0, 6, 31], [-1, -1, 0]]
    inv, _ = fa.rope_inv_freq(32)
    kc, ks = ref.codes8(g, 10, hkv, page, block, d)
    vc, vs = ref.codes8(g, 10, hkv, page, block, d)
    k_new, v_new = (rows(g, B, hkv, n, d, spread=2.0).cuda() for _ in range(2))
    want = ref.Cache8(kc, vc, ks, vs)
    want.copy(copies)
    want.append(table, lens, k_new, v_new, counts, (inv, 1.0, True))
    fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32(lens), k_new, v_new, fa.rope_freqs(inv), n_new=i32(counts),
                       copies=i32(copies), interleaved=True)
    same_cache((kc, vc, ks, vs), want, "copies")
    # copies alone: no rows, and pages that are no sequence's open one
    none = torch.zeros(B, hkv, 0, d, dtype=torch.bfloat16, device="cuda")
    want.copy([[3, 9, 11]])
    fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32(lens), none, none, copies=i32([[3, 9, 11]] + [[-1, -1, 0]] * 4))
    for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
        assert torch.equal(c.cpu().double()[9, :, :11], want.codes[i][9, :, :11]) or i == 0
        assert torch.equal(s.cpu().double()[9, :, :2], want.scales[i][9, :, :2])
    # bf16 rows likewise
    k16, v16 = (rows(g, 10, hkv, page, d).cuda() for _ in range(2))
    wk, wv = k16.cpu().double(), v16.cpu()
    at = torch.tensor(lens)[:, None] + torch.arange(n)
    turned = ref.turn64(k_new.cpu(), at[:, None], inv, 1.0, True)
    bound = torch.zeros_like(wk)
    serving_ref.append_rows(wk, table, lens, turned, counts, copies)
    serving_ref.append_rows(wv, table, lens, v_new.cpu(), counts, copies)
    serving_ref.append_rows(bound, table, lens, ref.turn_bound(k_new.cpu(), turned, at[:, None], 32, 1.0, True), counts)
    fa.cache_append_rope(k16, v16, i32(table), i32(lens), k_new, v_new, fa.rope_freqs(inv), n_new=i32(counts),
                         copies=i32(copies), interleaved=True)
    assert torch.equal(v16.cpu(), wv) and torch.all((k16.cpu().double() - wk).abs() <= bound)


def test_positions_of_a_tree(fa):
    """Rows that stand elsewhere than their keys: a tree's nodes by their depth."""
    g = torch.Generator().manual_seed(8)
    lens, n, hkv, hq, d, page = [7, 30], 6, 2, 4, 128, 16
    table, pages = tables(g, lens, n, page)
    at = torch.tensor([[7, 8, 8, 9, 9, 10], [30, 31, 31, 31, 32, 33]])
    inv, _ = fa.rope_inv_freq(d)
    k_new, v_new = (rows(g, 2, hkv, n, d).cuda() for _ in range(2))
    q = rows(g, 2, hq, n, d).cuda()
    kc, ks = ref.codes8(g, pages, hkv, page, 16, d)
    vc, vs = ref.codes8(g, pages, hkv, page, 16, d)
    want = ref.Cache8(kc, vc, ks, vs)
    want.append(table, lens, k_new, v_new, [n, n], (inv, 1.0, False), at)
    qo = fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32(lens), k_new, v_new, fa.rope_freqs(inv),
                            positions=at.to(torch.int32).cuda(), q=q)
    same_cache((kc, vc, ks, vs), want, "positions")
    wq = ref.turn64(q.cpu(), at[:, None], inv)
    assert torch.all((qo.cpu().double() - wq).abs() <= ref.turn_bound(q.cpu(), wq, at[:, None], d, 1.0, False))
    k16, v16 = (torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q2 = fa.cache_append_rope(k16, v16, i32(table), i32(lens), k_new, v_new, fa.rope_freqs(inv),
                              positions=at.to(torch.int32).cuda(), q=q)
    assert torch.equal(q2, qo)


def test_pages_that_are_none(fa):
    """Keys without a page are skipped, past the table too; nothing else changes."""
    g = torch.Generator().manual_seed(5)
    kc, ks = ref.codes8(g, 4, 1, 16, 16, 64)
    vc, vs = ref.codes8(g, 4, 1, 16, 16, 64)
    want = ref.Cache8(kc, vc, ks, vs)
    table, lens = [[0, 99, 1], [-7, 2, 4], [3, -1, -1]], [10, 12, 2 ** 31 - 3]
    k_new, v_new = (rows(g, 3, 1, 40, 64).cuda() for _ in range(2))
    want.append(table[:2] + [[]], lens, k_new, v_new, [40, 40, 0])
    fa.cache_append_q8(kc, vc, ks, vs, i32(table), i32(lens), k_new, v_new)
    same_cache((kc, vc, ks, vs), want, "no page")


EXTREMES = [0.0, 2.0 ** -100, 2.0 ** -60, 2.0 ** -40, 447.9, 448.0, 449.0, 2.0 ** 40, 2.0 ** 62, 2.0 ** 63, 3e38]


@pytest.mark.parametrize("size", EXTREMES)
def test_extreme_rows(fa, size):
    x = torch.zeros(1, 1, 3, 64)
    x[..., 0, 5], x[..., 1, 9], x[..., 2, 40] = size, -size / 3, size * 2.0 ** -9
    x = x.bfloat16().cuda()
    kc, vc = (torch.zeros(1, 1, 16, 64, device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.ones(1, 1, 1, device="cuda") for _ in range(2))
    want = ref.Cache8(kc, vc, ks, vs)
    want.append([[0]], [0], x, x, [3])
    fa.cache_append_q8(kc, vc, ks, vs, i32([[0]]), i32([0]), x, x)
    same_cache((kc, vc, ks, vs), want, f"size {size}")


def test_scales_of_other_kinds(fa):
    """A scale that is no power of two stays while it is the larger; codes go by it."""
    g = torch.Generator().manual_seed(6)
    kc, _ = ref.codes8(g, 1, 1, 16, 16, 64)
    vc, _ = ref.codes8(g, 1, 1, 16, 16, 64)
    for first, size in ((0.37, 1.0), (0.003, 900.0)):
        ks, vs = (torch.full((1, 1, 1), first, device="cuda") for _ in range(2))
        k, v = kc.clone(), vc.clone()
        x = (rows(g, 1, 1, 2, 64) * size).bfloat16().cuda()
        want = ref.Cache8(k, v, ks, vs)
        want.append([[0]], [5], x, x, [2])
        fa.cache_append_q8(k, v, ks, vs, i32([[0]]), i32([5]), x, x)
        for i, (c, s) in enumerate(((k, ks), (v, vs))):
            assert torch.equal(s.cpu().double(), want.scales[i])
            off = (c.cpu().double() - want.codes[i]).abs()   # (products with a reciprocal: next to a middle)
            assert torch.all(off <= 2 * ref.half_step(want.codes[i])) and (off > 0).sum() <= 2


@pytest.mark.parametrize("lens,hkv,d,page,block", [([1], 1, 64, 16, 16), ([0, 5, 300, 0, 64], 3, 128, 64, 16),
                                                   ([33, 1000], 2, 256, 100, 50), ([700, 17], 8, 80, 48, 12),
                                                   # many tokens to a CTA, one, heads past a CTA's threads
                                                   ([2500, 0, 37], 8, 128, 64, 64), ([6000, 3999], 1, 64, 64, 64),
                                                   ([40, 3], 1, 2048, 16, 16), ([9, 70], 40, 256, 32, 8)])
def test_read(fa, lens, hkv, d, page, block):
    g = torch.Generator().manual_seed(d)
    table, pages = tables(g, lens, 0, page)
    kc, ks = ref.codes8(g, pages, hkv, page, block, d)
    vc, vs = ref.codes8(g, pages, hkv, page, block, d)
    cache = ref.Cache8(kc, vc, ks, vs)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    k, v = fa.cache_read_q8(kc, vc, ks, vs, i32(table), i32(cu), cu[-1], max(lens))
    for i, got in enumerate((k, v)):
        x = cache.values(i)
        want = torch.cat([torch.stack([x[table[b][j // page], :, j % page] for j in range(n)])
                          for b, n in enumerate(lens) if n])
        assert torch.equal(got.cpu().double(), want)   # (three bits of fraction: bf16 holds them)


def test_read_bounds(fa):
    """Keys without a page read as zeros, lengths past max_seqlen and offsets past total are cut, rows
    behind the last stay."""
    g = torch.Generator().manual_seed(2)
    kc, ks = ref.codes8(g, 3, 2, 16, 16, 64)
    out = [torch.full((60, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = fa.cache_read_q8(kc, kc, ks, ks, i32([[0, 7], [1, 2]]), i32([0, 20, 55]), 60, 32, k_out=out[0], v_out=out[1])
    assert k is out[0] and torch.equal(k, v)
    assert torch.all(k[16:20] == 0) and torch.all(k[20 + 32:] == 5.0)
    x = ref.Cache8(kc, kc, ks, ks).values(0)
    for at, page in ((0, 0), (20, 1), (36, 2)):
        assert torch.equal(k[at:at + 16].cpu().double(), x[page].transpose(0, 1))
    k, _ = fa.cache_read_q8(kc, kc, ks, ks, i32([[0, 7], [1, 2]]), i32([0, 20, 999]), 30, 99)
    assert k.shape == (30, 2, 64)
    k, _ = fa.cache_read_q8(kc, kc, ks, ks, i32([[0, 7]]), i32([0, 0]), 0, 0)
    assert k.shape == (0, 2, 64)


def test_caches_without_pages(fa):
    """Every key reads as zeros, appended rows go nowhere; a table of no entries likewise."""
    g = torch.Generator().manual_seed(3)
    x = rows(g, 2, 2, 5, 64).cuda()
    for pages, width in ((0, 3), (3, 0), (0, 0)):
        kc, vc = (torch.zeros(pages, 2, 16, 64, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
        ks, vs = (torch.ones(pages, 2, 2, device="cuda") for _ in range(2))
        table, out = i32([[0] * width] * 2).reshape(2, width), [torch.full((70, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        assert fa.cache_append_q8(kc, vc, ks, vs, table, i32([0, 3]), x, x) is None
        k, v = fa.cache_read_q8(kc, vc, ks, vs, table, i32([0, 33, 60]), 70, 33, k_out=out[0], v_out=out[1])
        assert not k[:60].any() and not v[:60].any() and torch.all(k[60:] == 5.0) and torch.all(v[60:] == 5.0)
        assert not kc.view(torch.uint8).any() and torch.all(ks == 1.0)


def test_refusals(fa):
    g = torch.Generator().manual_seed(1)
    kc, ks = ref.codes8(g, 3, 2, 16, 8, 64)
    t, lens = i32([[0, 1]]), i32([3])
    x = rows(g, 1, 2, 4, 64).cuda()
    freqs = fa.rope_freqs(fa.rope_inv_freq(32)[0])
    k16 = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: fa.cache_append_q8(k16, k16, ks, ks, t, lens, x, x),
                lambda: fa.cache_append_q8(kc, kc, ks.double(), ks, t, lens, x, x),
                lambda: fa.cache_append_q8(kc, kc, ks[..., :1].expand(3, 2, 3).contiguous(), ks, t, lens, x, x),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens.long(), x, x),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x[:, :1]),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x, freqs, q=x[0]),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x, freqs, q_out=x),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x, freqs, q=x.clone(), q_out=x),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x, freqs, positions=i32([1, 2])),
                lambda: fa.cache_append_q8(kc, kc, ks, ks, t, lens, x, x, freqs, factor=float("nan")),
                lambda: fa.cache_append_rope(kc, kc, t, lens, x, x, freqs),
                lambda: fa.cache_append_rope(k16, k16, t, lens, x, x, None),
                lambda: fa.cache_append_rope(k16, k16, t, lens, x, x, fa.rope_freqs(fa.rope_inv_freq(128)[0])),
                lambda: fa.cache_read_q8(kc, kc, ks, ks, t, i32([0, 4, 5]), 5, 5),
                lambda: fa.cache_read_q8(kc, kc, ks, ks, t, i32([0, 4]), -1, 5),
                lambda: fa.cache_read_q8(kc, kc, ks, ks, t, i32([0, 4]), 4, 0)):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            bad()
