"""A sliding window whose first keys stay visible, through every entry point
that takes a window, against its definition in 64 bits."""
import math

import pytest
import torch

import serving_ref as ref
from gpu_parity import check_device_error, free_cuda, to_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def tensors(B, Hq, Hkv, Sq, Sk, d, seed, sinks=False):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, Sq, d, generator=g).bfloat16()
    k = torch.randn(B, Hkv, Sk, d, generator=g).bfloat16()
    v = torch.randn(B, Hkv, Sk, d, generator=g).bfloat16()
    return q, k, v, torch.randn(Hq, generator=g) if sinks else None


def poison(k, v, lens):
    for b, L in enumerate(lens):
        k[b, :, max(L, 0):] = math.nan
        v[b, :, max(L, 0):] = math.nan


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


PREFILL = [
    # B, Hq, Hkv, Sq, lens, d, window, first, causal, sinks
    (1, 2, 1, 700, [700], 128, 100, 4, True, False),
    (2, 2, 2, 600, [600, 450], 64, 64, 1, True, False),
    (1, 2, 1, 900, [900], 128, 1, 130, True, True),
    (1, 2, 1, 513, [513], 96, 200, 128, True, False),
    (2, 2, 1, 300, [1200, 999], 128, 150, 257, True, False),
    (1, 2, 2, 260, [900], 128, 100, 5, False, False),
    (1, 2, 1, 700, [700], 256, 90, 140, True, True),
    (2, 4, 2, 333, [800, 340], 256, 130, 3, True, False),
    (1, 1, 1, 400, [700], 512, 100, 10, True, False),
    (1, 2, 1, 130, [130], 128, 40, 1000, True, False),
    (2, 2, 1, 50, [0, 20], 128, 16, 2, True, True),
    (1, 1, 1, 1, [500], 64, 30, 7, True, False),
    (1, 2, 1, 256, [640], 256, 128, 128, False, False),
]


@pytest.mark.parametrize("case", PREFILL, ids=[f"{i}-q{c[3]}d{c[5]}w{c[6]}f{c[7]}"
                                               for i, c in enumerate(PREFILL)])
def test_prefill_first(case):
    from attention_forward_blackwell_gb300 import binding
    B, Hq, Hkv, Sq, lens, d, window, first, causal, sinks = case
    Sk = max(lens) + 3
    q, k, v, sk = tensors(B, Hq, Hkv, Sq, Sk, d, Sq + d, sinks)
    want = ref.attention64(q, k, v, ref.window_seen(Sq, lens, Sk, window, first, causal),
                           1 / math.sqrt(d), sk)
    poison(k, v, lens)
    o, lse = binding.prefill(q.cuda(), k.cuda(), v.cuda(), causal=causal, seqlens_k=i32(lens),
                             window=window, first=first, sinks=None if sk is None else sk.cuda())
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, lse, want, f"prefill first {case}")


PACKED = [
    # Hq, Hkv, [(q, k)], d, page, window, first, sinks
    (2, 1, [(300, 300), (1, 900), (0, 5), (129, 400)], 128, 0, 100, 4, False),
    (2, 1, [(300, 700), (200, 200)], 128, 128, 70, 130, True),
    (4, 2, [(257, 700), (40, 1000), (5, 5)], 256, 128, 64, 200, True),
    (2, 2, [(100, 600), (350, 350)], 64, 256, 30, 1, False),
    (2, 1, [(150, 500)], 96, 0, 60, 60, False),
    (1, 1, [(140, 600), (3, 300)], 512, 128, 50, 9, False),
]


@pytest.mark.parametrize("case", PACKED, ids=[f"{i}-d{c[3]}p{c[4]}w{c[5]}f{c[6]}"
                                              for i, c in enumerate(PACKED)])
def test_packed_first(case):
    from attention_forward_blackwell_gb300 import binding
    Hq, Hkv, seqs, d, page, window, first, sinks = case
    nq, nk = [s[0] for s in seqs], [s[1] for s in seqs]
    B, Sk = len(seqs), max(nk)
    g = torch.Generator().manual_seed(sum(nk))
    q = torch.randn(sum(nq), Hq, d, generator=g).bfloat16()
    k, v = (torch.randn(B, Hkv, Sk, d, generator=g).bfloat16() for _ in range(2))
    sk = torch.randn(Hq, generator=g) if sinks else None
    cu = torch.tensor([0] + nq).cumsum(0)
    more = dict(causal=True, window=window, first=first, sinks=None if sk is None else sk.cuda())
    if page:
        kc, vc, table, _ = to_pages(k.cuda(), v.cuda(), nk, page, seed=page)
        o, lse = binding.prefill_varlen_paged(q.cuda(), kc, vc, i32(cu.tolist()), max(nq), table,
                                              i32(nk), **more)
    else:
        kp, vp = (torch.cat([x[b, :, :n].transpose(0, 1) for b, n in enumerate(nk)]).contiguous()
                  for x in (k, v))
        ck = torch.tensor([0] + nk).cumsum(0)
        o, lse = binding.prefill_varlen(q.cuda(), kp.cuda(), vp.cuda(), i32(cu.tolist()),
                                        i32(ck.tolist()), max(nq), max(nk), **more)
    torch.cuda.synchronize()
    check_device_error()
    for b, (n, m) in enumerate(seqs):
        if n == 0:
            continue
        s = slice(int(cu[b]), int(cu[b + 1]))
        want = ref.attention64(q[s].transpose(0, 1)[None], k[b:b + 1, :, :m], v[b:b + 1, :, :m],
                               ref.window_seen(n, [m], m, window, first, True), 1 / math.sqrt(d), sk)
        ref.check(o[s].transpose(0, 1)[None], lse[None, :, s], want, f"packed first {b}")


DECODE = [
    # B, Hq, Hkv, Sq, lens, d, page, window, first, causal, sinks
    (3, 8, 2, 1, [700, 64, 5], 128, 0, 100, 4, True, False),
    (3, 8, 2, 1, [3000, 1, 0], 128, 16, 64, 64, True, True),
    (2, 4, 4, 1, [900, 513], 64, 0, 17, 65, False, False),
    (2, 16, 2, 5, [800, 333], 128, 64, 50, 130, True, False),
    (2, 10, 2, 4, [1000, 2], 256, 100, 200, 3, True, True),
    (1, 4, 1, 16, [400], 128, 0, 1, 1, True, False),
    (1, 2, 1, 1, [4096], 128, 128, 1000, 300, True, False),
    (2, 2, 1, 2, [130, 129], 64, 7, 10, 500, True, False),
    (1, 8, 1, 1, [191], 128, 0, 64, 64, True, False),
    (1, 8, 1, 1, [193], 128, 0, 64, 64, True, False),
]


@pytest.mark.parametrize("case", DECODE, ids=[f"{i}-q{c[3]}d{c[5]}p{c[6]}w{c[7]}f{c[8]}"
                                              for i, c in enumerate(DECODE)])
def test_decode_first(case):
    from attention_forward_blackwell_gb300 import binding
    B, Hq, Hkv, Sq, lens, d, page, window, first, causal, sinks = case
    Sk = max(lens) + 2
    q, k, v, sk = tensors(B, Hq, Hkv, Sq, Sk, d, Sk + d + window, sinks)
    seen = ref.window_seen(Sq, lens, Sk, window, first, causal)
    want = ref.attention64(q, k, v, seen, 1 / math.sqrt(d), sk)
    poison(k, v, lens)
    for b in range(B):       # decode reads no key that no row sees
        k[b, :, ~seen[b].any(0)] = math.nan
        v[b, :, ~seen[b].any(0)] = math.nan
    more = dict(causal=causal, window=window, first=first,
                sinks=None if sk is None else sk.cuda())
    kg, vg = k.cuda(), v.cuda()
    if page:
        kc, vc, table, _ = to_pages(kg, vg, lens, page, seed=page)
        o, lse = binding.decode_paged(q.cuda(), kc, vc, table, i32(lens), **more)
    else:
        o, lse = binding.decode(q.cuda(), kg, vg, seqlens_k=i32(lens), **more)
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, lse, want, f"decode first {case}")


def test_no_first_is_the_window():
    """first = 0 keeps the window's results bit for bit, and no window ignores first."""
    from attention_forward_blackwell_gb300 import binding
    q, k, v, sk = (x.cuda() for x in tensors(2, 4, 2, 200, 500, 128, 1, True))
    from attention_forward_blackwell_gb300.binding import lib, _ptr, _stream_ptr
    for window, first in ((64, 0), (0, 9)):
        o, lse = binding.prefill(q, k, v, causal=True, window=window, sinks=sk)
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        st = lib().fa_fwd_prefill_first(_ptr(q), _ptr(k), _ptr(v), _ptr(o2), _ptr(lse2), 2, 4, 2,
                                        200, 500, None, 128, 128 ** -0.5, 1, window, first,
                                        _ptr(sk), _stream_ptr())
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    L = i32([500, 77])
    for window in (0, 100):   # the paged window of decode is the contiguous one
        kc, vc, table, _ = to_pages(k, v, [500, 77], 50, seed=1)
        a = binding.decode(q[:, :, :3].contiguous(), k, v, causal=True, seqlens_k=L, window=window,
                           sinks=sk)
        b = binding.decode_paged(q[:, :, :3].contiguous(), kc, vc, table, L, causal=True,
                                 window=window, sinks=sk)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_long_offsets():
    """Pages past 2^31 elements of a cache."""
    from attention_forward_blackwell_gb300 import binding
    P, Hkv, d = 128, 8, 128
    pages = (2 ** 31) // (P * Hkv * d) + 40
    kc = torch.zeros(pages, Hkv, P, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    lens, window, first = [700], 200, 20
    q, k, v, _ = tensors(1, 8, 8, 6, 768, d, 4)
    table = torch.arange(6).flip(0)[None] * 5 + pages - 30
    for j in range(6):
        kc[int(table[0, j])] = k[0, :, j * P:(j + 1) * P].cuda()
        vc[int(table[0, j])] = v[0, :, j * P:(j + 1) * P].cuda()
    t = table.to(torch.int32).cuda()
    want = ref.attention64(q, k, v, ref.window_seen(6, lens, 768, window, first, True), d ** -0.5)
    o, lse = binding.decode_paged(q.cuda(), kc, vc, t, i32(lens), causal=True, window=window,
                                  first=first)
    ref.check(o, lse, want, "far pages, decode")
    o, lse = binding.prefill_varlen_paged(q[0].transpose(0, 1).contiguous().cuda(), kc, vc,
                                          i32([0, 6]), 6, t, i32(lens), causal=True, window=window,
                                          first=first)
    ref.check(o.transpose(0, 1)[None], lse[None], want, "far pages, prefill")
    mask = ref.pack_bits(torch.ones(6, 6).tril().bool()).cuda()
    want = ref.attention64(q, k, v, ref.window_seen(6, lens, 768, 0, 0, True), d ** -0.5)
    o, lse = binding.decode_tree_paged(q.cuda(), kc, vc, t, i32(lens), mask)
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, lse, want, "far pages, tree")
    del kc, vc
    free_cuda()
