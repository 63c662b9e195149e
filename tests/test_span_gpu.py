"""Trees and windows at the sizes where the work of the tensor-core kernel is cut
up differently: many sequences, many tiles, small pages, long lines of blocks."""
import math

import pytest
import torch

import serving_ref as ref
from gpu_parity import check_device_error, free_cuda, to_pages
from test_first_gpu import i32, poison, tensors
from test_tree_gpu import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def spread(n, lo, hi):
    """n lengths over lo .. hi in no order."""
    return [lo + (i * 7919) % n * (hi - lo) // max(1, n - 1) for i in range(n)]


TREES = [
    # Hq, Hkv, T, contexts, d, page, kind, ragged
    (32, 1, 12, [300, 40], 128, 0, "tree", False),            # 3 tiles
    (32, 1, 20, [700, 5, 260], 64, 64, "any", True),          # 5 tiles
    (16, 1, 65, [100, 900], 128, 32, "tree", False),          # 9 tiles, two groups
    (2, 1, 1024, [17], 64, 0, "chain", False),                # 16 tiles, the most nodes
    (8, 2, 16, spread(70, 0, 500), 128, 4, "tree", True),     # boxes of 4 rows
    (8, 1, 16, spread(9, 50, 700), 128, 12, "any", True),
    (8, 1, 32, spread(9, 50, 700), 64, 100, "tree", False),
    (8, 1, 24, spread(9, 50, 700), 256, 20, "tree", True),
    (4, 1, 8, spread(600, 0, 90), 64, 16, "tree", True),      # more sequences than threads
    (8, 8, 2, [66000], 256, 128, "tree", False),              # few rows, many bytes
    (130, 1, 3, [200, 90], 64, 0, "tree", False),             # a group larger than a tile
    (127, 1, 3, [200, 90], 128, 16, "any", True),
]


@pytest.mark.parametrize("case", TREES, ids=[f"{i}-b{len(c[3])}g{c[0] // c[1]}t{c[2]}d{c[4]}p{c[5]}"
                                             for i, c in enumerate(TREES)])
def test_trees(case):
    Hq, Hkv, T, ctx, d, page, kind, ragged = case
    run(len(ctx), Hq, Hkv, T, ctx, d, page, kind, ragged, seed=T + d + page)


DECODE = [
    # Hq, Hkv, Sq, lens, d, page, window, first, causal, sinks
    (16, 1, 5, [900, 333, 4], 128, 0, 50, 130, True, False),      # many rows
    (16, 1, 4, [900, 333, 1000], 128, 64, 300, 3, True, True),
    (32, 2, 8, [1500, 7], 64, 8, 200, 70, True, False),
    (8, 1, 4, [1000, 600, 0, 31], 256, 16, 100, 5, True, False),
    (16, 1, 9, [700, 260], 128, 4, 64, 64, True, False),          # boxes of 4 rows
    (16, 2, 8, [700, 260], 64, 100, 120, 9, False, True),
    (8, 8, 1, [9000, 10, 4500, 0], 256, 32, 8000, 100, True, False),   # many bytes
    (8, 4, 1, spread(40, 0, 900), 128, 16, 600, 4, True, False),
    (8, 4, 2, spread(520, 0, 700), 64, 0, 600, 4, True, False),
    (128, 1, 2, [300, 77], 64, 0, 90, 33, True, False),           # one position a tile
    (12, 2, 8, [700, 5, 410], 256, 32, 120, 10, True, True),      # six heads, 21 positions
    (33, 3, 16, [1200, 333], 128, 0, 333, 1, True, False),
    (7, 1, 16, [2000, 1, 0], 64, 48, 64, 200, False, False),
]


@pytest.mark.parametrize("case", DECODE, ids=[f"{i}-b{len(c[3])}q{c[2]}d{c[4]}p{c[5]}w{c[6]}f{c[7]}"
                                              for i, c in enumerate(DECODE)])
def test_window_decode(case):
    from attention_forward_blackwell_gb300 import binding
    Hq, Hkv, Sq, lens, d, page, window, first, causal, sinks = case
    B, Sk = len(lens), max(lens) + 2
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
    ref.check(o, lse, want, f"decode {case[:3]} {case[4:]}")


PREFILL = [
    # B, Hq, Hkv, Sq, Sk, d, window, first, causal
    (1, 4, 2, 900, 900, 128, 100, 4, True),        # two heads a tile
    (2, 6, 2, 300, 700, 64, 130, 70, True),        # three heads a tile: 126 rows
    (1, 8, 1, 400, 400, 256, 33, 1, True),
    (1, 16, 1, 200, 999, 128, 255, 256, True),
    (1, 4, 1, 150, 600, 128, 64, 16, False),
    (40, 2, 1, 30, 60, 64, 10, 3, True),           # many sequences
    (1, 2, 1, 4000, 4000, 64, 128, 64, True),      # a long line of blocks
    (70, 8, 2, 120, 1300, 128, 50, 20, True),      # many rows
    (12, 8, 2, 700, 700, 64, 100, 4, True),
    (41, 16, 1, 110, 300, 256, 33, 3, True),
    (66, 16, 1, 70, 300, 128, 130, 40, False),
]


@pytest.mark.parametrize("case", PREFILL, ids=[f"{i}-b{c[0]}g{c[1] // c[2]}q{c[3]}d{c[5]}w{c[6]}f{c[7]}"
                                               for i, c in enumerate(PREFILL)])
@pytest.mark.parametrize("more", [0, 600], ids=["short", "long"])   # each side of the kernels' border
def test_window_prefill(case, more):
    from attention_forward_blackwell_gb300 import binding
    B, Hq, Hkv, Sq, Sk, d, window, first, causal = case
    window += more
    lens = [max(0, Sk - 13 * b) for b in range(B)]
    q, k, v, _ = tensors(B, Hq, Hkv, Sq, Sk, d, Sk + d + window)
    want = ref.attention64(q, k, v, ref.window_seen(Sq, lens, Sk, window, first, causal),
                           1 / math.sqrt(d))
    poison(k, v, lens)
    o, lse = binding.prefill(q.cuda(), k.cuda(), v.cuda(), causal=causal, seqlens_k=i32(lens),
                             window=window, first=first)
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, lse, want, f"prefill {case} {more}")


PACKED = [
    # Hq, Hkv, [(q, k)], d, page, window, first
    (8, 2, [(700, 1000), (33, 2000), (0, 9), (513, 513)], 128, 0, 700, 40),   # pairs of CTAs and not
    (8, 2, [(700, 1000), (33, 2000), (0, 9), (513, 513)], 128, 128, 60, 40),
    (8, 1, [(260, 1000), (90, 300)], 256, 256, 90, 200),
    (4, 1, [(1, 50 + i) for i in range(60)] + [(90, 90)], 128, 128, 40, 6),
    (2, 2, [(3, 3 + i) for i in range(530)], 64, 0, 40, 6),
    (12, 4, [(300, 300), (41, 600)], 64, 128, 1000, 2000),
    (32, 4, [(1100, 1400), (0, 5), (33, 900)], 128, 128, 300, 20),             # many rows
    (32, 4, [(700, 700), (5, 900), (401, 555)], 128, 0, 30, 70),
    (16, 16, [(513, 700), (300, 300), (1, 40), (900, 901), (500, 1300)], 64, 0, 200, 9),
    (32, 8, [(300, 600), (290, 1000), (310, 310), (250, 400)], 256, 256, 90, 200),
    (32, 16, [(300, 600), (290, 1000), (310, 310), (250, 400)], 256, 0, 500, 130),
    (24, 8, [(700, 900), (690, 700)], 64, 0, 150, 20),        # three heads a tile, 42 positions
    (21, 7, [(800, 800), (1, 300), (777, 1000)], 256, 128, 90, 150),
    (40, 8, [(500, 800), (420, 430)], 128, 128, 64, 5),       # five heads, 25 positions
]


@pytest.mark.parametrize("case", PACKED, ids=[f"{i}-b{len(c[2])}d{c[3]}p{c[4]}w{c[5]}f{c[6]}"
                                              for i, c in enumerate(PACKED)])
def test_window_packed(case):
    from attention_forward_blackwell_gb300 import binding
    Hq, Hkv, seqs, d, page, window, first = case
    nq, nk = [s[0] for s in seqs], [s[1] for s in seqs]
    B, Sk = len(seqs), max(nk)
    g = torch.Generator().manual_seed(sum(nk))
    q = torch.randn(sum(nq), Hq, d, generator=g).bfloat16()
    k, v = (torch.randn(B, Hkv, Sk, d, generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0] + nq).cumsum(0)
    more = dict(causal=True, window=window, first=first)
    if page:
        kc, vc, table, _ = to_pages(k.cuda(), v.cuda(), nk, page, seed=page)
        call = lambda: binding.prefill_varlen_paged(args[0], kc, vc, args[1], max(nq), table,
                                                    args[2], **more)
        args = (q.cuda(), i32(cu.tolist()), i32(nk))
    else:
        kp, vp = (torch.cat([x[b, :, :n].transpose(0, 1) for b, n in enumerate(nk)]).cuda()
                  for x in (k, v))
        args = (q.cuda(), i32(cu.tolist()), i32(torch.tensor([0] + nk).cumsum(0).tolist()))
        call = lambda: binding.prefill_varlen(args[0], kp, vp, args[1], args[2], max(nq), max(nk),
                                              **more)
    o, lse = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()       # a replay gives the same bits
    with torch.cuda.graph(graph):
        o2, lse2 = call()
    o2.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    check_device_error()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b, (n, m) in enumerate(seqs):
        if n == 0:
            continue
        s = slice(int(cu[b]), int(cu[b + 1]))
        want = ref.attention64(q[s].transpose(0, 1)[None], k[b:b + 1, :, :m], v[b:b + 1, :, :m],
                               ref.window_seen(n, [m], m, window, first, True), 1 / math.sqrt(d))
        ref.check(o[s].transpose(0, 1)[None], lse[None, :, s], want, f"packed {b}")
