"""Attention of token trees over a cache, against its definition in 64 bits."""
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


def make_bits(kind, B, T, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "tree":
        parents = torch.randint(0, 1 << 20, (B, T), generator=g) % torch.arange(1, T + 1) - 1
        return ref.ancestors(parents), parents.to(torch.int32)
    if kind == "chain":
        return torch.ones(T, T).tril().bool().expand(B, T, T).clone(), None
    if kind == "full":
        return torch.ones(B, T, T, dtype=torch.bool), None
    bits = torch.rand(B, T, T, generator=g) < 0.3       # "any": some rows see nothing
    bits[:, :: 3] = False
    return bits, None


def run(B, Hq, Hkv, T, ctx, d, page, kind="tree", ragged=False, sinks=False, shared=False,
        seed=0, spare_sk=5):
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(1000 + seed)
    nodes = [(T, 0, 1, max(1, T // 2), T - 1)[b % 5] if ragged else T for b in range(B)]
    lens = [c + t for c, t in zip(ctx, nodes)]
    Sk = max(lens) + spare_sk
    q = torch.randn(B, Hq, T, d, generator=g).bfloat16()
    k = torch.randn(B, Hkv, Sk, d, generator=g).bfloat16()
    v = torch.randn(B, Hkv, Sk, d, generator=g).bfloat16()
    sk = torch.randn(Hq, generator=g) if sinks else None
    bits, parents = make_bits(kind, 1 if shared else B, T, seed)
    words = ref.pack_bits(bits).cuda()
    if parents is not None:
        assert torch.equal(binding.tree_mask(parents.cuda()), words)
    seen = ref.tree_seen(bits.expand(B, T, T), lens, nodes, Sk)
    rows = torch.arange(T)[None] < torch.tensor(nodes)[:, None]
    want = ref.attention64(q, k, v, seen, 1 / math.sqrt(d), sk)
    for b in range(B):
        k[b, :, lens[b]:] = math.nan
        v[b, :, lens[b]:] = math.nan
    out = torch.full((B, Hq, T, d), 7.0).bfloat16().cuda()
    lse = torch.full((B, Hq, T), 7.0).cuda()
    more = dict(sinks=None if sk is None else sk.cuda(), out=out, lse=lse,
                tree_lens=torch.tensor(nodes, dtype=torch.int32).cuda() if ragged else None)
    mask = words[0].contiguous() if shared else words
    L = torch.tensor(lens, dtype=torch.int32).cuda()
    kg, vg = k.cuda(), v.cuda()
    if page:
        kc, vc, table, _ = to_pages(kg, vg, lens, page, seed=seed)
        o, l = binding.decode_tree_paged(q.cuda(), kc, vc, table, L, mask, **more)
    else:
        o, l = binding.decode_tree(q.cuda(), kg, vg, mask, seqlens_k=L, **more)
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, l, want, f"tree {B, Hq, Hkv, T, d, page, kind}", rows)
    past = ~rows[:, None].expand(-1, Hq, -1)
    assert torch.all(out.cpu()[past] == 7) and torch.all(lse.cpu()[past] == 7)


CASES = [
    # B, Hq, Hkv, T, contexts, d, page, kind, ragged, sinks, shared
    (1, 1, 1, 1, [0], 64, 0, "tree", False, False, False),
    (1, 2, 2, 1, [100], 128, 0, "tree", False, False, False),
    (2, 4, 4, 7, [63, 64], 64, 0, "tree", False, True, False),
    (3, 8, 2, 5, [0, 700, 129], 128, 0, "any", False, False, False),
    (2, 8, 1, 16, [255, 256], 128, 0, "tree", False, False, True),
    (5, 4, 2, 33, [300, 0, 17, 512, 1000], 128, 0, "tree", True, False, False),
    (5, 4, 2, 33, [300, 0, 17, 512, 1000], 128, 64, "any", True, True, False),
    (2, 10, 2, 25, [1000, 31], 256, 0, "tree", False, True, False),
    (5, 6, 2, 40, [140, 0, 260, 128, 900], 256, 128, "any", True, False, False),
    (2, 16, 2, 64, [640, 2000], 128, 128, "tree", False, False, False),
    (1, 8, 1, 100, [1500], 64, 100, "tree", False, False, False),
    (2, 3, 1, 70, [333, 90], 64, 16, "any", False, False, False),
    (2, 6, 3, 129, [250, 513], 128, 48, "chain", False, False, False),
    (1, 4, 1, 300, [40], 128, 0, "full", False, False, True),
    (3, 8, 2, 20, [1, 2, 3], 128, 7, "tree", False, False, False),
    (2, 8, 8, 12, [2048, 4096], 128, 256, "tree", False, False, False),
    (4, 12, 4, 17, [900, 20, 0, 411], 128, 32, "any", False, True, False),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-b{c[0]}h{c[1]}t{c[3]}d{c[5]}p{c[6]}{c[7]}"
                                             for i, c in enumerate(CASES)])
def test_tree(case):
    B, Hq, Hkv, T, ctx, d, page, kind, ragged, sinks, shared = case
    run(B, Hq, Hkv, T, ctx, d, page, kind, ragged, sinks, shared, seed=T + d + page)


def test_tree_without_keys():
    """sk = 0, lengths 0, and no nodes at all."""
    from attention_forward_blackwell_gb300 import binding
    q = torch.randn(2, 4, 3, 128).bfloat16().cuda()
    k = torch.zeros(2, 2, 0, 128).bfloat16().cuda()
    mask = torch.full((2, 3, 1), 7, dtype=torch.int32).cuda()
    o, lse = binding.decode_tree(q, k, k, mask)
    assert torch.all(o == 0) and torch.all(lse == -math.inf)
    k = torch.full((2, 2, 4, 128), math.nan).bfloat16().cuda()
    L = torch.tensor([0, -5], dtype=torch.int32).cuda()
    sinks = torch.randn(4).cuda()
    o, lse = binding.decode_tree(q, k, k, mask, seqlens_k=L, sinks=sinks)
    assert torch.all(o == 0) and torch.allclose(lse, sinks[None, :, None].expand_as(lse), atol=1e-5)
    out, lse = torch.full_like(q, 3), torch.full((2, 4, 3), 3.0).cuda()
    binding.decode_tree(q, k, k, mask, tree_lens=torch.zeros(2, dtype=torch.int32).cuda(),
                        seqlens_k=L, out=out, lse=lse)
    assert torch.all(out == 3) and torch.all(lse == 3)


def test_chain_is_causal_decode():
    """A chain is what causal decode computes for the same queries."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda()
               for s in ((2, 8, 9, 128), (2, 2, 777, 128), (2, 2, 777, 128)))
    mask = ref.pack_bits(torch.ones(9, 9).tril().bool()).cuda()
    o, lse = binding.decode_tree(q, k, v, mask)
    o2, lse2 = binding.decode(q, k, v, causal=True)
    torch.cuda.synchronize()
    # each is within half a step of bf16 (2^-8 relative) twice over of the same value
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * 4
    assert (lse - lse2).abs().max() <= 1e-4


def test_tree_mask():
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(5)
    for B, T in ((1, 1), (3, 31), (2, 32), (4, 33), (2, 500), (1, 1024)):
        parents = torch.randint(0, 1 << 20, (B, T), generator=g) % torch.arange(1, T + 1) - 1
        parents[:, T // 2] = T + 3            # no smaller node: a root
        words = binding.tree_mask(parents.to(torch.int32).cuda())
        assert torch.equal(words.cpu(), ref.pack_bits(ref.ancestors(parents)))
    chain = torch.arange(1024, dtype=torch.int32)[None] - 1
    words = binding.tree_mask(chain.cuda())
    assert torch.equal(words.cpu()[0], ref.pack_bits(torch.ones(1024, 1024).tril().bool()))


def test_extreme_scores():
    """A basis that grows late, and scores of both signs of 2^7."""
    from attention_forward_blackwell_gb300 import binding
    B, Hq, Hkv, T, L, d = 1, 8, 1, 20, 1300, 128
    g = torch.Generator().manual_seed(9)
    q = torch.randn(B, Hq, T, d, generator=g).bfloat16()
    k = (torch.randn(B, Hkv, L, d, generator=g) * (1 + 3 * torch.arange(L)[:, None] / L)).bfloat16()
    v = torch.randn(B, Hkv, L, d, generator=g).bfloat16()
    bits, _ = make_bits("tree", B, T, 1)
    seen = ref.tree_seen(bits, [L], [T], L)
    want = ref.attention64(q, k, v, seen, 0.3)
    o, lse = binding.decode_tree(q.cuda(), k.cuda(), v.cuda(), ref.pack_bits(bits).cuda(), scale=0.3)
    torch.cuda.synchronize()
    ref.check(o, lse, want, "extreme")


def test_bad_pages_stay_in_bounds():
    """Table entries outside the cache never address memory outside it."""
    from attention_forward_blackwell_gb300 import binding
    q = torch.randn(2, 8, 24, 128).bfloat16().cuda()
    kc = torch.randn(4, 2, 64, 128).bfloat16().cuda()
    table = torch.tensor([[0, 1 << 30, -7, 2], [-(1 << 31), 3, 99, 4]], dtype=torch.int32).cuda()
    L = torch.tensor([256, 200], dtype=torch.int32).cuda()
    mask = ref.pack_bits(torch.ones(24, 24).tril().bool()).cuda()
    o, lse = binding.decode_tree_paged(q, kc, kc, table, L, mask)
    torch.cuda.synchronize()
    check_device_error()
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


def test_streams_and_graph():
    """Two captured calls and an eager one, on streams of their own, at once."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(11)
    sets = []
    for i in range(3):
        T = (5, 40, 24)[i]
        q, k, v = (torch.randn(*s, generator=g).bfloat16()
                   for s in ((4, 8, T, 128), (4, 2, 1500, 128), (4, 2, 1500, 128)))
        bits, _ = make_bits("tree", 4, T, i)
        want = ref.attention64(q, k, v, ref.tree_seen(bits, [1500] * 4, [T] * 4, 1500), 0.09)
        sets.append((q.cuda(), k.cuda(), v.cuda(), ref.pack_bits(bits).cuda(), want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], []
    for i in range(2):
        q, k, v, m, _ = sets[i]
        binding.decode_tree(q, k, v, m, scale=0.09)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            outs.append(binding.decode_tree(q, k, v, m, scale=0.09))
        graphs.append(graph)
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        q, k, v, m, _ = sets[2]
        last = binding.decode_tree(q, k, v, m, scale=0.09, stream=streams[2])
    torch.cuda.synchronize()
    check_device_error()
    for (o, lse), s in zip(outs + [last], sets):
        ref.check(o, lse, s[4], "streams")
