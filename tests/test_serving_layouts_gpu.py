"""Inputs in other layouts: a call with first keys takes what the same call
without them takes."""
import pytest
import torch

from gpu_parity import check_device_error, free_cuda

pytestmark = pytest.mark.gpu

WINDOW = dict(causal=True, window=30, first=3)


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def strided(t):
    wide = torch.full((*t.shape[:-1], 2 * t.shape[-1]), 1, dtype=t.dtype, device="cuda")
    wide[..., ::2] = t
    return wide[..., ::2]


def randn(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).bfloat16().cuda() for s in shapes]


def same(call, args, kw, wide_args, wide_kw, **more):
    """The call over dense inputs and over the same in other layouts, on the current
    stream and, while that is busy, on another."""
    want = call(*args, **kw, **more)
    got = call(*wide_args, **wide_kw, **more)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    late = call(*wide_args, **wide_kw, **more, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(side):
        late = [t.cpu() for t in late]
    torch.cuda.synchronize()
    check_device_error()
    for a, b, c in zip(want, got, late):
        assert torch.equal(a, b) and torch.equal(a.cpu(), c)


@pytest.mark.parametrize("heads", [4, 32], ids=["few rows", "many rows"])
@pytest.mark.parametrize("more", [{}, WINDOW], ids=["plain", "first keys"])
def test_decode(more, heads):
    from attention_forward_blackwell_gb300 import binding
    q, k, v = randn(1, (3, heads, 9, 64), (3, 2, 700, 64), (3, 2, 700, 64))
    lens, sinks = i32([700, 31, 0]), torch.randn(heads, device="cuda")
    same(binding.decode, (q, k, v), dict(seqlens_k=lens, sinks=sinks), (q, k, v),
         dict(seqlens_k=strided(lens), sinks=strided(sinks)), **more)


@pytest.mark.parametrize("more", [{}, WINDOW], ids=["plain", "first keys"])
def test_decode_paged(more):
    from attention_forward_blackwell_gb300 import binding
    q, k, v = randn(2, (3, 4, 5, 64), (9, 2, 16, 64), (9, 2, 16, 64))
    table, lens = i32([[0, 4, 2], [5, 6, -1], [8, 1, 3]]), i32([48, 17, 40])
    dense = (q, k, v, table, lens)
    same(binding.decode_paged, dense, {}, tuple(strided(t) for t in dense), {}, **more)
    if more:
        sinks = torch.randn(4, device="cuda")
        same(binding.decode_paged, dense, dict(sinks=sinks), dense, dict(sinks=strided(sinks)), **more)
    for i in range(3):
        wrong = [t.half() if i == j else t for j, t in enumerate(dense)]
        with pytest.raises(ValueError):
            binding.decode_paged(*wrong, **more)


def test_trees():
    from attention_forward_blackwell_gb300 import binding
    q, k, v = randn(3, (3, 4, 5, 64), (9, 2, 16, 64), (9, 2, 16, 64))
    table, lens, nodes = i32([[0, 4, 2], [5, 6, -1], [8, 1, 3]]), i32([48, 17, 40]), i32([5, 5, 5])
    sinks = torch.randn(4, device="cuda")
    mask = binding.tree_mask(i32([[-1, 0, 0, 1, 3]] * 3))
    same(binding.decode_tree_paged, (q, k, v, table, lens, mask), dict(tree_lens=nodes, sinks=sinks),
         (q, k, v, strided(table), strided(lens), mask),
         dict(tree_lens=strided(nodes), sinks=strided(sinks)))
    with pytest.raises(ValueError):
        binding.decode_tree_paged(q, k, v, table.cpu(), lens, mask)
    with pytest.raises(ValueError):
        binding.decode_tree_paged(q, k, v, table, lens.long(), mask)
