"""Calls of the serving operators at their edges: nothing to do, trees longer than
their keys, rows in other layouts and on other streams, wide numbers."""
import math

import pytest
import torch

import serving_ref as ref
from gpu_parity import check_device_error, free_cuda, to_pages
from test_first_gpu import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


@pytest.mark.parametrize("Hq,Hkv,T", [(4, 2, 7), (16, 1, 70)], ids=["few rows", "many rows"])
def test_trees_longer_than_their_keys(Hq, Hkv, T):
    """t_b > L_b: the first t_b - L_b nodes have no key of their own."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(T)
    B, d, lens = 3, 128, [3, 0, T + 40]
    q, k, v = (torch.randn(*s, generator=g).bfloat16()
               for s in ((B, Hq, T, d), (B, Hkv, T + 40, d), (B, Hkv, T + 40, d)))
    bits = torch.rand(B, T, T, generator=g) < 0.5
    seen = torch.zeros(B, T, T + 40, dtype=torch.bool)
    for b, L in enumerate(lens):
        for j in range(L):
            n = j - (L - T)
            seen[b, :, j] = True if n < 0 else bits[b, :, n]
    want = ref.attention64(q, k, v, seen, d ** -0.5)
    for b, L in enumerate(lens):
        k[b, :, L:] = v[b, :, L:] = math.nan
    o, lse = binding.decode_tree(q.cuda(), k.cuda(), v.cuda(), ref.pack_bits(bits).cuda(),
                                 seqlens_k=i32(lens))
    torch.cuda.synchronize()
    check_device_error()
    ref.check(o, lse, want, "long trees")


def test_nothing_to_do():
    from attention_forward_blackwell_gb300 import binding
    kc = torch.full((4, 2, 16, 64), 5.0).bfloat16().cuda()
    vc = kc.clone()
    table, lens, refs = i32([[0, 1], [2, -1]]), i32([20, 3]), i32([1, 1, 1, 0])
    none = torch.empty(0, dtype=torch.int32).cuda()
    assert binding.cache_fork(refs, table, lens, none, none).item() == 0
    binding.cache_free(refs, table, lens, none)
    copies, status = binding.cache_reserve(refs, table, lens, i32([-1, -1]), 16)
    assert status.item() == 0 and copies.tolist() == [[-1, -1, 0]] * 2
    new = torch.zeros(2, 2, 0, 64).bfloat16().cuda()
    binding.cache_append(kc, vc, table, lens, new, new)
    binding.cache_append(kc, vc, table, lens, torch.zeros(2, 2, 3, 64).bfloat16().cuda(),
                         torch.zeros(2, 2, 3, 64).bfloat16().cuda(), n_new=i32([0, -4]))
    binding.cache_copy(kc, vc, torch.empty(0, 3, dtype=torch.int32).cuda())
    binding.cache_compact(kc, vc, table, lens, torch.empty(2, 0, dtype=torch.int32).cuda(), i32([0, 0]))
    binding.cache_compact(kc, vc, table, lens, i32([[0, 5], [0, 5]]), i32([-1, 0]))
    torch.cuda.synchronize()
    assert torch.all(kc == 5) and torch.all(vc == 5)
    assert table.tolist() == [[0, 1], [2, -1]] and lens.tolist() == [20, 3]
    assert refs.tolist() == [1, 1, 1, 0]
    assert binding.tree_mask(torch.empty(0, 5, dtype=torch.int32).cuda()).shape == (0, 5, 1)
    assert binding.tree_mask(torch.empty(3, 0, dtype=torch.int32).cuda()).shape == (3, 0, 0)
    q = torch.zeros(0, 4, 2, 64).bfloat16().cuda()
    k = torch.zeros(0, 2, 9, 64).bfloat16().cuda()
    o, lse = binding.decode(q, k, k, window=3, first=1)
    assert o.shape == q.shape and lse.shape == (0, 4, 2)


def test_packed_without_keys():
    """Packed queries of a sequence without keys: O = 0, LSE = -inf or the sink."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(2)
    for n in (5, 1100):   # each of the kernels of a packed window
        nq, nk = [n, 6, n], [0, 30, n + 7]
        q = torch.randn(sum(nq), 16, 128, generator=g).bfloat16()
        k, v = (torch.randn(sum(nk), 4, 128, generator=g).bfloat16() for _ in range(2))
        sinks = torch.randn(16, generator=g)
        cu = lambda x: i32([0, x[0], x[0] + x[1], sum(x)])
        o, lse = binding.prefill_varlen(q.cuda(), k.cuda(), v.cuda(), cu(nq), cu(nk), max(nq), max(nk),
                                        causal=True, window=9, first=3, sinks=sinks.cuda())
        torch.cuda.synchronize()
        check_device_error()
        assert torch.all(o[:n] == 0)
        # (the sink's logit goes through log2 units: two roundings of fp32)
        assert (lse[:, :n].cpu() - sinks[:, None]).abs().max() <= 4 * 2.0 ** -23 * 4
        q0 = k0 = 0
        for a, m in zip(nq, nk):
            if m:
                want = ref.attention64(q[q0:q0 + a].transpose(0, 1)[None], k[k0:k0 + m].transpose(0, 1)[None],
                                       v[k0:k0 + m].transpose(0, 1)[None],
                                       ref.window_seen(a, [m], m, 9, 3, True), 128 ** -0.5, sinks)
                ref.check(o[q0:q0 + a].transpose(0, 1)[None], lse[None, :, q0:q0 + a], want, "packed")
            q0, k0 = q0 + a, k0 + m


def test_rows_of_other_layouts_on_another_stream():
    """New rows that have to be laid out first, while the call's stream is busy and
    the current one goes on and reuses memory."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(3)
    B, Hkv, n, d, P = 4, 3, 33, 96, 16
    wide = torch.randn(B, n, Hkv, d + 1, generator=g).bfloat16().cuda()
    new = wide[..., :d].transpose(1, 2)          # odd strides
    table = i32([[4 * b + j for j in range(4)] for b in range(B)])
    kc = torch.zeros(16, Hkv, P, d).bfloat16().cuda()
    vc = torch.zeros_like(kc)
    lens = i32([0, 5, 16, 31])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    binding.cache_append(kc, vc, table, lens, new, new, stream=side)
    for _ in range(20):
        torch.full((B, Hkv, n, d), math.nan, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    want = torch.zeros(16, Hkv, P, d).bfloat16()
    ref.append_rows(want, table.tolist(), lens.tolist(), new.cpu(), [n] * B)
    assert torch.equal(kc.cpu(), want) and torch.equal(vc.cpu(), want)


def test_outputs_outlive_another_stream():
    """What a call on another stream returns may be dropped while it is at work."""
    from attention_forward_blackwell_gb300 import binding
    P, Hkv, d, B = 16, 2, 64, 6
    g = torch.Generator().manual_seed(8)
    kc = torch.randn(40, Hkv, P, d, generator=g).bfloat16().cuda()
    vc = torch.randn(40, Hkv, P, d, generator=g).bfloat16().cuda()
    table = torch.full((B, 3), -1, dtype=torch.int32)
    table[:, 0] = 7                              # one page, shared by all rows
    lens = i32([11] * B)
    refs = torch.zeros(40, dtype=torch.int32)
    refs[7] = B
    table, refs = table.cuda(), refs.cuda()
    new = torch.randn(B, Hkv, 1, d, generator=g).bfloat16().cuda()
    want = kc.cpu()
    ref.append_rows(want, [[b] for b in range(B)], [11] * B, new.cpu(), [1] * B,
                    [(7, b, 11) for b in range(B)])
    side = torch.cuda.Stream()
    one = i32([1] * B)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    copies, status = binding.cache_reserve(refs, table, lens, one, P, stream=side)
    binding.cache_append(kc, vc, table, lens, new, new, copies=copies, stream=side)
    del copies, status
    for _ in range(20):
        torch.full((B, 3), 1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert table[:, 0].tolist() == list(range(B)) and refs[:8].tolist() == [1] * B + [0, 0]
    assert torch.equal(kc.cpu(), want)


@pytest.mark.parametrize("rows", [1, 40], ids=["few rows", "many rows"])
def test_wide_numbers(rows):
    """Windows and first keys far past the keys, extras past the table."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(rows)
    q, k, v = (torch.randn(*s, generator=g).bfloat16()
               for s in ((2, 32, 4, 128), (2, 32 // rows if rows == 1 else 1, 300, 128),
                         (2, 32 // rows if rows == 1 else 1, 300, 128)))
    big = 2 ** 31 - 1
    for window, first in ((big, 1), (1, big), (big, big), (2 ** 30 + 5, 2)):
        lens = [300, 7]
        want = ref.attention64(q, k, v, ref.window_seen(4, lens, 300, window, first, True), 128 ** -0.5)
        o, lse = binding.decode(q.cuda(), k.cuda(), v.cuda(), causal=True, seqlens_k=i32(lens),
                                window=window, first=first)
        kc, vc, table, _ = to_pages(k.cuda(), v.cuda(), lens, 32, seed=1)
        o2, lse2 = binding.decode_paged(q.cuda(), kc, vc, table, i32(lens), causal=True, window=window,
                                        first=first)
        torch.cuda.synchronize()
        check_device_error()
        ref.check(o, lse, want, f"wide {window} {first}")
        ref.check(o2, lse2, want, f"wide, paged {window} {first}")
    table, lens, refs = i32([[0, -1], [1, -1]]), i32([3, 2]), i32([1, 1, 0, 0])
    copies, status = binding.cache_reserve(refs, table, lens, i32([1, big]), 4)
    assert status.item() == -2 and refs.tolist() == [1, 1, 0, 0]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_windows_past_32_bits(d):
    """The longest window a call can name, rows that stand before the first key."""
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(d)
    big = 2 ** 31 - 1
    lens = [40, 3, 1, 0]
    q, k, v = (torch.randn(*s, generator=g).bfloat16()
               for s in ((4, 2, 40, d), (4, 1, 40, d), (4, 1, 40, d)))
    want = ref.attention64(q, k, v, ref.window_seen(40, lens, 40, 0, 0, True), d ** -0.5)
    for first in (0, 1, big):
        o, lse = binding.prefill(q.cuda(), k.cuda(), v.cuda(), causal=True, seqlens_k=i32(lens),
                                 window=big, first=first)
        torch.cuda.synchronize()
        ref.check(o, lse, want, f"prefill {first}")
        if d == 512:
            continue
        qs = q[:, :, :9].contiguous()
        o, lse = binding.decode(qs.cuda(), k.cuda(), v.cuda(), causal=True, seqlens_k=i32(lens),
                                window=big, first=first)
        torch.cuda.synchronize()
        short = ref.attention64(qs, k, v, ref.window_seen(9, lens, 40, 0, 0, True), d ** -0.5)
        ref.check(o, lse, short, f"decode {first}")
    check_device_error()


def test_another_device_is_refused():
    from attention_forward_blackwell_gb300 import binding
    q = torch.zeros(1, 2, 1, 64).bfloat16()
    with pytest.raises(ValueError):
        binding.decode_tree(q, q, q, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.decode_tree(q.cuda(), q.cuda(), q, torch.zeros(1, 1, dtype=torch.int32).cuda())
    with pytest.raises(TypeError):
        binding.decode(q.cuda(), q.cuda(), q.cuda(), window=2, first=1, causal=torch.zeros(3))
