"""Rotated positions against the rotation's definition in 64 bits (GPU)."""
import math

import pytest
import torch

import q8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from attention_forward_blackwell_gb300 import binding
    binding.lib()
    return binding


def rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).bfloat16().cuda()


def near(y, x, positions, inv, factor, interleaved, inverse, what):
    want = ref.turn64(x.cpu(), positions.cpu(), inv, factor, interleaved, inverse)
    off = (y.cpu().double() - want).abs()
    over = off - ref.turn_bound(x.cpu(), want, positions.cpu(), 2 * len(inv), factor, interleaved)
    print(f"{what}: off by {off.max().item():.2e}")
    assert over.max().item() <= 0, f"{what}: {over.max().item():.2e} over its bound"


CASES = [  # tokens, hq, hk, d, rot, start, method
    (1, 32, 8, 128, 128, 100000, "yarn"), (1, 1, 1, 16, 16, 0, None), (5, 3, 1, 64, 32, 7, "ntk"),
    (130, 4, 4, 96, 48, 1000, "linear"), (33, 2, 2, 80, 80, 2 ** 20, None), (17, 5, 0, 256, 64, 12, "yarn"),
    (700, 40, 8, 128, 128, 0, None), (3, 2, 1, 512, 512, 2 ** 31 - 4, None), (9, 1, 1, 48, 16, -5, None)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot,start,method", CASES)
def test_packed(fa, n, hq, hk, d, rot, start, method, interleaved):
    inv, factor = fa.rope_inv_freq(rot, method=method, stretch=8.0, original=4096)
    at = (torch.arange(n) + start).to(torch.int32).cuda()
    q = rows(n + d, n, hq, d)
    k = rows(n + d + 1, n, hk, d) if hk else None
    for inverse in (False, True):
        qo, ko = fa.rope(q, k, at, fa.rope_freqs(inv), interleaved=interleaved, inverse=inverse, factor=factor)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                assert y is None
                continue
            near(y.transpose(0, 1), x.transpose(0, 1), at, inv, factor, interleaved, inverse, "packed")
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("per_entry", [False, True])
@pytest.mark.parametrize("B,hq,hk,n,d,rot", [(1, 2, 1, 1, 64, 64), (5, 4, 2, 1, 128, 64), (3, 4, 2, 37, 128, 96),
                                           (2, 16, 16, 600, 96, 48)])
def test_batched_positions_strides_in_place(fa, B, hq, hk, n, d, rot, per_entry):
    inv, _ = fa.rope_inv_freq(rot)
    freqs = fa.rope_freqs(inv)
    g = torch.Generator().manual_seed(3)
    shape = (B, n) if per_entry else (n,)
    at = torch.randint(0, 5000, shape, generator=g).to(torch.int32).cuda()
    # one projection's output, queries and keys side by side: strided views
    x = rows(5, B, n, hq + 2 * hk, d)
    before = x.clone()
    q, k = x[:, :, :hq].transpose(1, 2), x[:, :, hq:hq + hk].transpose(1, 2)
    q0, k0 = q.clone(), k.clone()
    where = at[:, None] if per_entry else at
    qo, ko = fa.rope(q, k, at, freqs)
    near(qo, q0, where, inv, 1.0, False, False, "strided")
    near(ko, k0, where, inv, 1.0, False, False, "strided")
    assert torch.equal(x, before)
    q2, k2 = fa.rope(q, k, at, freqs, q_out=q, k_out=k)   # in place, in the projection's own memory
    assert q2.data_ptr() == q.data_ptr() and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, :, hq + hk:], before[:, :, hq + hk:])
    # side by side in memory of its own, and parts of one projection that share heads
    wide = torch.zeros_like(x)
    q3, k3 = fa.rope(q0, k0, at, freqs, q_out=wide[:, :, :hq].transpose(1, 2),
                     k_out=wide[:, :, hq:hq + hk].transpose(1, 2))
    assert torch.equal(q3, qo) and torch.equal(k3, ko) and not wide[:, :, hq + hk:].any()
    if n > 1:
        with pytest.raises(ValueError):
            fa.rope(q0, k0, at, freqs, q_out=wide[:, :, :hq].transpose(1, 2),
                    k_out=wide[:, :, hq - 1:hq - 1 + hk].transpose(1, 2))
    # an unaligned view, and an input expanded over the heads
    odd = rows(6, B, hq, n, d + 4)[..., 4:]
    near(fa.rope(odd, None, at, freqs)[0], odd, where, inv, 1.0, False, False, "unaligned")
    wide = rows(7, B, 1, n, d).expand(B, hq, n, d)
    near(fa.rope(wide, None, at, freqs)[0], wide, where, inv, 1.0, False, False, "expanded")


def test_many_rows_and_far_apart(fa):
    """The form of many heads a thread, and rows past 2^31 elements of each other."""
    inv, _ = fa.rope_inv_freq(128)
    freqs = fa.rope_freqs(inv)
    q = rows(1, 4096, 41, 128)
    at = torch.arange(4096, dtype=torch.int32, device="cuda") * 7
    y, _ = fa.rope(q, None, at, freqs)
    near(y.transpose(0, 1), q.transpose(0, 1), at, inv, 1.0, False, False, "many")
    far = torch.zeros(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    two = far.as_strided((2, 3, 128), (2 ** 31, 128, 1))
    two.copy_(rows(2, 2, 3, 128))
    y, _ = fa.rope(two, None, at[:2].contiguous(), freqs)
    near(y.transpose(0, 1), two.transpose(0, 1), at[:2], inv, 1.0, False, False, "far apart")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(fa, interleaved):
    """inverse gives the gradient: autograd's of the 64-bit formula, and the differences of the call itself
    (it is linear, so that a difference over a unit step is a column of its matrix)."""
    n, h, d, rot = 6, 2, 64, 32
    inv, factor = fa.rope_inv_freq(rot, method="yarn", stretch=4.0, original=64)
    freqs = fa.rope_freqs(inv)
    at = torch.arange(11, 11 + n, dtype=torch.int32)
    x, up = rows(1, h, n, d).cpu(), rows(2, h, n, d).cpu()
    leaf = x.double().requires_grad_()
    a, b = (leaf[..., 0:rot:2], leaf[..., 1:rot:2]) if interleaved else (leaf[..., :rot // 2], leaf[..., rot // 2:rot])
    angle = at.double()[:, None] * inv
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    ((a * c - b * s) * up[..., 0:rot:2 if interleaved else 1][..., :rot // 2].double()).sum().backward(retain_graph=True)
    second = up[..., 1:rot:2] if interleaved else up[..., rot // 2:rot]
    ((b * c + a * s) * second.double()).sum().backward()
    want = leaf.grad.clone()
    want[..., rot:] = up[..., rot:].double()
    got, _ = fa.rope(up.transpose(0, 1).contiguous().cuda(), None, at.cuda(), freqs, interleaved=interleaved,
                     inverse=True, factor=factor)
    got = got.cpu().double().transpose(0, 1)
    bound = ref.turn_bound(up, want, at, rot, factor, interleaved)
    assert torch.all((got - want).abs() <= bound)
    # one token: f(e_i) - f(0) for every i
    unit = torch.eye(d).bfloat16()[:, None].cuda()                      # d tokens of one head
    here = torch.full((d,), 13, dtype=torch.int32).cuda()
    col, _ = fa.rope(unit, None, here, freqs, interleaved=interleaved, factor=factor)
    zero, _ = fa.rope(torch.zeros_like(unit), None, here, freqs, interleaved=interleaved, factor=factor)
    diff = (col - zero)[:, 0].cpu().double() @ up[0, 2].double()        # sum_j dy_j/dx_i up_j
    # columns are rounded to bf16 (2^-8 of at most factor), and so is the gradient
    assert torch.all((diff - got[0, 2]).abs() <= 2.0 ** -8 * (factor * 2 * up[0, 2].abs().max() + got[0, 2].abs()) + 1e-6)


def test_empty_and_refused(fa):
    freqs = fa.rope_freqs(fa.rope_inv_freq(32)[0])
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(0, dtype=torch.int32, device="cuda")
    q, k = fa.rope(z, None, at, freqs)
    assert q.shape == z.shape and k is None
    x = rows(1, 4, 2, 64)
    at = torch.arange(4, dtype=torch.int32, device="cuda")
    none = fa.rope_freqs([])
    assert torch.equal(fa.rope(x, None, at, none)[0], x)               # nothing is turned
    big = rows(2, 6, 2, 64)
    for bad in (lambda: fa.rope(x.float(), None, at, freqs), lambda: fa.rope(x, x[:3], at, freqs),
                lambda: fa.rope(x, None, at.long(), freqs), lambda: fa.rope(x, None, at[:3], freqs),
                lambda: fa.rope(x, None, at, freqs.int()), lambda: fa.rope(x, None, at.cpu(), freqs),
                lambda: fa.rope(x, None, at, freqs, q_out=x[:, :1].expand(4, 2, 64)),
                lambda: fa.rope(big[:4], None, at, freqs, q_out=big[2:]),
                lambda: fa.rope(x, big[:4], at, freqs, k_out=x), lambda: fa.rope(big[:4], x, at, freqs, q_out=x),
                lambda: fa.rope(x, big[:4], at, freqs, q_out=big[2:], k_out=big[:4]),
                lambda: fa.rope(x, None, at, freqs, factor=0.0),
                lambda: fa.rope(x, None, at, fa.rope_freqs(fa.rope_inv_freq(128)[0])),
                lambda: fa.rope(x, None, at, fa.rope_freqs(fa.rope_inv_freq(24)[0])),
                lambda: fa.rope(rows(1, 4, 2, 60), None, at, freqs)):
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            bad()


@pytest.mark.parametrize("order", ["BPHN", "PBHN", "BHPN", "BHNP", "HBNP", "NBPH"])
@pytest.mark.parametrize("B,H,n", [(2, 4, 6), (1, 3, 5), (3, 1, 7), (2, 5, 1), (1, 1, 4)])
def test_in_place_in_any_order_of_the_dimensions(fa, order, B, H, n):
    """Queries and keys of one projection (P), turned where they lie or into another one's parts."""
    size = dict(B=B, P=3, H=H, N=n)
    x = rows(4, *(size[c] for c in order), 64)
    part = lambda t, p: t.permute(*(order.index(c) for c in "PBHN"), 4)[p]
    at, freqs = torch.arange(n, dtype=torch.int32, device="cuda") + 3, fa.rope_freqs(fa.rope_inv_freq(64)[0])
    before, wide = x.clone(), torch.zeros_like(x)
    q, k = fa.rope(part(x, 0), part(x, 1), at, freqs)
    fa.rope(part(x, 0), part(x, 1), at, freqs, q_out=part(wide, 2), k_out=part(wide, 0))
    assert torch.equal(part(wide, 2), q) and torch.equal(part(wide, 0), k) and not part(wide, 1).any()
    assert torch.equal(x, before)
    for bad in (dict(q_out=part(x, 1), k_out=part(x, 0)), dict(q_out=part(x, 2), k_out=part(x, 0)),
                dict(q_out=part(x, 2), k_out=part(x, 2))):   # swapped, or both in one place
        with pytest.raises(ValueError, match="share memory"):
            fa.rope(part(x, 0), part(x, 1), at, freqs, **bad)
    fa.rope(part(x, 0), part(x, 1), at, freqs, q_out=part(x, 2), k_out=part(x, 1))
    assert torch.equal(part(x, 2), q) and torch.equal(part(x, 1), k) and torch.equal(part(x, 0), part(before, 0))
    fa.rope(part(x, 0), None, at, freqs, q_out=part(x, 0))
    assert torch.equal(part(x, 0), q)


def test_outputs_that_overlap_themselves(fa):
    """Outputs whose own rows share memory are refused (two threads would write there), rows that only
    pass one another by are not; of two outputs neither may lie in the other."""
    x, at = rows(1, 2, 4, 6, 64), torch.arange(6, dtype=torch.int32, device="cuda")
    freqs = fa.rope_freqs(fa.rope_inv_freq(32)[0])
    want, _ = fa.rope(x, None, at, freqs)
    mem = torch.zeros(20000, dtype=torch.bfloat16, device="cuda")
    for strides in ((2000, 400, 32, 1), (2000, 56, 250, 1), (1000, 400, 64, 1), (0, 400, 64, 1)):
        with pytest.raises(ValueError, match="overlap|16-byte"):
            fa.rope(x, None, at, freqs, q_out=mem.as_strided(x.shape, strides))
        with pytest.raises(ValueError, match="overlap|16-byte"):   # in place too
            y = mem.as_strided(x.shape, strides)
            fa.rope(y, None, at, freqs, q_out=y)
    for strides in ((1600, 400, 64, 1), (2000, 64, 304, 1), (64, 1000, 128, 1)):
        assert torch.equal(fa.rope(x, None, at, freqs, q_out=mem.as_strided(x.shape, strides))[0], want)
    one = rows(2, 1, 1, 6, 64)   # (strides of dimensions of one element say nothing)
    assert torch.equal(fa.rope(one, None, at, freqs, q_out=mem.as_strided(one.shape, (0, 8, 64, 1)))[0],
                       fa.rope(one, None, at, freqs)[0])
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.uint8, device="cuda").view(ref.F8)
    scale, table = torch.ones(3, 2, 1, device="cuda"), torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    k = mem[:40 * 128].view(40, 2, 64)
    for v in (k, mem[64:64 + 40 * 128].view(40, 2, 64)):
        with pytest.raises(ValueError, match="share memory"):
            fa.cache_read_q8(cache, cache, scale, scale, table, cu, 40, 40, k_out=k, v_out=v)
    fa.cache_read_q8(cache, cache, scale, scale, table, cu, 40, 40, k_out=k, v_out=mem[40 * 128:80 * 128].view(40, 2, 64))


def test_k_out_without_k(fa):
    """Refused: it would stay as it is."""
    x, at = rows(1, 6, 4, 64), torch.arange(6, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="k_out without k"):
        fa.rope(x, None, at, fa.rope_freqs(fa.rope_inv_freq(32)[0]), k_out=torch.zeros_like(x))


def test_angles_against_cuda(fa):
    """The call's sines and cosines, through pairs (1, 0) whose products are exact, in bf16."""
    g = torch.Generator().manual_seed(9)
    turns = torch.rand(8, generator=g, dtype=torch.float64) * 2 * math.pi
    freqs = fa.rope_freqs(turns)
    at = torch.randint(-2 ** 31, 2 ** 31 - 1, (4000,), generator=g).to(torch.int32)
    x = torch.zeros(4000, 1, 16, dtype=torch.bfloat16)
    x[..., :8] = 1
    y, _ = fa.rope(x.cuda(), None, at.cuda(), freqs)
    # the table's own whole numbers, reduced without rounding
    part = [[(p * f) % 2 ** 64 for f in freqs.tolist()] for p in at.tolist()]
    angle = torch.tensor([[v / 2 ** 64 for v in row] for row in part], dtype=torch.float64) * 2 * math.pi
    want = torch.cat([torch.cos(angle), torch.sin(angle)], 1)
    off = (y[:, 0].cpu().double() - want).abs()
    assert torch.all(off <= 2.0 ** -8 * want.abs() + 2.0 ** -22)
