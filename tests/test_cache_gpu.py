"""Page operators of a cache against their definition, and a speculative step
over a forked cache with everything together."""
import math

import pytest
import torch

import serving_ref as ref
from gpu_parity import check_device_error, free_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class State:
    """A pool of pages with some rows filled, on the GPU and as lists."""

    def __init__(self, rows, max_pages, pages, P, lens, seed):
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((rows, max_pages), -1, dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32)
        for b, n in enumerate(lens):
            for j in range(-(-n // P)):
                table[b, j] = order.pop()
                refs[table[b, j]] += 1
        self.P = P
        self.plain = ref.Pool(refs, table, torch.tensor(lens))
        self.refs, self.table = refs.cuda(), table.cuda()
        self.lens = i32(lens)

    def same(self):
        assert self.refs.tolist() == self.plain.refs
        assert self.table.tolist() == self.plain.table
        assert self.lens.tolist() == self.plain.lens

    def args(self):
        return self.refs, self.table, self.lens

    def fork(self, src, dst):
        from attention_forward_blackwell_gb300 import binding
        status = binding.cache_fork(*self.args(), i32(src), i32(dst))
        assert status.item() == self.plain.fork(src, dst)
        self.same()
        return status.item()

    def free(self, rows):
        from attention_forward_blackwell_gb300 import binding
        binding.cache_free(*self.args(), i32(rows))
        self.plain.free(rows)
        self.same()

    def reserve(self, extra):
        from attention_forward_blackwell_gb300 import binding
        copies, status = binding.cache_reserve(*self.args(), i32(extra), self.P)
        c, s = self.plain.reserve(extra, self.P)
        assert status.item() == s and copies.tolist() == c
        self.same()
        return c, s


@pytest.mark.parametrize("P", [1, 16, 100])
def test_fork_reserve_free(P):
    rows, L = 9, [3 * P, 2 * P + 1, 0, 0, 0, P, 0, 0, 0]
    s = State(rows, 6, 40, P, L, seed=P)
    assert s.fork([0, 0, 1], [2, 3, 4]) == 0
    s.reserve([0, 0, 1, P + 1, 2, 0, 0, 0, 0])
    assert s.fork([3, 1], [6, 7]) == 0
    s.reserve([1, 1, 1, 1, 1, 1, 1, 1, P])
    s.free([3, 3, 0, -1, 99, 2])
    s.reserve([2 * P] * 4 + [0] * 5)
    s.free(list(range(rows)))
    assert sum(s.plain.refs) == 0


def test_refused_forks_change_nothing():
    s = State(6, 4, 30, 16, [40, 20, 0, 0, 5, 0], seed=1)
    assert s.fork([0, 1], [2, 4]) == 2            # row 4 holds pages
    assert s.fork([0, 0], [2, 2]) == 2            # the same row twice
    assert s.fork([0, 2], [2, 3]) == 1            # a row forked into and from
    assert s.fork([0, 3], [2, 3]) == 2            # onto itself
    assert s.fork([6, 0], [2, 3]) == 1            # no such row
    assert s.fork([0, 0], [2, -1]) == 2
    assert s.fork([], []) == 0
    assert s.fork([5, 0], [2, 3]) == 0            # forking an empty row is allowed


def test_reserve_refuses_as_a_whole():
    s = State(4, 5, 12, 16, [70, 33, 0, 16], seed=2)
    assert s.fork([0], [2]) == 0
    assert s.reserve([1, 16, 1, 100])[1] == -1 - 3     # 116 keys need 8 entries of 5
    assert s.reserve([9, 40, 9, 60])[1] == 5           # 1 + 2 + 1 + 4 pages, 3 are free
    assert s.reserve([0, -5, 0, 0])[1] == 0
    assert s.reserve([9, 0, 9, 0])[1] == 0
    s.free([1])
    s.reserve([0, 48, 0, 0])


@pytest.mark.parametrize("entries,pages,extra", [(6, 12, [4, 4, 4]), (60, 16, [24, 4, 6])],
                         ids=["short spans", "long spans"])
def test_a_refused_reserve_leaves_entries_that_are_no_page(entries, pages, extra):
    """Whatever they hold, that of a shared page's mark among it."""
    s = State(3, entries, pages, 4, [6, 0, 9], seed=6)
    assert s.fork([0], [1]) == 0
    page = s.plain.table[0][0]
    junk = [-2 - page, -2, pages, 2 ** 31 - 1, -2 ** 31, -1 - pages]
    for b in range(3):
        for j in range(3, entries):
            s.plain.table[b][j] = junk[(b + j) % len(junk)]
    s.table.copy_(i32(s.plain.table))
    assert s.reserve([4 * entries - 6, 4, 4])[1] > 0     # pages are lacking
    assert s.reserve([4, 4 * entries, 4])[1] == -2       # row 1 is too short
    assert s.reserve(extra)[1] == 0
    assert s.reserve([1, 1, 4 * entries])[1] == -3


def test_long_spans_and_many_rows():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 200, (1500,), generator=g).tolist()
    lens[-20:] = [0] * 20
    s = State(1500, 60, 50000, 8, lens, seed=4)
    assert s.fork([i % 7 for i in range(20)], list(range(1480, 1500))) == 0
    extra = torch.randint(0, 260, (1500,), generator=g).tolist()
    assert s.reserve(extra)[1] == 0
    s.free(list(range(0, 1500, 2)))
    assert s.reserve([1] * 1500)[1] == 0


def test_reserve_the_last_page():
    s = State(2, 3, 5, 4, [4, 4], seed=5)
    assert s.reserve([4, 8])[1] == 0
    assert min(s.plain.refs) == 1
    assert s.reserve([5, 8])[1] == 1
    s.free([1])
    assert s.reserve([5, 1])[1] == 0


@pytest.mark.parametrize("d,Hkv,P", [(128, 4, 16), (64, 3, 100), (256, 1, 7), (96, 2, 1)])
def test_append_copy_compact(d, Hkv, P):
    from attention_forward_blackwell_gb300 import binding
    g = torch.Generator().manual_seed(d + P)
    lens, n = [3 * P + 2, 0, P - 1, 2 * P, 5], 70
    width = max(-(-(L + n) // P) for L in lens)
    s = State(5, width, 5 * width + 9, P, lens, seed=3)
    caches = [torch.randn(5 * width + 9, Hkv, P, d, generator=g).bfloat16() for _ in range(2)]
    gpu = [c.cuda() for c in caches]
    assert s.reserve([n] * 5)[1] == 0
    counts = [n, 3, 0, 65, 99]
    table = s.plain.table
    new = [torch.randn(5, n, Hkv, d, generator=g).bfloat16() for _ in range(2)]   # by token
    binding.cache_append(*gpu, s.table, s.lens, *(x.cuda().transpose(1, 2) for x in new),
                         n_new=i32(counts))
    for c, x, y in zip(caches, new, gpu):
        ref.append_rows(c, table, lens, x.transpose(1, 2), [min(x_, n) for x_ in counts])
        assert torch.equal(y.cpu(), c)
    # strides that are no multiple of 16 bytes, a contiguous tensor, no n_new
    odd = [torch.randn(5, Hkv, 4, d + 3, generator=g).bfloat16()[..., 1:d + 1] for _ in range(2)]
    binding.cache_append(*gpu, s.table, s.lens, odd[0].cuda(), odd[1].contiguous().cuda())
    for c, x, y in zip(caches, odd, gpu):
        ref.append_rows(c, table, lens, x, [4] * 5)
        assert torch.equal(y.cpu(), c)
    keep = [sorted(torch.randperm(n, generator=g)[:m].tolist()) for m in (n, 9, 0, 33, 1)]
    kt = torch.full((5, n), 12345, dtype=torch.int32)
    for b, ks in enumerate(keep):
        kt[b, :len(ks)] = torch.tensor(ks, dtype=torch.int32)
    binding.cache_compact(*gpu, s.table, s.lens, kt.cuda(), i32([len(x) for x in keep]))
    for c, y in zip(caches, gpu):
        ref.compact_rows(c, table, lens, keep)
        assert torch.equal(y.cpu(), c)
    moves = [[0, 3, P], [1, 4, P // 2], [2, 5, 0], [-1, 6, 3], [7, 10 ** 9, 3], [8, 7, 10 ** 6]]
    binding.cache_copy(*gpu, i32(moves))
    for c, y in zip(caches, gpu):
        before = c.clone()
        for a, b, r in moves:
            if 0 <= a < c.shape[0] and 0 <= b < c.shape[0]:
                c[b, :, :r] = before[a, :, :r]
        assert torch.equal(y.cpu(), c)


def test_append_skips_what_has_no_page():
    from attention_forward_blackwell_gb300 import binding
    kc = torch.randn(4, 2, 8, 64).bfloat16().cuda()
    vc = torch.randn(4, 2, 8, 64).bfloat16().cuda()
    k0 = kc.clone()
    table = i32([[1, -1, 9], [-5, 2, 3]])
    new = torch.ones(2, 2, 30, 64).bfloat16().cuda()
    binding.cache_append(kc, vc, table, i32([6, 0]), new, new)
    want = k0.clone()
    want[1, :, 6:] = 1
    want[2], want[3] = 1, 1
    torch.cuda.synchronize()
    assert torch.equal(kc, want)
    binding.cache_compact(kc, vc, table, i32([6, 2 ** 31 - 1]), i32([[3, 2 ** 31 - 1], [1, 2]]),
                          i32([2, 2]))
    torch.cuda.synchronize()
    assert torch.equal(kc, want)


def speculative_step(capture):
    """A prompt forked to three samples, a drafted tree appended to each, the
    tree attended, one path accepted, and the next token decoded."""
    from attention_forward_blackwell_gb300 import binding
    P, Hkv, Hq, d, T = 16, 2, 8, 128, 12
    g = torch.Generator().manual_seed(21)
    L = 37
    s = State(4, 8, 24, P, [L, 0, 0, 0], seed=8)
    kc, vc = (torch.randn(24, Hkv, P, d, generator=g).bfloat16().cuda() for _ in range(2))
    k_all, v_all = (torch.stack([c.cpu()[s.plain.table[0][j // P], :, j % P] for j in range(L)], 1)
                    for c in (kc, vc))                      # the prompt's rows [Hkv, L, d]
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 3, 5, 6, 8, 9]] * 4, dtype=torch.int32)
    q = torch.randn(4, Hq, T, d, generator=g).bfloat16()
    k_new, v_new = (torch.randn(4, T, Hkv, d, generator=g).bfloat16() for _ in range(2))
    q1 = torch.randn(4, Hq, 1, d, generator=g).bfloat16()
    k1, v1 = (torch.randn(4, Hkv, 1, d, generator=g).bfloat16() for _ in range(2))
    nodes = [0, 12, 5, 1]
    keep = [[], [0, 1, 3, 6, 9], [0, 2], [0]]
    kt = torch.zeros(4, T, dtype=torch.int32)
    for b, x in enumerate(keep):
        kt[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    dev = dict(q=q.cuda(), kn=k_new.cuda().transpose(1, 2), vn=v_new.cuda().transpose(1, 2),
               q1=q1.cuda(), k1=k1.cuda(), v1=v1.cuda(), parents=parents.cuda(), kt=kt.cuda(),
               nodes=i32(nodes), nk=i32([len(x) for x in keep]), src=i32([0] * 3),
               dst=i32([1, 2, 3]), lens0=s.lens.clone(), table0=s.table.clone(),
               refs0=s.refs.clone(), one=i32([0, 1, 1, 1]))
    kc0, vc0 = kc.clone(), vc.clone()
    out = torch.zeros_like(dev["q"])
    lse = torch.zeros(4, Hq, T).cuda()

    def step():
        s.lens.copy_(dev["lens0"]), s.table.copy_(dev["table0"]), s.refs.copy_(dev["refs0"])
        kc.copy_(kc0), vc.copy_(vc0)
        binding.cache_fork(*s.args(), dev["src"], dev["dst"])
        copies, status = binding.cache_reserve(*s.args(), dev["nodes"], P)
        binding.cache_append(kc, vc, s.table, s.lens, dev["kn"], dev["vn"], n_new=dev["nodes"],
                             copies=copies)
        start = s.lens.clone()
        s.lens.add_(dev["nodes"])
        mask = binding.tree_mask(dev["parents"])
        binding.decode_tree_paged(dev["q"], kc, vc, s.table, s.lens, mask, tree_lens=dev["nodes"],
                                  out=out, lse=lse)
        binding.cache_compact(kc, vc, s.table, start, dev["kt"], dev["nk"])
        s.lens.copy_(start + dev["nk"])
        copies, status2 = binding.cache_reserve(*s.args(), dev["one"], P)
        binding.cache_append(kc, vc, s.table, s.lens, dev["k1"], dev["v1"], n_new=dev["one"],
                             copies=copies)
        s.lens.add_(dev["one"])
        o1, lse1 = binding.decode_paged(dev["q1"], kc, vc, s.table, s.lens)
        return status, status2, o1, lse1

    status, status2, o1, lse1 = step()
    if capture:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            status, status2, o1, lse1 = step()
        for _ in range(3):
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    check_device_error()
    assert status.item() == 0 and status2.item() == 0
    bits = ref.ancestors(parents)
    rows = torch.arange(T)[None] < torch.tensor(nodes)[:, None]
    for b in range(1, 4):
        kk = torch.cat([k_all, k_new[b, :nodes[b]].transpose(0, 1)], 1)[None]
        vv = torch.cat([v_all, v_new[b, :nodes[b]].transpose(0, 1)], 1)[None]
        seen = ref.tree_seen(bits[b:b + 1], [L + nodes[b]], [nodes[b]], L + nodes[b])
        ref.check(out[b:b + 1], lse[b:b + 1], ref.attention64(q[b:b + 1], kk, vv, seen, d ** -0.5),
                  f"step tree {b}", rows[b:b + 1])
        kk = torch.cat([k_all, k_new[b, keep[b]].transpose(0, 1), k1[b]], 1)[None]
        vv = torch.cat([v_all, v_new[b, keep[b]].transpose(0, 1), v1[b]], 1)[None]
        seen = torch.ones(1, 1, kk.shape[2], dtype=torch.bool)
        ref.check(o1[b:b + 1], lse1[b:b + 1],
                  ref.attention64(q1[b:b + 1], kk, vv, seen, d ** -0.5), f"step next {b}")
    # the prompt's own row is as it was
    seen = torch.ones(1, 1, L, dtype=torch.bool)
    ref.check(o1[:1], lse1[:1], ref.attention64(q1[:1], k_all[None], v_all[None], seen, d ** -0.5),
              "step prompt")


@pytest.mark.parametrize("capture", [False, True])
def test_speculative_step(capture):
    speculative_step(capture)
