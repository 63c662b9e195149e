"""The rotation, the appends and the 8-bit cache's calls together, as a serving loop uses them: steps over
forked sequences, prompts in chunks, captured and replayed, on streams of their own, and as the README writes
them (GPU)."""
import os
import re

import pytest
import torch

import q8_line
import q8_ref as ref
import serving_ref
from gpu_parity import check_device_error, free_cuda

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BUSY = 100_000_000


@pytest.fixture(scope="module")
def fa():
    from attention_forward_blackwell_gb300 import binding, build
    build.build()
    yield binding
    free_cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(g, *shape):
    return torch.randn(*shape, generator=g).bfloat16()


def gathered(cache, table, lens):
    """Values and scales of the sequences' keys on the CPU, as the kernels left them (in 64 bits)."""
    out = []
    m = max(lens)
    for codes, scale in cache:
        codes, scale = codes.cpu().double(), scale.cpu().double()
        page, block = codes.shape[2], codes.shape[2] // scale.shape[2]
        x = torch.zeros(len(lens), codes.shape[1], m, codes.shape[3], dtype=torch.float64)
        s = torch.zeros(len(lens), codes.shape[1], m, dtype=torch.float64)
        for b, n in enumerate(lens):
            for j in range(n):
                p = int(table[b][j // page])
                s[b, :, j] = scale[p, :, j % page // block]
                x[b, :, j] = codes[p, :, j % page] * s[b, :, j, None]
        out.append((x, s))
    return out


def near_rows(values, scales, rows, what):
    """Values of a cache against the rows that were appended: within half a step of a code of the scale
    (two roundings where a scale grew: a step)."""
    step = 2 * ref.half_step(values / scales[..., None]) * scales[..., None]
    assert torch.all((values - rows).abs() <= step * 1.01), what


def test_steps_over_forked_sequences(fa):
    """A prompt, three samples that go on from it: pages shared, the open one copied with its scales when a
    sample writes; every step turns, appends and attends in two calls."""
    g = torch.Generator().manual_seed(1)
    P, block, hq, hkv, d, L0, steps = 16, 8, 8, 2, 128, 37, 12
    inv, factor = fa.rope_inv_freq(d, method="yarn", stretch=4.0, original=32)
    freqs, turn = fa.rope_freqs(inv), dict(factor=factor)
    kc, vc = (torch.zeros(40, hkv, P, d, device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.zeros(40, hkv, P // block, device="cuda") for _ in range(2))
    refs, table, lens = i32([0] * 40), i32([[-1] * 8] * 4), i32([0] * 4)
    k0, v0 = randn(g, 4, hkv, L0, d), randn(g, 4, hkv, L0, d)
    n0 = i32([L0, 0, 0, 0])
    _, status = fa.cache_reserve(refs, table, lens, n0, P)
    fa.cache_append_q8(kc, vc, ks, vs, table, lens, k0.cuda(), v0.cuda(), freqs, n_new=n0, **turn)
    lens += n0
    assert status.item() == 0 and fa.cache_fork(refs, table, lens, i32([0, 0, 0]), i32([1, 2, 3])).item() == 0
    history = [[k0[0], v0[0]] for _ in range(4)]
    for step in range(steps):
        k1, v1, q = randn(g, 4, hkv, 1, d) * 2 ** (step % 3), randn(g, 4, hkv, 1, d), randn(g, 4, hq, 1, d)
        n1 = [0 if step < 3 else 1, 1, 1, 1]              # the prompt's own row waits: its page stays shared
        extra = i32([x if x else -1 for x in n1])
        copies, status = fa.cache_reserve(refs, table, lens, extra, P)
        qr = fa.cache_append_q8(kc, vc, ks, vs, table, lens, k1.cuda(), v1.cuda(), freqs, n_new=i32(n1),
                                copies=copies, q=q.cuda(), q_out=torch.zeros_like(q).cuda(), **turn)
        assert status.item() == 0
        lens += i32(n1)
        o, lse = fa.decode_paged_q8(qr, kc, vc, ks, vs, table, lens, causal=True)
        for b in range(4):
            if n1[b]:
                history[b] = [torch.cat([history[b][0], k1[b]], 1), torch.cat([history[b][1], v1[b]], 1)]
        n = lens.tolist()
        (k, sk), (v, sv) = gathered(((kc, ks), (vc, vs)), table.cpu(), n)
        for b in range(4):
            want = ref.turn64(history[b][0], torch.arange(n[b]), inv, factor)
            near_rows(k[b, :, :n[b]], sk[b, :, :n[b]], want, f"step {step}, keys of {b}")
            near_rows(v[b, :, :n[b]], sv[b, :, :n[b]], history[b][1].double(), f"step {step}, values of {b}")
        want = ref.attention8(qr, k, v, sv, serving_ref.window_seen(1, n, max(n), 0, 0, True), d ** -0.5)
        serving_ref.check(o, lse, want, f"step {step}")
    check_device_error()


@pytest.mark.parametrize("window,first", [(0, 0), (50, 3)])
def test_prompts_in_chunks(fa, window, first):
    """Chunks of prompts: turned and appended, read back packed, attended by the packed prefill."""
    g = torch.Generator().manual_seed(2)
    P, block, hq, hkv, d = 32, 32, 4, 2, 64
    inv, _ = fa.rope_inv_freq(d)
    freqs = fa.rope_freqs(inv)
    kc, vc = (torch.zeros(40, hkv, P, d, device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.zeros(40, hkv, 1, device="cuda") for _ in range(2))
    refs, table, lens = i32([0] * 40), i32([[-1] * 10] * 3), i32([0] * 3)
    for chunk in ([100, 3, 64], [40, 77, 1], [1, 64, 90]):
        n = max(chunk)
        q, k, v = randn(g, 3, hq, n, d), randn(g, 3, hkv, n, d), randn(g, 3, hkv, n, d)
        new = i32(chunk)
        copies, status = fa.cache_reserve(refs, table, lens, new, P)
        qr = fa.cache_append_q8(kc, vc, ks, vs, table, lens, k.cuda(), v.cuda(), freqs, n_new=new, copies=copies, q=q.cuda())
        assert status.item() == 0
        lens += new
        total = lens.tolist()
        cu_k = [0, total[0], total[0] + total[1], sum(total)]
        cu_q = [0, chunk[0], chunk[0] + chunk[1], sum(chunk)]
        kr, vr = fa.cache_read_q8(kc, vc, ks, vs, table, i32(cu_k), cu_k[-1], max(total))
        packed = torch.cat([qr[b, :, :c].transpose(0, 1) for b, c in enumerate(chunk)])
        o, lse = fa.prefill_varlen(packed, kr, vr, i32(cu_q), i32(cu_k), n, max(total), causal=True, window=window, first=first)
        (kk, _), (vv, _) = gathered(((kc, ks), (vc, vs)), table.cpu(), total)
        for b, c in enumerate(chunk):
            m = total[b]
            assert torch.equal(kr[cu_k[b]:cu_k[b + 1]].cpu().double(), kk[b, :, :m].transpose(0, 1))
            seen = serving_ref.window_seen(c, [m], m, window, first, True)
            want = serving_ref.attention64(packed[cu_q[b]:cu_q[b + 1]].transpose(0, 1)[None], kk[b:b + 1, :, :m],
                                           vv[b:b + 1, :, :m], seen, d ** -0.5)
            serving_ref.check(o[cu_q[b]:cu_q[b + 1]].transpose(0, 1)[None], lse[:, cu_q[b]:cu_q[b + 1]][None], want, f"chunk {b}")
    check_device_error()


def state(seed, B, hq, hkv, d, lens, page=32, width=None):
    """A step's tensors."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + 1) // page) for n in lens]
    order = torch.randperm(sum(need), generator=g).tolist()
    width = width or max(need)
    table = []
    for n in need:
        table.append(order[:n] + [-1] * (width - n))
        order = order[n:]
    kc, ks = ref.codes8(g, sum(need) + 1, hkv, page, page // 2, d)
    vc, vs = ref.codes8(g, sum(need) + 1, hkv, page, page // 2, d)
    return dict(kc=kc, vc=vc, ks=ks, vs=vs, table=i32(table), lens=i32(lens), k=randn(g, B, hkv, 1, d).cuda(),
                v=randn(g, B, hkv, 1, d).cuda(), q=randn(g, B, hq, 1, d).cuda())


def step(fa, s, freqs, stream=None):
    qr = fa.cache_append_q8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["k"], s["v"], freqs, q=s["q"],
                            stream=stream)
    return fa.decode_paged_q8(qr, s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"] + 1, causal=True,
                              stream=stream)


SIZES = [  # one cluster for each unit; pieces that end with their units; a line with cuts; few units in many pieces
    (2, 8, 2, 128, [100, 700], None), (5, 16, 4, 64, [3000, 100, 2500, 2900, 5], 200),
    (40, 8, 8, 128, [50 + 97 * i for i in range(40)], 200), (1, 4, 1, 256, [9000], 400)]


@pytest.mark.parametrize("B,hq,hkv,d,lens,width", SIZES)
def test_captured_steps(fa, B, hq, hkv, d, lens, width):
    """A step captured twice into graphs of their own, which replay at once on two streams while eager calls
    run on a third; lengths and rows change between replays."""
    freqs = fa.rope_freqs(fa.rope_inv_freq(d)[0])
    states = [state(s, B, hq, hkv, d, lens, width=width) for s in (1, 2, 3)]
    for s in states:
        step(fa, s, freqs)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in states[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(fa, s, freqs))
        graphs.append(graph)
    for turn in range(3):
        g = torch.Generator().manual_seed(10 + turn)
        now = [max(0, n - 7 * turn) for n in lens]
        for s in states:
            s["lens"].copy_(i32(now))
            for x in "kvq":
                s[x].copy_(randn(g, *s[x].shape))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = step(fa, states[2], freqs)
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs] + [[t.clone() for t in eager]]
        for s, o in zip(states, got):   # the same step alone gives the same bits
            alone = step(fa, s, freqs)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, alone))
    check_device_error()


def calls(fa):
    """The calls that make their outputs, as name -> f(**more)."""
    s = state(5, 2, 4, 2, 64, [100, 31])
    freqs = fa.rope_freqs(fa.rope_inv_freq(64)[0])
    at = torch.arange(2, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 4, 64, device="cuda").bfloat16()
    k16, v16 = (torch.zeros(9, 2, 32, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = (s["kc"], s["vc"], s["ks"], s["vs"], s["table"])
    rows = (s["table"], s["lens"], s["k"], s["v"], freqs)
    return {
        "rope": lambda **m: fa.rope(x, x[:, :2], at, freqs, **m),
        "append_rope": lambda **m: (fa.cache_append_rope(k16, v16, *rows, q=s["q"], **m),),
        "append_q8": lambda **m: (fa.cache_append_q8(*cache[:4], *rows, q=s["q"], **m),),
        "read_q8": lambda **m: fa.cache_read_q8(*cache, i32([0, 100, 131]), 131, 100, **m),
        "decode_q8": lambda **m: fa.decode_paged_q8(s["q"], *cache, s["lens"], **m),
    }


NAMES = ["rope", "append_rope", "append_q8", "read_q8", "decode_q8"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_and_streams(fa, name):
    """On another stream: the same bits, outputs from that stream's own memory that stay until the current
    stream has read them; and on the default stream from another one."""
    call = calls(fa)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for out in call(stream=side):
        owners = [s["stream"] for s in torch.cuda.memory_snapshot()
                  if s["address"] <= out.data_ptr() < s["address"] + s["total_size"]]
        assert owners == [side.cuda_stream]
    torch.cuda.synchronize()
    out = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    got, at = [t.clone() for t in out], out[0].data_ptr()
    del out
    states = [b["state"] for s in torch.cuda.memory_snapshot() for b in s["blocks"]
              if b["address"] <= at < b["address"] + b["size"]]
    for _ in range(3):
        call(stream=side)
    torch.cuda.synchronize()
    assert states == ["active_pending_free"]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(stream=torch.cuda.default_stream())
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        got = [t.clone() for t in got]
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def strided(t):
    wide = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")
    wide[..., ::2] = t
    return wide[..., ::2]


def test_inputs_of_other_layouts_are_copied_on_the_calls_stream(fa):
    """The current stream is busy: copies made there would come after the kernel."""
    s = state(6, 2, 4, 2, 64, [100, 31])
    freqs = fa.rope_freqs(fa.rope_inv_freq(64)[0])
    at = torch.arange(2, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 4, 64, device="cuda").bfloat16()
    want = list(fa.rope(x, x, at, freqs)) + list(step(fa, s, freqs))
    wide = {n: strided(s[n]) for n in "kvq"}
    wx, wat, wf, wl = strided(x), strided(at), strided(freqs), strided(s["lens"] + 1)
    side = torch.cuda.Stream()
    args = (s["kc"], s["vc"], s["ks"], s["vs"], s["table"])
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = list(fa.rope(wx, wx, wat, wf, stream=side))
    qr = fa.cache_append_q8(*args, s["lens"], wide["k"], wide["v"], wf, q=wide["q"], stream=side)
    got += fa.decode_paged_q8(strided_on(qr, side), *args, wl, causal=True, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()   # still busy
    with torch.cuda.stream(side):
        got = [t.cpu() for t in got]
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


def strided_on(t, stream):
    with torch.cuda.stream(stream):
        return strided(t)


def test_odd_batches(fa):
    """More sequences than lanes and threads, most of them empty: every row of the outputs is written."""
    B, d = 700, 64
    g = torch.Generator().manual_seed(3)
    lens = [0] * B
    for b in range(0, B, 23):
        lens[b] = 1 + b % 40
    s = state(7, B, 3, 1, d, lens, page=16, width=100)
    kw = dict(kc=s["kc"].cpu(), vc=s["vc"].cpu())
    o = torch.full((B, 3, 1, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, 3, 1), 9.0, device="cuda")
    fa.decode_paged_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], out=o, lse=lse)
    (k, _), (v, sv) = gathered(((s["kc"], s["ks"]), (s["vc"], s["vs"])), s["table"].cpu(), lens)
    want = ref.attention8(s["q"], k, v, sv, serving_ref.window_seen(1, lens, max(lens), 0, 0, False), d ** -0.5)
    serving_ref.check(o, lse, want, "odd batch")


def test_long_lines(fa):
    """Shares of many blocks a CTA: large pieces, then small ones for the SMs that are done."""
    d, page = 64, 64
    lens = [90000, 300, 60000, 1, 70000, 80001]
    s = state(8, 6, 8, 8, d, lens, page=page)
    o, lse = fa.decode_paged_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"])
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    kr, vr = fa.cache_read_q8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], i32(ends), ends[-1], max(lens))
    for b, n in enumerate(lens):   # (the bounds of ref.attention8, by the device in 64 bits)
        q, k, v = s["q"][b].double(), kr[ends[b]:ends[b + 1]].double(), vr[ends[b]:ends[b + 1]].double()
        x = torch.einsum("hnd,mhd->hnm", q, k) / d ** 0.5
        e = torch.einsum("hnd,mhd->hnm", q.abs(), k.abs()).amax(-1) / d ** 0.5 * (d + 8) * 2.0 ** -24
        e = e + q.abs().amax(-1) * k.abs().sum(-1).amax(0)[:, None] / d ** 0.5 * 2.0 ** -25
        l = torch.logsumexp(x, -1)
        p = torch.exp(x - l[..., None])
        want, a = torch.einsum("hnm,mhd->hnd", p, v), torch.einsum("hnm,mhd->hnd", p, v.abs())
        r = n * 2.0 ** -24 + 2.0 ** -16
        low = 448 * n * 2.0 ** -31 * s["vs"].max().item() * p.amax(-1, keepdim=True)
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * e[..., None] + r) * (1 + 2.0 ** -8) * a + low
        assert torch.all((o[b].double() - want).abs() <= bound), f"sequence {b}"
        assert torch.all((lse[b].double() - l).abs() <= e + r * (1 + l.abs())), f"sequence {b}"
    check_device_error()


LINES = [  # head_dim, query heads a key head, key heads, lengths (as long as they are: the cut goes by them), cut
    (64, 8, 8, [200000, 300, 170000, 1, 140001, 50000], "two sizes"), (128, 5, 8, [160000, 0, 120033, 129, 130000], "two sizes"),
    (128, 8, 4, [3, 350000, 500, 330001, 70000], "two sizes"), (64, 16, 8, [500 + 3777 * i % 8500 for i in range(61)], "uneven"),
    (256, 7, 8, [977 * i % 5900 for i in range(43)], "uneven"), (64, 3, 2, [90001, 70000, 0, 1], "aligned")]


@pytest.mark.parametrize("d,group,hkv,lens,kind", LINES)
def test_cuts_of_long_lines(fa, d, group, hkv, lens, kind):
    """Each way of cutting the line: large pieces with small ones behind them, even pieces over the ends of
    units, pieces that end with their units.  What the cut is comes from the kernels' own arithmetic."""
    page, B, hq = 64, len(lens), group * hkv
    width = -(-max(lens) // page)
    tile, block, line = 8 if group <= 8 else 16, q8_line.lib().line_block(d), q8_line.lib()
    units, sms = hkv * -(-group // tile), torch.cuda.get_device_properties(0).multi_processor_count
    slots = min(sms * line.line_ctas(d, tile), B * units * -(-width * page // block))
    levels = line.line_levels(d, tile, float(B * units * -(-width * page // block)), slots)
    bad, cut = q8_line.line(lens, units, block, slots, levels)
    assert bad == 0
    assert kind == ("aligned" if cut["aligned"] > 0 else "two sizes" if cut["small"] > 1 else "uneven"), cut
    # A lane's sums of a segment have at most four terms a block and the product's instructions two, each
    # off by at most 2^-22, and merges, exponents and rescalings add 2^-16 as in ref.attention8: so a piece
    # left out or taken twice shows in the LSE, whatever the length.
    r = 4 * max(cut["share"], cut["aligned"]) * 2.0 ** -22 + 2.0 ** -16
    # (a pool of pages that the sequences share; the values of a block are of their scale's size)
    g = torch.Generator(device="cuda").manual_seed(d + B)
    pages = 3001
    codes = [(60 * torch.randn(pages, hkv, page, d, device="cuda", generator=g)).clamp(-448, 448).to(F8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-8, -4, (pages, hkv, 1), device="cuda", generator=g).float()) for _ in range(2)]
    table = torch.randint(0, pages, (B, width), device="cuda", generator=g, dtype=torch.int32)
    q = torch.randn(B, hq, 1, d, device="cuda", generator=g).bfloat16()
    o, lse = fa.decode_paged_q8(q, *codes, *scales, table, i32(lens))
    for b, n in enumerate(lens):   # (the bounds of ref.attention8, by the device in 64 bits)
        if n == 0:
            assert torch.all(o[b] == 0) and torch.all(lse[b] == float("-inf"))
            continue
        k, v = fa.cache_read_q8(*codes, *scales, table[b:b + 1], i32([0, n]), n, n)
        x, k, v = q[b].double().reshape(hkv, group, d), k.double(), v.double()
        e = torch.einsum("hgd,mhd->hgm", x.abs(), k.abs()).amax(-1) / d ** 0.5 * (d + 8) * 2.0 ** -24
        e = e + x.abs().amax(-1) * k.abs().sum(-1).amax(0)[:, None] / d ** 0.5 * 2.0 ** -25
        x = torch.einsum("hgd,mhd->hgm", x, k) / d ** 0.5
        l = torch.logsumexp(x, -1)
        p = torch.exp(x - l[..., None])
        want, a = torch.einsum("hgm,mhd->hgd", p, v), torch.einsum("hgm,mhd->hgd", p, v.abs())
        low = 448 * n * 2.0 ** -31 * scales[1].max().item() * p.amax(-1, keepdim=True)
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * e[..., None] + r) * (1 + 2.0 ** -8) * a + low
        off = (o[b].double().reshape(hkv, group, d) - want).abs()
        assert torch.all(off <= bound), f"sequence {b}: {(off / bound).max().item()}"
        assert torch.all((lse[b].double().reshape(hkv, group) - l).abs() <= e + r * (1 + l.abs())), f"sequence {b}"
        del x, k, v, p
    check_device_error()


def test_largest_batch(fa):
    """As many sequences as a call takes: a step of all of them, most still empty before it."""
    B, d, page = 65535, 64, 16
    g = torch.Generator(device="cuda").manual_seed(7)
    kc, vc = (torch.zeros(B, 1, page, d, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    ks, vs = (torch.zeros(B, 1, 1, device="cuda") for _ in range(2))
    table = torch.randperm(B, device="cuda", generator=g).to(torch.int32)[:, None].contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = {w: torch.randn(B, h, 1, d, device="cuda", generator=g).bfloat16() for w, h in (("k", 1), ("v", 1), ("q", 2))}
    inv = fa.rope_inv_freq(d)[0]
    freqs = fa.rope_freqs(inv)
    qr = fa.cache_append_q8(kc, vc, ks, vs, table, lens, x["k"], x["v"], freqs, q=x["q"])
    at = torch.zeros(B, 1, dtype=torch.int32, device="cuda")   # (position 0: as it was)
    assert torch.equal(qr, x["q"]) and torch.equal(fa.rope(x["q"], None, at, freqs)[0], x["q"])
    lens[::3] += 1
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    total = int(cu[-1])
    k, v = fa.cache_read_q8(kc, vc, ks, vs, table, cu, total, 1)
    assert torch.all((v.double() - x["v"][::3, :, 0].double()).abs() <= 2.0 ** -4 * x["v"][::3, :, 0].double().abs() + vs.max() * 2.0 ** -10)
    o, lse = fa.decode_paged_q8(qr, kc, vc, ks, vs, table, lens, causal=True)
    # one key: its value, and its score to fp32's d + 8 roundings and the LSE's 2^-16
    assert torch.equal(o[::3], v[:, :, None].expand(-1, 2, 1, d))
    want = torch.einsum("bhnd,bkd->bhn", qr[::3].double(), k.double()) / d ** 0.5
    size = torch.einsum("bhnd,bkd->bhn", qr[::3].double().abs(), k.double().abs()) / d ** 0.5
    low = qr[::3].double().abs().amax(-1) * k.double().abs().sum((1, 2))[:, None, None] / d ** 0.5 * 2.0 ** -25
    assert torch.all((lse[::3].double() - want).abs() <= size * (d + 8) * 2.0 ** -24 + low + (1 + want.abs()) * 2.0 ** -16)
    empty = lens == 0
    assert torch.all(o[empty] == 0) and torch.all(lse[empty] == float("-inf"))
    check_device_error()


def test_readme(fa):
    """The README's steps over an 8-bit cache, run as they are written."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        code = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "cache_append_q8" in c]
    assert len(code) == 1
    g = torch.Generator().manual_seed(9)
    B, hq, hkv, d, P, lens, chunks = 3, 4, 2, 128, 16, [40, 0, 17], [5, 30, 1]
    kc, ks = ref.codes8(g, 20, hkv, P, P, d)
    vc, vs = ref.codes8(g, 20, hkv, P, P, d)
    table = i32([[4, 9, 2, 7], [1, 3, -1, -1], [12, 11, 10, -1]])
    old = gathered(((kc, ks), (vc, vs)), table.cpu(), [max(n, 1) for n in lens])
    n, now = max(chunks), [a + c for a, c in zip(lens, chunks)]
    x = {w: randn(g, B, h, m, d) for w, h, m in (("q", hq, n), ("k_new", hkv, n), ("v_new", hkv, n),
                                                 ("q1", hq, 1), ("k1", hkv, 1), ("v1", hkv, 1))}
    cu = lambda v: i32([sum(v[:i]) for i in range(len(v) + 1)])
    names = dict(torch=torch, binding=fa, k8=kc, v8=vc, ks=ks, vs=vs, table=table, lens=i32(lens), chunks=chunks,
                 n_new=i32(chunks), cu_k=cu(now), cu_q=cu(chunks), total_k=sum(now), longest=max(now),
                 **{w: t.cuda() for w, t in x.items()})
    exec(code[0], names)
    check_device_error()
    m = [a + 1 for a in now]
    assert names["lens"].tolist() == m
    (k, sk), (v, sv) = gathered(((kc, ks), (vc, vs)), table.cpu(), m)
    inv, factor = names["inv_freq"], names["factor"]
    assert factor > 1
    for b in range(B):
        rows = torch.cat([x["k_new"][b, :, :chunks[b]], x["k1"][b]], 1)
        want = ref.turn64(rows, torch.arange(lens[b], m[b]), inv, factor)
        near_rows(k[b, :, lens[b]:m[b]], sk[b, :, lens[b]:m[b]], want, f"keys of {b}")
        near_rows(k[b, :, :lens[b]], sk[b, :, :lens[b]], old[0][0][b, :, :lens[b]], f"earlier keys of {b}")
        qr = names["qr"][b, :, :chunks[b]]
        want = ref.turn64(x["q"][b, :, :chunks[b]], torch.arange(lens[b], now[b]), inv, factor)
        assert torch.all((qr.cpu().double() - want).abs() <=
                         ref.turn_bound(x["q"][b, :, :chunks[b]], want, torch.arange(lens[b], now[b]), d, factor, False))
        at = slice(sum(now[:b]), sum(now[:b + 1]))
        kk, vv = (names[w][at].transpose(0, 1)[None] for w in ("k", "v"))
        seen = serving_ref.window_seen(chunks[b], [now[b]], now[b], 0, 0, True)
        at = slice(sum(chunks[:b]), sum(chunks[:b + 1]))
        serving_ref.check(names["o"][at].transpose(0, 1)[None], names["lse"][:, at][None],
                          serving_ref.attention64(qr[None], kk, vv, seen, d ** -0.5), f"chunk {b}")
    want = ref.attention8(names["q1r"], k, v, sv, serving_ref.window_seen(1, m, max(m), 0, 0, True), d ** -0.5)
    serving_ref.check(names["o1"], names["lse1"], want, "next token")
