"""Calls on another stream than the current one: the memory of their outputs
while either stream is busy."""
import pytest
import torch

from gpu_parity import check_device_error, free_cuda

pytestmark = pytest.mark.gpu

BUSY = 100_000_000   # cycles that a stream sleeps: far longer than any call here


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prompt(seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).bfloat16().cuda()
            for s in ((1, 4, 200, 64), (1, 2, 256, 64), (1, 2, 256, 64))]


def packed(t):
    return t[0].transpose(0, 1).contiguous()


def pages(t):   # [1, H, 256, d] as two pages of 128
    return torch.stack([t[0, :, :128], t[0, :, 128:]]).contiguous()


def calls():
    """The calls over 256 keys, as f(q, k, v, **more); inputs() has their tensors."""
    from attention_forward_blackwell_gb300 import binding
    cu_q, cu_k, lens, table = i32([0, 200]), i32([0, 256]), i32([256]), i32([[0, 1]])
    win = dict(causal=True, window=30, first=3)
    return {
        "prefill": lambda q, k, v, **m: binding.prefill(q, k, v, **win, **m),
        "prefill, plain": lambda q, k, v, **m: binding.prefill(q, k, v, **m),
        "prefill_varlen": lambda q, k, v, **m: binding.prefill_varlen(
            q, k, v, cu_q, cu_k, 200, 256, **win, **m),
        "prefill_varlen_paged": lambda q, k, v, **m: binding.prefill_varlen_paged(
            q, k, v, cu_q, 200, table, lens, **win, **m),
        "prefill_paged": lambda q, k, v, **m: binding.prefill_paged(q, k, v, table, lens, **m),
        "decode": lambda q, k, v, **m: binding.decode(q, k, v, **m),
        "decode_paged": lambda q, k, v, **m: binding.decode_paged(q, k, v, table, lens, **m),
    }


def inputs(name, seed):
    q, k, v = prompt(seed)
    if name == "prefill_varlen":
        return packed(q), packed(k), packed(v)
    if name == "prefill_varlen_paged":
        return packed(q), pages(k), pages(v)
    if name.startswith("decode"):
        q = q[:, :, :9].contiguous()
    if name.endswith("paged"):
        return q, pages(k), pages(v)
    return q, k, v


NAMES = ["prefill", "prefill, plain", "prefill_varlen", "prefill_varlen_paged", "prefill_paged",
         "decode", "decode_paged"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_may_be_dropped(name):
    """Outputs dropped while the call's stream has not begun: what the current
    stream allocates meanwhile stays as it is."""
    call, args = calls()[name], inputs(name, 1)
    side = torch.cuda.Stream()
    o, lse = call(*args)
    shapes = [(o.shape, o.dtype), (lse.shape, lse.dtype)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    o, lse = call(*args, stream=side)
    del o, lse
    held = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in shapes for _ in range(6)]
    torch.cuda.synchronize()
    check_device_error()
    assert all(bool((t == 7).all()) for t in held)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_leave_memory_in_use_alone(name):
    """The current stream is yet to read what was dropped just before the call."""
    call, args = calls()[name], inputs(name, 2)
    side = torch.cuda.Stream()
    o, lse = call(*args)
    kinds = [(o.shape, o.dtype), (lse.shape, lse.dtype)]
    del o, lse
    was = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in kinds for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    now = [t.clone() for t in was]
    del was
    call(*args, stream=side)
    torch.cuda.synchronize()
    check_device_error()
    assert all(bool((t == 7).all()) for t in now)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_while_they_are_read(name):
    """Outputs dropped before the current stream has read them, then another call."""
    call, args, others = calls()[name], inputs(name, 3), inputs(name, 4)
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(*args)]
    torch.cuda.synchronize()
    o, lse = call(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    got = [o.clone(), lse.clone()]
    del o, lse
    for _ in range(3):
        call(*others, stream=side)
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def strided(t):
    wide = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")
    wide[..., ::2] = t
    return wide[..., ::2]


def test_inputs_of_other_layouts_are_copied_on_the_calls_stream():
    """The current stream is busy: copies made there would come after the kernel."""
    from attention_forward_blackwell_gb300 import binding
    q, k, v = prompt(5)
    q, k, v = (t.expand(3, -1, -1, -1).contiguous() for t in (q, k, v))
    lens, sinks = i32([256, 40, 0]), torch.randn(4, device="cuda")
    win = dict(causal=True, window=30, first=3)
    want = binding.prefill(q, k, v, seqlens_k=lens, sinks=sinks, **win)
    wide = strided(lens), strided(sinks)
    binding.prefill(q, k, v, seqlens_k=wide[0], sinks=wide[1], **win)   # (every kernel loaded)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = binding.prefill(q, k, v, seqlens_k=wide[0], sinks=wide[1], stream=side, **win)
    side.synchronize()
    assert not torch.cuda.current_stream().query()   # still busy
    with torch.cuda.stream(side):
        got = [t.cpu() for t in got]
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


def serving():
    """The serving calls that make their outputs, as name -> f(**more)."""
    from attention_forward_blackwell_gb300 import binding
    q, k, v = prompt(6)
    q = q[:, :, :9].contiguous()
    kc, vc, table, lens = pages(k), pages(v), i32([[0, 1]]), i32([256])
    parents = torch.arange(-1, 8, dtype=torch.int32, device="cuda")[None]
    mask = binding.tree_mask(parents)
    refs, none = i32([1, 1]), torch.empty(0, dtype=torch.int32, device="cuda")
    return {
        "tree_mask": lambda **m: (binding.tree_mask(parents, **m),),
        "decode_tree": lambda **m: binding.decode_tree(q, k, v, mask, **m),
        "decode_tree_paged": lambda **m: binding.decode_tree_paged(q, kc, vc, table, lens, mask, **m),
        "decode": lambda **m: binding.decode(q, k, v, window=30, first=3, **m),
        "decode_paged": lambda **m: binding.decode_paged(q, kc, vc, table, lens, window=30, first=3, **m),
        "cache_fork": lambda **m: (binding.cache_fork(refs, table, lens, none, none, **m),),
        "cache_reserve": lambda **m: binding.cache_reserve(refs, table, lens, i32([0]), 128, **m),
    }


SERVING = ["tree_mask", "decode_tree", "decode_tree_paged", "decode", "decode_paged", "cache_fork",
           "cache_reserve"]


@pytest.mark.parametrize("name", SERVING)
def test_serving_outputs_come_from_the_calls_stream(name):
    """By the allocator's own account: each stream's memory is its own, and an
    output that the current stream may read is kept until it has."""
    call = serving()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for out in call(stream=side):
        owners = [s["stream"] for s in torch.cuda.memory_snapshot()
                  if s["address"] <= out.data_ptr() < s["address"] + s["total_size"]]
        assert owners == [side.cuda_stream]
    torch.cuda.synchronize()
    out = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    at = out.data_ptr()
    del out
    states = [b["state"] for s in torch.cuda.memory_snapshot() for b in s["blocks"]
              if b["address"] <= at < b["address"] + b["size"]]
    torch.cuda.synchronize()
    check_device_error()
    assert states == ["active_pending_free"]


@pytest.mark.parametrize("name", SERVING)
def test_serving_outputs_leave_memory_in_use_alone(name):
    """The current stream is yet to read what was dropped just before the call."""
    call = serving()[name]
    side = torch.cuda.Stream()
    kinds = [(t.shape, t.dtype) for t in call()]
    was = [torch.full(s, 7, dtype=t, device="cuda") for s, t in kinds for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    now = [t.clone() for t in was]
    del was
    call(stream=side)
    torch.cuda.synchronize()
    check_device_error()
    assert all(bool((t == 7).all()) for t in now)


def test_captured_calls_on_a_forked_stream():
    """A captured step whose calls run on a stream of their own, their outputs
    dropped inside the capture; replayed over other inputs."""
    from attention_forward_blackwell_gb300 import binding
    q, k, v = prompt(7)
    q = q[:, :, :9].contiguous()
    lens = i32([256])
    parents = torch.arange(-1, 8, dtype=torch.int32, device="cuda")[None].contiguous()
    win = dict(causal=True, window=30, first=3)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        mask = binding.tree_mask(parents, stream=side)
        a = binding.decode_tree(q, k, v, mask, seqlens_k=lens, stream=side)[0]
        b = binding.decode(q, k, v, seqlens_k=lens, stream=side, **win)[0]
        c = binding.prefill(q, k, v, seqlens_k=lens, stream=side, **win)[0]
        main.wait_stream(side)
        return a + b + c

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed, n in ((8, 256), (9, 100)):
        for t, new in zip((q, k, v), prompt(seed)):
            t.copy_(new[:, :, :t.shape[2]])
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
    torch.cuda.synchronize()
    check_device_error()


@pytest.mark.parametrize("name", NAMES + ["tree_mask", "decode_tree_paged"])
def test_calls_on_the_default_stream_from_another(name):
    """The call's stream is the legacy default one, the current one is not."""
    if name in NAMES:
        args = inputs(name, 10)
        call = lambda **m: calls()[name](*args, **m)
    else:
        call = serving()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(stream=torch.cuda.default_stream())
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        got = [t.clone() for t in got]
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
