"""Where the memory of a call on another stream than the current one comes from
(CPU only: tensors without memory, streams that are names, a library that does
nothing)."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

from attention_forward_blackwell_gb300 import binding
from test_binding_device import CALLS, Library

CASES = [(call, i) for call, (tensors, more) in CALLS.items() for i in range(len(more))]
CURRENT, OTHER = 11, 22


class Side:
    cuda_stream = OTHER


class Allocations(TorchDispatchMode):
    """Notes every new tensor with the stream that was current."""

    def __init__(self, at):
        super().__init__()
        self.at, self.outputs, self.copies = at, [], []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "empty" in func.__name__:
            self.outputs.append(self.at[-1])
        elif "clone" in func.__name__:
            self.copies.append(self.at[-1])
        return func(*args, **(kwargs or {}))


@pytest.fixture
def at(monkeypatch):
    """The current stream: the last of the list; torch and the library stand still."""
    streams = [CURRENT]

    @contextlib.contextmanager
    def within(stream):
        streams.append(getattr(stream, "cuda_stream", stream))
        yield
        streams.pop()

    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_ptr", lambda t: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: streams[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: streams[-1])
    monkeypatch.setattr(torch.cuda, "stream", within)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    return streams


@pytest.mark.parametrize("stream", [None, Side], ids=["current", "other"])
@pytest.mark.parametrize("call,i", CASES)
def test_outputs_come_from_the_calls_stream(call, i, stream, at, monkeypatch):
    used = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append(s))
    tensors, more = CALLS[call]
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device="cuda:0")
                for n, (shape, dtype) in tensors.items() if n not in ("out", "lse")}
        with Allocations(at) as made:
            getattr(binding, call)(**args, **more[i], stream=stream)
    if stream is None:
        assert made.outputs == [CURRENT] * 2 and used == []
    else:   # (and kept until what the current stream does with them is done)
        assert made.outputs == [OTHER] * 2 and used == [CURRENT] * 2
    assert made.copies == [] and at == [CURRENT]


# inputs that each call takes in other layouts
LAID_OUT = {"prefill": ["seqlens_k", "sinks"], "decode": ["seqlens_k", "sinks"],
            "prefill_paged": ["q", "k_cache", "v_cache", "block_table", "seqlens_k"],
            "decode_paged": ["q", "k_cache", "v_cache", "block_table", "seqlens_k"],
            "prefill_varlen": ["q", "k", "v", "cu_seqlens_q", "cu_seqlens_k", "sinks"],
            "prefill_varlen_paged": ["q", "k_cache", "v_cache", "cu_seqlens_q", "seqlens_k",
                                     "block_table", "sinks"]}


@pytest.mark.parametrize("stream", [None, Side], ids=["current", "other"])
@pytest.mark.parametrize("call,i", CASES)
def test_inputs_are_laid_out_on_the_calls_stream(call, i, stream, at, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    tensors, more = CALLS[call]
    with FakeTensorMode():
        args, copied = {}, 0
        for n, (shape, dtype) in tensors.items():
            args[n] = torch.empty(shape, dtype=dtype, device="cuda:0")
            if n in LAID_OUT[call] and args[n].numel() > 1:   # every other element of a wider one
                args[n] = torch.empty((*shape[:-1], 2 * shape[-1]), dtype=dtype, device="cuda:0")[..., ::2]
                copied += 1
        with Allocations(at) as made:
            getattr(binding, call)(**args, **more[i], stream=stream)
    assert made.copies == [CURRENT if stream is None else OTHER] * copied and copied > 0
    assert at == [CURRENT]
