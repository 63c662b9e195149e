"""Every tensor of an attention call lies on the current device: a launch that
reads another device's memory, or the host's, is refused before it is made (CPU
only: tensors without memory, a library that only notes that it was called)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from attention_forward_blackwell_gb300 import binding

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32
DENSE = dict(q=((1, 4, 8, 64), BF), k=((1, 2, 32, 64), BF), v=((1, 2, 32, 64), BF))
PAGED = dict(q=((1, 4, 8, 64), BF), k_cache=((3, 2, 128, 64), BF), v_cache=((3, 2, 128, 64), BF),
             block_table=((1, 2), I32), seqlens_k=((1,), I32))
OUT = dict(out=((1, 4, 8, 64), BF), lse=((1, 4, 8), F32))
PACKED_OUT = dict(out=((8, 4, 64), BF), lse=((4, 8), F32))
SINKS = dict(sinks=((4,), F32))
CALLS = {
    "prefill": (dict(**DENSE, seqlens_k=((1,), I32), **OUT, **SINKS), [dict(), dict(window=3, first=1)]),
    "decode": (dict(**DENSE, seqlens_k=((1,), I32), **OUT, **SINKS), [dict()]),
    "prefill_paged": (dict(**PAGED, **OUT), [dict()]),
    "decode_paged": (dict(**PAGED, **OUT), [dict()]),
    "prefill_varlen": (dict(q=((8, 4, 64), BF), k=((32, 2, 64), BF), v=((32, 2, 64), BF),
                            cu_seqlens_q=((2,), I32), cu_seqlens_k=((2,), I32), **PACKED_OUT, **SINKS),
                       [dict(max_seqlen_q=8, max_seqlen_k=32),
                        dict(max_seqlen_q=8, max_seqlen_k=32, window=3, first=1)]),
    "prefill_varlen_paged": (dict(q=((8, 4, 64), BF), k_cache=((3, 2, 128, 64), BF),
                                  v_cache=((3, 2, 128, 64), BF), cu_seqlens_q=((2,), I32),
                                  block_table=((1, 2), I32), seqlens_k=((1,), I32), **PACKED_OUT,
                                  **SINKS),
                             [dict(max_seqlen_q=8), dict(max_seqlen_q=8, window=3, first=1)]),
}
CASES = [(call, i, name) for call, (tensors, more) in CALLS.items() for i in range(len(more))
         for name in (None, *tensors)]


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


@pytest.mark.parametrize("where", ["cuda:1", "cpu"])
@pytest.mark.parametrize("call,i,name", CASES, ids=[f"{c}-{i}-{n}" for c, i, n in CASES])
def test_tensors_elsewhere_are_refused(call, i, name, where, monkeypatch):
    library = Library()
    monkeypatch.setattr(binding, "_lib", library)
    monkeypatch.setattr(binding, "_ptr", lambda t: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    tensors, more = CALLS[call]
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device=where if n == name else "cuda:0")
                for n, (shape, dtype) in tensors.items()}
        if name is None:   # (all where they belong)
            getattr(binding, call)(**args, **more[i])
            assert library.calls == 1
        else:
            with pytest.raises(ValueError):
                getattr(binding, call)(**args, **more[i])
            assert library.calls == 0
