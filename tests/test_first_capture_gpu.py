"""A process's first call of the library made while its stream is captured: a program that loads its model and
captures the step at once (GPU)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, torch
from attention_forward_blackwell_gb300 import binding as fa
F8, bf = torch.float8_e4m3fn, torch.bfloat16
g = torch.Generator().manual_seed(1)
randn = lambda *s: torch.randn(*s, generator=g).cuda()
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q, k, v = randn(2, 8, 2, 128).to(bf), randn(60, 2, 16, 128).to(bf), randn(60, 2, 16, 128).to(bf)
k8, v8, s = k.to(F8), v.to(F8), torch.ones(60, 2, 1, device="cuda")
table, lens = torch.randperm(60, generator=g).to(torch.int32).view(2, 30).cuda(), i32([400, 33])
wide = torch.cat([table] * 40, 1).contiguous()
kd, vd = randn(2, 2, 300, 128).to(bf), randn(2, 2, 300, 128).to(bf)
mask = i32([[1], [3]])
calls = dict(
    decode=lambda: fa.decode(q, kd, vd),
    decode_paged=lambda: fa.decode_paged(q, k, v, table, lens, causal=True),
    decode_tree=lambda: fa.decode_tree_paged(q, k, v, table, lens, mask),
    prefill=lambda: fa.prefill(q, kd, vd, causal=True),
    decode_paged_q8=lambda: fa.decode_paged_q8(q, k8, v8, s, s, table, lens, causal=True),
    decode_paged_q8_line=lambda: fa.decode_paged_q8(q, k8, v8, s, s, wide, lens, causal=True))
call = calls[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    o, lse = call()
o.fill_(7.0)
graph.replay()
torch.cuda.synchronize()
got = o.clone(), lse.clone()
want = call()
torch.cuda.synchronize()
assert fa.get_device_error() == fa.FA_OK
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""


@pytest.mark.parametrize("name", ["decode", "decode_paged", "decode_tree", "prefill", "decode_paged_q8",
                                  "decode_paged_q8_line"])
def test_first_call_captured(name):
    r = subprocess.run([sys.executable, "-c", PROGRAM, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
