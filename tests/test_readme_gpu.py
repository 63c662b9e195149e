"""The serving step of the README, run as it is written, against plain attention
over the keys that each sequence then has."""
import os
import re

import pytest
import torch

import serving_ref as ref
from gpu_parity import check_device_error, free_cuda, to_pages

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_serving_step():
    from attention_forward_blackwell_gb300 import binding
    with open(README) as f:
        steps = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "cache_reserve" in c]
    assert len(steps) == 1
    B, Hq, Hkv, d, T, P = 3, 4, 2, 64, 6, 16
    lens, nodes = [4500, 31, 0], [6, 4, 1]              # (the window of 4,096 cuts the first)
    parents = [[-1, 0, 0, 1, 1, 4], [-1, 0, 1, 0, 3, 4], [-1] * T]
    paths = [[0, 1, 4, 5], [0, 3], []]                  # accepted nodes, root first
    g = torch.Generator().manual_seed(12)
    randn = lambda *s: torch.randn(*s, generator=g).bfloat16()
    k, v = randn(B, Hkv, max(lens), d), randn(B, Hkv, max(lens), d)
    q, k_new, v_new = randn(B, Hq, T, d), randn(B, Hkv, T, d), randn(B, Hkv, T, d)
    q1, k1, v1 = randn(B, Hq, 1, d), randn(B, Hkv, 1, d), randn(B, Hkv, 1, d)
    kc, vc, pages, _ = to_pages(k.cuda(), v.cuda(), lens, P, seed=3, spare=8)
    table = torch.full((B, pages.shape[1] + 2), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(kc.shape[0], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        used = pages[b, :-(-n // P)]
        table[b, :used.numel()] = used
        refs[used.long()] = 1
    keep = torch.zeros(B, T, dtype=torch.int32)
    for b, x in enumerate(paths):
        keep[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    names = dict(torch=torch, binding=binding, refs=refs, table=table, lens=i32(lens), page_size=P,
                 n_new=i32(nodes), k_cache=kc, v_cache=vc, k_new=k_new.cuda(), v_new=v_new.cuda(),
                 parents=i32(parents), q=q.cuda(), keep=keep.cuda(), n_keep=i32([len(x) for x in paths]),
                 q1=q1.cuda(), k1=k1.cuda(), v1=v1.cuda())
    exec(steps[0], names)
    torch.cuda.synchronize()
    check_device_error()
    assert names["status"].item() == 0
    assert names["lens"].tolist() == [n + len(x) + 1 for n, x in zip(lens, paths)]
    bits = ref.ancestors(torch.tensor(parents, dtype=torch.int32))
    for b in range(B):
        n, t, path = lens[b], nodes[b], paths[b]
        kk = torch.cat([k[b, :, :n], k_new[b, :, :t]], 1)[None]
        vv = torch.cat([v[b, :, :n], v_new[b, :, :t]], 1)[None]
        want = ref.attention64(q[b:b + 1], kk, vv, ref.tree_seen(bits[b:b + 1], [n + t], [t], n + t),
                               d ** -0.5)
        ref.check(names["o"][b:b + 1], names["lse"][b:b + 1], want, f"tree {b}",
                  torch.arange(T)[None] < t)
        kk = torch.cat([k[b, :, :n], k_new[b][:, path], k1[b]], 1)[None]
        vv = torch.cat([v[b, :, :n], v_new[b][:, path], v1[b]], 1)[None]
        m = kk.shape[2]
        want = ref.attention64(q1[b:b + 1], kk, vv, ref.window_seen(1, [m], m, 4096, 4, True), d ** -0.5)
        ref.check(names["o1"][b:b + 1], names["lse1"][b:b + 1], want, f"next token {b}")
