"""Refusals of the rotation's and the 8-bit cache's calls on the host, before any launch, the table of
frequencies, and the plain forms that the GPU tests compare with (CPU only)."""
import ctypes
import math

import pytest
import torch

import q8_ref as ref

P16 = ctypes.c_void_p(1 << 12)
P_ODD = ctypes.c_void_p((1 << 12) + 8)
P_MIS4 = ctypes.c_void_p((1 << 12) + 2)
ST = (ctypes.c_longlong * 3)(64, 64, 64)
ST_ODD = (ctypes.c_longlong * 3)(64, 60, 64)


@pytest.fixture(scope="module")
def fa():
    from attention_forward_blackwell_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


def variants(ok):
    def call(fn, **kw):
        a = list(ok)
        for i, val in kw.items():
            a[int(i[1:])] = val
        return fn(*a)
    return call


def turn(fa, **kw):
    a = dict(freqs=1 << 12, rot=32, interleaved=0, factor=1.0, positions=None, position_stride=0, q=None,
             q_strides=None, q_out=None, hq=0)
    a.update(kw)
    return ctypes.byref(fa.Turn(**a))


def test_rope(fa):
    # q qs q_out qos hq k ks k_out kos hk B n d positions stride freqs rot interleaved inverse factor stream
    call = variants([P16, ST, P16, ST, 4, P16, ST, P16, ST, 2, 2, 3, 64, P16, 0, P16, 32, 0, 0, 1.0, None])
    fn = fa.lib().fa_rope
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 13, 15):
        assert call(fn, **{f"a{i}": None}) == 1
    for i in (4, 9, 10, 11, 14, 16):
        assert call(fn, **{f"a{i}": -1}) == 1
    assert call(fn, a10=70000) == 1 and call(fn, a4=65000, a9=65000) == 1
    assert call(fn, a16=80) == 1                                   # more than the row
    assert call(fn, a16=24) == 2 and call(fn, a12=40, a16=32) == 2 and call(fn, a12=0, a16=0) == 2
    for f in (0.0, -1.0, math.nan, math.inf):
        assert call(fn, a19=f) == 1
    assert call(fn, a0=P_ODD) == 3 and call(fn, a7=P_ODD) == 3 and call(fn, a15=P_ODD) == 3
    assert call(fn, a1=ST_ODD) == 3 and call(fn, a8=ST_ODD) == 3 and call(fn, a13=P_MIS4) == 3
    assert call(fn, a10=0) == 0 and call(fn, a11=0) == 0 and call(fn, a4=0, a9=0) == 0


def test_append_rope(fa):
    # k v pages hkv P d table max_pages lens B kn ks vn vs n n_new copies turn stream
    call = variants([P16, P16, 8, 2, 16, 64, P16, 4, P16, 2, P16, ST, P16, ST, 3, None, None, turn(fa), None])
    fn = fa.lib().fa_cache_append_rope
    for i in (0, 1, 6, 8, 10, 11, 12, 13, 17):
        assert call(fn, **{f"a{i}": None}) == 1
    for i in (2, 3, 4, 7, 9, 14):
        assert call(fn, **{f"a{i}": -1}) == 1
    assert call(fn, a9=70000) == 1 and call(fn, a4=0) == 1 and call(fn, a7=1 << 20, a4=1 << 12) == 1
    assert call(fn, a0=P_ODD) == 3 and call(fn, a10=P_ODD) == 3 and call(fn, a11=ST_ODD) == 3
    assert call(fn, a8=P_MIS4) == 3 and call(fn, a15=P_MIS4) == 3 and call(fn, a16=P_MIS4) == 3
    assert call(fn, a5=40) == 2
    assert call(fn, a17=turn(fa, rot=24)) == 2 and call(fn, a17=turn(fa, rot=80)) == 1
    assert call(fn, a17=turn(fa, freqs=None)) == 1 and call(fn, a17=turn(fa, factor=0.0)) == 1
    assert call(fn, a17=turn(fa, hq=-1)) == 1 and call(fn, a17=turn(fa, position_stride=-1)) == 1
    q = dict(hq=4, q=1 << 12, q_strides=ctypes.addressof(ST), q_out=1 << 12)
    for gone in ("q", "q_strides", "q_out"):
        assert call(fn, a17=turn(fa, **{**q, gone: None})) == 1
    assert call(fn, a17=turn(fa, **{**q, "q_out": (1 << 12) + 8})) == 3
    assert call(fn, a3=0, a17=turn(fa, **q)) == 1                  # queries come beside keys
    assert call(fn, a9=0) == 0 and call(fn, a14=0) == 0 and call(fn, a3=0) == 0


def test_append_q8(fa):
    # k v ksc vsc pages hkv P block d table max_pages lens B kn ks vn vs n n_new copies turn stream
    call = variants([P16, P16, P16, P16, 8, 2, 16, 8, 64, P16, 4, P16, 2, P16, ST, P16, ST, 3, None, None, None, None])
    fn = fa.lib().fa_cache_append_q8
    for i in (0, 1, 2, 3, 9, 11, 13, 14, 15, 16):
        assert call(fn, **{f"a{i}": None}) == 1
    for i in (4, 5, 6, 7, 10, 12, 17):
        assert call(fn, **{f"a{i}": -1}) == 1
    assert call(fn, a7=0) == 1 and call(fn, a7=5) == 1 and call(fn, a12=70000) == 1
    assert call(fn, a10=1 << 20, a6=1 << 12, a7=1 << 12) == 1
    assert call(fn, a8=40) == 2 and call(fn, a8=0) == 2
    assert call(fn, a1=P_ODD) == 3 and call(fn, a3=P_MIS4) == 3 and call(fn, a13=P_ODD) == 3
    assert call(fn, a14=ST_ODD) == 3 and call(fn, a11=P_MIS4) == 3
    assert call(fn, a20=turn(fa, rot=24)) == 2 and call(fn, a20=turn(fa, freqs=None)) == 1
    assert call(fn, a17=1 << 30) == 1
    assert call(fn, a12=0) == 0 and call(fn, a17=0) == 0 and call(fn, a4=0) == 0


def test_read_q8(fa):
    # k v ksc vsc pages hkv P block d table max_pages cu B max_seqlen total k_out v_out stream
    call = variants([P16, P16, P16, P16, 8, 2, 16, 8, 64, P16, 4, P16, 2, 9, 9, P16, P16, None])
    fn = fa.lib().fa_cache_read_q8
    for i in (0, 1, 2, 3, 9, 11, 15, 16):
        assert call(fn, **{f"a{i}": None}) == 1
    for i in (4, 5, 6, 7, 10, 12, 13, 14):
        assert call(fn, **{f"a{i}": -1}) == 1
    assert call(fn, a13=0) == 1 and call(fn, a7=3) == 1 and call(fn, a8=40) == 2
    assert call(fn, a15=P_ODD) == 3 and call(fn, a11=P_MIS4) == 3
    assert call(fn, a12=0) == 0 and call(fn, a14=0) == 0 and call(fn, a5=0) == 0


def test_decode_q8(fa):
    # q k v ksc vsc o lse B hq hkv n lens table max_pages P pages block d scale causal window first sinks stream
    call = variants([P16, P16, P16, P16, P16, P16, P16, 1, 4, 2, 1, P16, P16, 4, 16, 9, 8, 64, 0.1, 0, 0, 0, None, None])
    fn = fa.lib().fa_fwd_decode_paged_q8
    for i in (0, 1, 2, 3, 4, 5, 6, 11, 12):
        assert call(fn, **{f"a{i}": None}) == 1
    for i in (7, 8, 9, 10, 13, 14, 15, 16, 21):
        assert call(fn, **{f"a{i}": -1}) == 1
    assert call(fn, a9=3) == 1 and call(fn, a10=17) == 1 and call(fn, a16=5) == 1 and call(fn, a18=0.0) == 1
    assert call(fn, a13=1 << 20, a14=1 << 12) == 1
    assert call(fn, a15=1 << 30) == 1                              # planes of the cache past 2^31
    assert call(fn, a17=96) == 2 and call(fn, a17=512) == 2
    assert call(fn, a0=P_ODD) == 3 and call(fn, a2=P_ODD) == 3 and call(fn, a3=P_MIS4) == 3
    assert call(fn, a22=P_MIS4) == 3 and call(fn, a11=P_MIS4) == 3
    assert call(fn, a7=0) == 0 and call(fn, a10=0) == 0


def test_binding_refuses_cpu_tensors(fa):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(3, 2, 16, 64).to(ref.F8), torch.ones(3, 2, 2)
    t, lens, f = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(16, dtype=torch.int64)
    for call in (lambda: fa.rope(x, None, t[0], f), lambda: fa.cache_append_rope(x, x, t, lens, x, x, f),
                 lambda: fa.cache_append_q8(c, c, s, s, t, lens, x, x), lambda: fa.cache_read_q8(c, c, s, s, t, lens, 1, 1),
                 lambda: fa.decode_paged_q8(x, c, c, s, s, t, lens)):
        with pytest.raises(ValueError):
            call()


def test_frequencies(fa):
    w, factor = fa.rope_inv_freq(8)
    assert factor == 1.0 and torch.allclose(w, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    turns = fa.rope_freqs(w, device="cpu")
    assert turns.dtype == torch.int64
    for f, x in zip(turns.tolist(), w.tolist()):
        assert abs(f / 2.0 ** 64 * 2 * math.pi - x) <= 1e-15 * x
    assert torch.equal(fa.rope_inv_freq(8, method="linear", stretch=4.0)[0], w / 4)
    ntk = fa.rope_inv_freq(8, method="ntk", stretch=4.0)[0]
    assert ntk[0] == 1.0 and abs(ntk[-1].item() - 0.001 / 4) < 1e-12   # the slowest pair is stretched whole
    yarn, factor = fa.rope_inv_freq(64, method="yarn", stretch=4.0, original=4096)
    plain = fa.rope_inv_freq(64)[0]
    assert yarn[0] == plain[0] and abs(yarn[-1] / plain[-1] - 0.25) < 1e-12 and factor > 1.0
    assert torch.all(yarn <= plain + 1e-18) and torch.all(yarn >= plain / 4 - 1e-18)
    assert fa.rope_inv_freq(64, method="yarn", stretch=1.0, original=4096)[1] == 1.0
    # angles past half a turn wrap
    assert fa.rope_freqs([1.5 * math.pi, -0.5 * math.pi], device="cpu").tolist() == [-2 ** 62, -2 ** 62]
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, method="other"), dict(rot=8, method="yarn", stretch=2.0),
                dict(rot=2, method="ntk"), dict(rot=8, base=-1.0)):
        with pytest.raises(ValueError):
            fa.rope_inv_freq(**bad)
    with pytest.raises(ValueError):
        fa.rope_freqs([math.inf])


def test_plain_forms():
    """The definitions that the GPU tests compare with, on values worked out by hand."""
    x = torch.tensor([[3.0, 0.0, 0.0, 4.0, 9.0]])
    y = ref.turn64(x, torch.tensor([1]), [math.pi / 2, math.pi])
    assert torch.allclose(y, torch.tensor([[0.0, 0.0, 3.0, -4.0, 9.0]], dtype=torch.float64), atol=1e-12)
    y = ref.turn64(x, torch.tensor([1]), [math.pi / 2, math.pi], interleaved=True)
    assert torch.allclose(y, torch.tensor([[0.0, 3.0, 0.0, -4.0, 9.0]], dtype=torch.float64), atol=1e-12)
    back = ref.turn64(y, torch.tensor([1]), [math.pi / 2, math.pi], interleaved=True, inverse=True)
    assert torch.allclose(back, x.double(), atol=1e-12)
    codes = torch.arange(256, dtype=torch.uint8).view(ref.F8).double()
    codes = codes[codes.isfinite()].sort().values.unique()
    assert torch.equal(ref.round8(codes), codes)
    mids = (codes[1:] + codes[:-1]) / 2
    got = ref.round8(mids).float().to(ref.F8).view(torch.uint8)
    assert torch.all(got % 2 == 0)                                 # ties go to even codes
    assert torch.equal(ref.round8(mids), mids.float().to(ref.F8).double())
    assert ref.scale_for(448.0) == 1.0 and ref.scale_for(448.1) == 2.0 and ref.scale_for(224.0) == 0.5
    assert ref.scale_for(0.0) == 2.0 ** -54 and ref.scale_for(1e30) == 2.0 ** 54
    assert ref.reach64(torch.tensor([[3.0, 4.0, 4.5]]), 2, 1.0, True) == 5.0
    assert ref.reach64(torch.tensor([[3.0, 4.0, 5.5]]), 2, 1.0, False) == 5.5
