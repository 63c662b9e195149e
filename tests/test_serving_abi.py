"""Refusals of the serving operators (token trees, a window with first tokens,
cache pages): on the host, before any launch (CPU only)."""
import ctypes

import pytest
import torch

P16 = ctypes.c_void_p(1 << 12)
P_ODD = ctypes.c_void_p((1 << 12) + 8)
P_MIS4 = ctypes.c_void_p((1 << 12) + 2)


@pytest.fixture(scope="module")
def lib():
    from attention_forward_blackwell_gb300 import binding, build
    build.build()
    return binding.lib()


def variants(ok):
    def call(fn, **kw):
        a = list(ok)
        for i, val in kw.items():
            a[int(i[1:])] = val
        return fn(*a)
    return call


def test_tree(lib):
    # q k v o lse B hq hkv nodes sk lens mask shared tree_lens d scale sinks stream
    call = variants([P16, P16, P16, P16, P16, 1, 4, 2, 8, 64, None, P16, 0, None, 128, 0.1, None, None])
    fn = lib.fa_fwd_decode_tree
    assert call(fn, a11=None) == 1           # no mask
    assert call(fn, a11=P_MIS4) == 3
    assert call(fn, a13=P_MIS4) == 3
    assert call(fn, a16=P_MIS4) == 3
    assert call(fn, a8=1025) == 1            # more nodes than a tree may have
    assert call(fn, a8=-1) == 1
    assert call(fn, a6=3) == 1               # hq % hkv
    assert call(fn, a14=96) == 2
    assert call(fn, a15=0.0) == 1
    assert call(fn, a0=P_ODD) == 3
    assert call(fn, a5=4096, a6=512, a8=1024) == 1   # q of 2^31 elements
    assert call(fn, a8=0) == 0               # nothing to compute
    assert call(fn, a5=0) == 0


def test_tree_paged(lib):
    # q k v o lse B hq hkv nodes lens table max_pages P pages mask shared tree_lens d scale sinks st
    call = variants([P16, P16, P16, P16, P16, 1, 4, 2, 8, P16, P16, 4, 16, 9, P16, 0, None, 128, 0.1,
                     None, None])
    fn = lib.fa_fwd_decode_tree_paged
    assert call(fn, a9=None) == 1
    assert call(fn, a10=None) == 1
    assert call(fn, a12=0) == 1
    assert call(fn, a13=0) == 1
    assert call(fn, a11=1 << 20, a12=1 << 12) == 1
    assert call(fn, a14=None) == 1
    assert call(fn, a8=0) == 0


def test_first(lib):
    ok = [P16, P16, P16, P16, P16, 1, 2, 1, 4, 64, None, 64, 1.0, 1, 16, 4, None, None]
    for fn in (lib.fa_fwd_prefill_first, lib.fa_fwd_decode_first):
        call = variants(ok)
        assert call(fn, a15=-1) == 1         # first < 0
        assert call(fn, a7=3) == 1
        assert call(fn, a16=P_MIS4) == 3
        assert call(fn, a5=0) == 0
    assert variants(ok)(lib.fa_fwd_decode_first, a8=17) == 1
    call = variants([P16, P16, P16, P16, P16, 1, 2, 1, 4, P16, P16, 2, 16, 4, 64, 1.0, 1, 16, 4, None,
                     None])
    assert call(lib.fa_fwd_decode_paged_first, a18=-1) == 1
    assert call(lib.fa_fwd_decode_paged_first, a10=None) == 1
    call = variants([P16, P16, P16, P16, P16, P16, P16, 2, 8, 8, 8, 8, 2, 1, 64, 1.0, 1, 4, -1, None,
                     None])
    assert call(lib.fa_fwd_prefill_varlen_first) == 1
    call = variants([P16, P16, P16, P16, P16, P16, P16, P16, 2, 128, 4, 1, 8, 8, 2, 1, 64, 1.0, 1, 4,
                     -1, None, None])
    assert call(lib.fa_fwd_prefill_varlen_paged_first) == 1
    assert call(lib.fa_fwd_prefill_varlen_paged_first, a20=4, a9=100) == 2


def test_cache(lib):
    # refs pages table max_pages lens B src dst n status stream
    call = variants([P16, 8, P16, 4, P16, 2, P16, P16, 1, P16, None])
    fn = lib.fa_cache_fork
    assert call(fn, a0=None) == 1 and call(fn, a2=None) == 1 and call(fn, a4=None) == 1
    assert call(fn, a9=None) == 1 and call(fn, a6=None) == 1 and call(fn, a8=-1) == 1
    assert call(fn, a1=-1) == 1 and call(fn, a3=-1) == 1 and call(fn, a5=-1) == 1
    assert call(fn, a0=P_MIS4) == 3 and call(fn, a7=P_MIS4) == 3
    # refs pages table max_pages lens B extra P copies status stream
    call = variants([P16, 8, P16, 4, P16, 2, P16, 16, P16, P16, None])
    fn = lib.fa_cache_reserve
    assert call(fn, a6=None) == 1 and call(fn, a7=0) == 1 and call(fn, a8=None) == 1
    assert call(fn, a3=1 << 20, a7=1 << 12) == 1 and call(fn, a8=P_MIS4) == 3
    # refs pages table max_pages lens B rows n stream
    call = variants([P16, 8, P16, 4, P16, 2, P16, 1, None])
    fn = lib.fa_cache_free
    assert call(fn, a6=None) == 1 and call(fn, a7=-1) == 1 and call(fn, a6=P_MIS4) == 3
    assert call(fn, a7=0) == 0 and call(fn, a5=0) == 0
    # k v pages hkv P d table max_pages lens B kn ks vn vs n n_new copies stream
    st = (ctypes.c_longlong * 3)(64, 64, 64)
    call = variants([P16, P16, 8, 2, 16, 64, P16, 4, P16, 2, P16, st, P16, st, 3, None, None, None])
    fn = lib.fa_cache_append
    assert call(fn, a0=None) == 1 and call(fn, a6=None) == 1 and call(fn, a8=None) == 1
    assert call(fn, a10=None) == 1 and call(fn, a11=None) == 1 and call(fn, a14=-1) == 1
    assert call(fn, a5=60) == 2 and call(fn, a5=0) == 2
    assert call(fn, a0=P_ODD) == 3 and call(fn, a10=P_ODD) == 3 and call(fn, a15=P_MIS4) == 3
    assert call(fn, a11=(ctypes.c_longlong * 3)(64, 64, 63)) == 3
    assert call(fn, a9=70000) == 1 and call(fn, a3=70000) == 1
    assert call(fn, a14=0) == 0 and call(fn, a9=0) == 0 and call(fn, a2=0) == 0
    # k v pages hkv P d copies n stream
    call = variants([P16, P16, 8, 2, 16, 64, P16, 1, None])
    fn = lib.fa_cache_copy
    assert call(fn, a6=None) == 1 and call(fn, a6=P_MIS4) == 3 and call(fn, a7=-1) == 1
    assert call(fn, a7=0) == 0 and call(fn, a5=12) == 2
    # k v pages hkv P d table max_pages start B keep stride n_keep stream
    call = variants([P16, P16, 8, 2, 16, 64, P16, 4, P16, 2, P16, 3, P16, None])
    fn = lib.fa_cache_compact
    assert call(fn, a10=None) == 1 and call(fn, a12=None) == 1 and call(fn, a11=-1) == 1
    assert call(fn, a10=P_MIS4) == 3 and call(fn, a11=0) == 0 and call(fn, a9=0) == 0
    # parents mask B nodes stream
    call = variants([P16, P16, 2, 8, None])
    fn = lib.fa_tree_mask
    assert call(fn, a0=None) == 1 and call(fn, a1=P_MIS4) == 3 and call(fn, a3=1025) == 1
    assert call(fn, a2=0) == 0 and call(fn, a3=0) == 0


def test_binding_refuses_cpu_tensors():
    from attention_forward_blackwell_gb300 import binding
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: binding.decode_tree(q, q, q, torch.zeros(1, 4, 1, dtype=torch.int32)),
                 lambda: binding.decode_tree_paged(q, q, q, i, one, torch.zeros(1, 4, 1, dtype=torch.int32)),
                 lambda: binding.tree_mask(i),
                 lambda: binding.cache_fork(one, i, one, one, one),
                 lambda: binding.cache_reserve(one, i, one, one, 16),
                 lambda: binding.cache_free(one, i, one, one),
                 lambda: binding.cache_append(q, q, i, one, q, q),
                 lambda: binding.cache_copy(q, q, i),
                 lambda: binding.cache_compact(q, q, i, one, i, one)):
        with pytest.raises(ValueError):
            call()


def test_plain_page_operators():
    """The definition the GPU tests compare with, on a case worked out by hand."""
    import serving_ref as ref
    pool = ref.Pool(torch.tensor([1, 0, 1, 0, 0]), torch.tensor([[2, 0, -1], [-1] * 3, [-1] * 3]),
                    torch.tensor([6, 0, 0]))
    assert pool.fork([0, 0], [1, 2]) == 0
    assert pool.refs == [3, 0, 3, 0, 0] and pool.lens == [6, 6, 6]
    copies, status = pool.reserve([-1, 1, 3], 4)
    assert status == 0 and copies == [[-1, -1, 0], [0, 1, 2], [0, 3, 2]]
    assert pool.table == [[2, 0, -1], [2, 1, -1], [2, 3, 4]] and pool.refs == [1, 1, 3, 1, 1]
    assert pool.reserve([0, 4, 0], 4) == ([[-1, -1, 0]] * 3, 1)
    pool.free([1, 1])
    assert pool.refs == [1, 0, 2, 1, 1] and pool.lens[1] == 0


def test_pages_need_their_counts(lib):
    """Counts may be absent only where there are no pages, whatever the rows: the
    kernel that reserves looks for free pages before it knows what is needed."""
    # refs pages table max_pages lens B extra P copies status stream
    call = variants([None, 8, None, 4, None, 0, None, 16, None, P16, None])
    assert call(lib.fa_cache_reserve) == 1
    # refs pages table max_pages lens B src dst n status stream
    call = variants([None, 8, None, 4, None, 0, None, None, 0, P16, None])
    assert call(lib.fa_cache_fork) == 1
    # refs pages table max_pages lens B rows n stream
    call = variants([None, 8, None, 4, None, 0, None, 0, None])
    assert call(lib.fa_cache_free) == 1
