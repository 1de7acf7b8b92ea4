"""The 64-bit references themselves: the gradient's formulas against autograd, the cache's number
format against torch's own conversion, and refusals of the calls on a cache, all on the CPU."""
import ctypes

import pytest
import torch

import long_context_prefill_block_b200 as moba
import reference64 as ref


def test_gradient_formulas_are_autograds():
    g = torch.Generator().manual_seed(1)
    cu = [0, 9, 10, 30]
    q = torch.randn(30, 4, 8, generator=g, dtype=torch.float64, requires_grad=True)
    k, v = (torch.randn(30, 2, 8, generator=g, dtype=torch.float64, requires_grad=True)
            for _ in range(2))
    do = torch.randn(30, 4, 8, generator=g, dtype=torch.float64)
    res = []
    for a, e in zip(cu, cu[1:]):
        kk, vv = (x[a:e].repeat_interleave(2, 1) for x in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[a:e], kk) / 8 ** 0.5
        s = s.masked_fill(torch.ones(e - a, e - a, dtype=torch.bool).triu(1), float("-inf"))
        res.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv))
    torch.cat(res).backward(do)
    with torch.no_grad():
        out, lse = ref.dense_forward(q, k, v, cu)
        assert torch.allclose(out, torch.cat(res), atol=1e-12)
        for x, t in zip(ref.dense_backward(q, k, v, cu, out, lse, do), (q, k, v)):
            assert torch.allclose(x, t.grad, atol=1e-12)


def test_quantiser_rounds_as_the_type_does():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(500, 64, generator=g) * torch.exp2(torch.randint(-40, 40, (500, 1), generator=g))
    x[0] = 0
    x[1] = 448.0 * 2 ** 5
    x[2] = torch.nextafter(torch.tensor(448.0 * 2 ** 5), torch.tensor(1e9))
    c, e, fine = ref.quantise(x)
    assert fine.all() and e[0] == -127 and e[1] == 5 and e[2] == 6
    y = torch.ldexp(x, -e[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(y.to(torch.float64), c)
    assert torch.equal(ref.stored_value(y, (e + 127).to(torch.uint8)),
                       c * torch.exp2(e.double())[:, None])


def _cache(pages=4, heads=2, page=16, d=64):
    return moba.MobaCache(*(torch.zeros(pages, heads, page, d, dtype=torch.uint8).view(
        torch.float8_e4m3fn) for _ in range(2)), *(torch.zeros(
            pages, heads, page, dtype=torch.uint8).view(torch.float8_e8m0fnu) for _ in range(2)))


TABLE = torch.zeros(3, 2, dtype=torch.int32)
LENS = torch.zeros(3, dtype=torch.int32)
CU = torch.zeros(4, dtype=torch.int32)
ROWS = torch.zeros(5, 2, 64)


@pytest.mark.parametrize("change,error", [
    (dict(cache=_cache(page=24)), ValueError), (dict(cache=_cache(page=8)), ValueError),
    (dict(cache=_cache(heads=3)), ValueError), (dict(cache=_cache(d=128)), ValueError),
    (dict(cache=_cache()._replace(k=torch.zeros(4, 2, 16, 64))), TypeError),
    (dict(cache=_cache()._replace(v=_cache(pages=5).v)), ValueError),
    (dict(cache=_cache()._replace(k_scale=_cache(page=32).k_scale)), ValueError),
    (dict(cache=_cache()._replace(v_scale=torch.zeros(4, 2, 16))), TypeError),
    (dict(page_table=TABLE.long()), ValueError), (dict(page_table=TABLE[0]), ValueError),
    (dict(seqlens=LENS[:2]), ValueError), (dict(seqlens=LENS.long()), ValueError),
    (dict(cu=CU[:3]), ValueError), (dict(cu=CU.long()), ValueError),
    (dict(), ValueError),  # sound, but not on a GPU
])
def test_cache_calls_refuse_what_does_not_fit(change, error):
    a = dict(cache=_cache(), page_table=TABLE, seqlens=LENS, cu=CU)
    a.update(change)
    with pytest.raises(error):
        moba.moba_cache_write(a["cache"], ROWS, ROWS, a["page_table"], a["seqlens"], a["cu"])
    if a["cache"].k.shape[1] == 2 and a["cache"].k.shape[3] == 64:
        with pytest.raises(error):
            moba.moba_cache_read(a["cache"], a["page_table"], a["seqlens"], a["cu"], 5)
    with pytest.raises(error):
        moba.moba_decode_cache(torch.zeros(5, 4, 64), a["cache"], a["page_table"], a["seqlens"],
                               a["cu"], torch.zeros(3, 2, 2, 64), 16, 2)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(5, 3, 64)), dict(q=torch.zeros(5, 4, 128)), dict(q=torch.zeros(5, 4)),
    dict(kbar=torch.zeros(3, 2, 1, 64)), dict(kbar=torch.zeros(2, 2, 2, 64)),
    dict(kbar=torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16)), dict(max_seqlen=16),
    dict(max_seqlen=33), dict(out=torch.zeros(5, 4, 128)), dict(block=0)])
def test_decode_refuses_what_does_not_fit(kw):
    q, kbar = kw.get("q", torch.zeros(5, 4, 64)), kw.get("kbar", torch.zeros(3, 2, 2, 64))
    with pytest.raises(ValueError):
        moba.moba_decode_cache(q, _cache(), TABLE, LENS, CU, kbar, kw.get("block", 16), 2,
                               max_seqlen=kw.get("max_seqlen"), out=kw.get("out"))


def test_alloc_refuses_odd_pages():
    for page in (0, 8, 24, 131072):
        with pytest.raises(ValueError):
            moba.moba_cache_alloc(4, page, 2, 64, device="cpu")
    c = moba.moba_cache_alloc(4, 32, 2, 64, device="cpu")
    assert c.k.shape == (4, 2, 32, 64) and c.k_scale.shape == (4, 2, 32)
    assert c.k.dtype == torch.float8_e4m3fn and c.v_scale.dtype == torch.float8_e8m0fnu


def test_dense_backward_refuses_what_does_not_fit():
    q, k = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64)
    cu, lse = torch.tensor([0, 6], dtype=torch.int32), torch.zeros(6, 4)
    ok = dict(q=q, k=k, v=k, cu=cu, out=q, lse=lse, dout=q)
    for bad, error in ((dict(dout=q[:5]), ValueError), (dict(dout=q.bfloat16()), ValueError),
                       (dict(lse=lse[:, :2]), ValueError), (dict(lse=lse.double()), ValueError),
                       (dict(out=k), ValueError), (dict(k=k.bfloat16()), TypeError),
                       (dict(cu=torch.tensor([0, 5], dtype=torch.int32)), ValueError),
                       (dict(), ValueError)):
        a = {**ok, **bad}
        with pytest.raises(error):
            moba.dense_causal_backward(a["q"], a["k"], a["v"], a["cu"], a["out"], a["lse"],
                                       a["dout"])


FAKE, ODD = 1 << 20, (1 << 20) + 16


def _struct(**kw):
    a = dict(num_pages=4, page_size=16, max_pages=2, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE,
             page_table=FAKE, seqlens=FAKE)
    a.update(kw)
    return moba._CacheStruct(**a)


def _params(**kw):
    a = dict(batch=3, total_tokens=5, max_seqlen=32, num_q_heads=4, num_kv_heads=2, head_dim=64,
             block_size=16, topk=2, dtype=moba.MOBA_BF16)
    a.update(kw)
    return moba.MobaParams(**a)


@pytest.mark.parametrize("cache", [
    dict(num_pages=0), dict(page_size=24), dict(page_size=8), dict(page_size=1 << 17),
    dict(max_pages=0), dict(k=None), dict(v_scale=None), dict(page_table=None),
    dict(seqlens=None), dict(k=ODD), dict(k_scale=ODD)])
def test_entry_points_refuse_a_bad_cache_before_any_launch(cache):
    L, V = moba.lib(), ctypes.c_void_p
    p, c = _params(), _struct(**cache)
    a, b = ctypes.byref(p), ctypes.byref(c)
    f = V(FAKE)
    for fn, args in (
            (L.moba_cache_write, (a, b, f, f, f, f, f, ctypes.c_size_t(1 << 40), None)),
            (L.moba_cache_read, (a, b, f, f, f, None)),
            (L.moba_decode_cache, (a, f, b, f, f, f, None, None, f, ctypes.c_size_t(1 << 40), None))):
        fn.argtypes, fn.restype = None, ctypes.c_int
        assert fn(*args) == moba.MOBA_ERR_INVALID_ARG


def test_entry_points_refuse_bad_pointers_workspaces_and_variants():
    L, V, Z = moba.lib(), ctypes.c_void_p, ctypes.c_size_t
    c = _struct()
    b, f, odd, big = ctypes.byref(c), V(FAKE), V(ODD), Z(1 << 40)
    dec, bwd = L.moba_decode_cache, L.dense_causal_backward
    dec.argtypes = bwd.argtypes = None
    dec.restype = bwd.restype = ctypes.c_int
    for size in (L.moba_decode_cache_workspace_size, L.dense_causal_backward_workspace_size,
                 L.moba_cache_write_workspace_size):
        size.argtypes, size.restype = None, ctypes.c_size_t
        assert size(ctypes.byref(_params(total_tokens=1 << 16))) > 0
        assert size(ctypes.byref(_params(head_dim=96))) == 0
    a = ctypes.byref(_params())
    assert dec(a, odd, b, f, f, f, None, None, f, big, None) == moba.MOBA_ERR_INVALID_ARG
    assert dec(a, f, b, None, f, f, None, None, f, big, None) == moba.MOBA_ERR_INVALID_ARG
    assert dec(a, f, b, f, f, f, None, None, f, Z(1), None) == moba.MOBA_ERR_WORKSPACE
    assert dec(a, f, b, f, f, f, None, None, None, big, None) == moba.MOBA_ERR_WORKSPACE
    for bad in (dict(own_block=1), dict(head_dim=96), dict(topk=33), dict(dtype=5)):
        assert dec(ctypes.byref(_params(**bad)), f, b, f, f, f, None, None, f, big,
                   None) == moba.MOBA_ERR_UNSUPPORTED
    wr, many = L.moba_cache_write, ctypes.byref(_params(total_tokens=1 << 16, num_q_heads=2))
    wr.argtypes, wr.restype = None, ctypes.c_int
    assert wr(many, b, f, f, f, f, f, Z(1), None) == moba.MOBA_ERR_WORKSPACE
    assert wr(many, b, f, f, f, f, None, big, None) == moba.MOBA_ERR_WORKSPACE
    assert wr(many, b, f, odd, f, f, f, big, None) == moba.MOBA_ERR_INVALID_ARG
    ptrs = [f] * 10  # q k v cu out lse dout dq dk dv
    assert bwd(a, *ptrs, f, Z(1), None) == moba.MOBA_ERR_WORKSPACE
    assert bwd(ctypes.byref(_params(kv_layout=1)), *ptrs, f, big, None) == \
        moba.MOBA_ERR_UNSUPPORTED
    for i in range(10):
        q = list(ptrs)
        q[i] = None
        assert bwd(a, *q, f, big, None) == moba.MOBA_ERR_INVALID_ARG
        if i != 3:  # the offsets need no alignment
            q[i] = odd
            assert bwd(a, *q, f, big, None) == moba.MOBA_ERR_INVALID_ARG
    # empty calls launch nothing and need nothing
    empty = ctypes.byref(_params(total_tokens=0))
    assert dec(empty, None, None, None, None, None, None, None, None, Z(0), None) == moba.MOBA_OK
    assert bwd(empty, *([None] * 11), Z(0), None) == moba.MOBA_OK


@pytest.mark.parametrize("B,nb", [(65536, 32769), (2 ** 30, 3), (2 ** 31 - 1, 2)])
def test_means_of_more_blocks_than_positions_are_refused(B, nb):
    """A length ends at 2^31 - 1, so the kernels count at most that many positions' blocks: with more
    in kbar, its second request's means would be looked for in the wrong place."""
    kbar = torch.zeros(3, 1, 2, 64).expand(3, nb, 2, 64)
    assert moba._check_kbar(kbar[:, :-1], 3, 2, 64, B) == min((nb - 1) * B, 2 ** 31 - 1)
    with pytest.raises(ValueError, match="more than there are positions"):
        moba._check_kbar(kbar, 3, 2, 64, B)


@pytest.mark.parametrize("dtype", [moba.MOBA_BF16, moba.MOBA_F32])
@pytest.mark.parametrize("length", [1, 200, 5000])
@pytest.mark.parametrize("B", [8192, 1 << 20, 1 << 30])
def test_decode_workspace_is_bounded_by_the_length(B, length, dtype):
    """Blocks longer than any request: one part at least 128 keys long each, so no more partials a
    row than ceil(length / 128), whatever the block size."""
    size = moba.lib().moba_decode_cache_workspace_size
    size.argtypes, size.restype = None, ctypes.c_size_t
    rows = 4 * 8 * -(-length // 128)
    p = _params(batch=4, total_tokens=4, max_seqlen=length, num_q_heads=8, num_kv_heads=8,
                block_size=B, topk=1, dtype=dtype)
    assert 0 < size(ctypes.byref(p)) <= rows * 65 * 4 + 4 * 8 * 4 + 3 * 256
