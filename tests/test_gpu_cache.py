"""The paged 8-bit cache on the GPU: writing, block means, reading back and decoding over it,
against 64-bit references on the same bits.

Codes, scales and values read back are exact: one rounding, defined by the type. Block means are
sums of B fp32 values: B * 2^-24 relative to their mean magnitude at worst. Decode, relative
2-norm: a logit is off by at most 128 * 2^-24 * sum|q k| / sqrt(d) ~ 128 * 6e-8 * 3.6 = 2.8e-5, a
weight by that relatively, and the sum over n <= 3000 keys by n * 2^-24 = 1.8e-4 at worst: 2.4e-4
in fp32 (and absolutely for lse); bf16 queries: the weights may be rounded to 11 bits (2^-11) and
the result is rounded once (2^-8): 2^-8 + 2^-11 + 2.4e-4 = 4.7e-3."""
import pytest
import torch

import long_context_prefill_block_b200 as moba
import reference64 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 2.4e-4, torch.bfloat16: 4.7e-3}
LSE_TOL = 2.4e-4


class Pool:
    """A cache with shuffled pages, the table of `lens` (positions reserved per request)."""

    def __init__(self, reserve, page, heads, d, seed=0, spare=2):
        need = [-(-n // page) for n in reserve]
        total = sum(need) + spare
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(total, generator=g)
        self.table = torch.full((len(reserve), max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.table = self.table.to(DEV)
        fill = torch.randint(0, 255, (2, total, heads, page, d + 1), generator=g, dtype=torch.uint8)
        fill[fill == 127] = 0  # the two NaN codes
        self.cache = moba.MobaCache(*(fill[i, ..., :d].contiguous().to(DEV).view(
            torch.float8_e4m3fn) for i in range(2)), *(fill[i, ..., d].contiguous().to(DEV).view(
                torch.float8_e8m0fnu) for i in range(2)))

    def bits(self):
        return [x.view(torch.uint8).cpu().clone() for x in self.cache]


def offsets(n):
    return torch.tensor([0] + list(torch.cumsum(torch.tensor(n), 0)), dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def expected(pool, before, x, table, new, lens, which):
    """The bits after writing rows x of K (which 0) or V (1), on the CPU."""
    codes, scales = before[which].clone(), before[which + 2].clone()
    c, e, fine = ref.quantise(x.cpu())
    c = c.float().to(torch.float8_e4m3fn).view(torch.uint8)
    page, i = codes.shape[2], 0
    for r in range(len(new)):
        for j in range(new[r]):
            pos = lens[r] - new[r] + j
            p = int(table[r, pos // page])
            codes[p, :, pos % page] = c[i]
            scales[p, :, pos % page] = torch.where(fine[i], e[i] + 127, 255).to(torch.uint8)
            i += 1
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,old,heads,d,page,B", [
    ([1], [0], 1, 64, 16, 16), ([1, 1, 1], [15, 16, 31], 2, 128, 16, 16),
    ([5, 0, 70, 1], [3, 9, 0, 99], 3, 64, 32, 20), ([300, 129], [0, 7], 2, 128, 64, 100),
    ([257], [255], 8, 128, 128, 64)])
def test_write_is_exact_and_touches_nothing_else(new, old, heads, d, page, B, dtype):
    lens = [a + b for a, b in zip(new, old)]
    pool = Pool(lens, page, heads, d, seed=len(new))
    g = torch.Generator().manual_seed(4)
    n = sum(new)
    k, v = ((torch.randn(n, heads, d, generator=g) * torch.exp2(torch.randint(
        -12, 12, (n, heads, 1), generator=g).float())).to(dtype).to(DEV) for _ in range(2))
    k[0, 0] = 0
    nb = -(-max(lens) // B)
    kbar = torch.full((len(new), nb, heads, d), 7.0, device=DEV)
    before = pool.bits()
    moba.moba_cache_write(pool.cache, k, v, pool.table, i32(lens), offsets(new), kbar, B)
    torch.cuda.synchronize()
    assert moba.moba_device_status() == 0
    after, table = pool.bits(), pool.table.cpu()
    for w, x in enumerate((k, v)):
        codes, scales = expected(pool, before, x, table, new, lens, w)
        # -0 and 0 are one value: compare what the codes stand for, and untouched bytes as bytes
        a, b = (t.view(torch.float8_e4m3fn).float() for t in (after[w], codes))
        assert torch.equal(a, b)
        same = codes == before[w]
        assert torch.equal(after[w + 2], scales) and torch.equal(after[w][same], codes[same])
    for r in range(len(new)):
        rows = ref.cached_rows(pool.cache.k, pool.cache.k_scale, pool.table[r], lens[r])
        for i in range(nb):
            got = kbar[r, i].double().cpu()
            if old[r] // B <= i < lens[r] // B and new[r]:
                blk = rows[i * B:(i + 1) * B]
                tol = B * 2.0 ** -24 * blk.abs().mean(dim=0) + 1e-30
                # the old rows are drawn bytes: where a sum of their magnitudes passes 2^128 it
                # is no 32-bit number, and the mean is not either
                held = blk.abs().sum(dim=0) < 2.0 ** 128
                assert held.any() and ((got - blk.mean(dim=0)).abs() <= tol)[held].all()
            else:
                assert (got == 7.0).all()


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64),
                                     (torch.float32, 128), (torch.float32, 64)])
@pytest.mark.parametrize("B", [1000, 64, 4096])
def test_means_of_long_appends(dtype, d, B):
    """Enough rows that the write leaves sums of 32: blocks that begin in older rows, end inside a
    group or hold none, requests whose rows begin inside a group."""
    old, new, heads, page = [0, 777, 4000, 31], [5003, 4100, 96, 3000], 8, 32
    lens = [a + b for a, b in zip(old, new)]
    pool, _ = filled(lens, heads, d, page, B, seed=41)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = ((torch.randn(sum(new), heads, d, generator=g, device=DEV) + 0.5).to(dtype)
            for _ in range(2))
    nb = -(-max(lens) // B)
    kbar = torch.full((4, nb, heads, d), 7.0, device=DEV)
    moba.moba_cache_write(pool.cache, k, v, pool.table, i32(lens), offsets(new), kbar, B)
    assert moba.moba_device_status() == 0
    for r in range(4):
        rows = contents(pool, r, lens[r])[0]
        for i in range(nb):
            got = kbar[r, i].double().cpu()
            if old[r] // B <= i < lens[r] // B:
                blk = rows[i * B:(i + 1) * B]
                tol = B * 2.0 ** -24 * blk.abs().mean(dim=0)
                assert ((got - blk.mean(dim=0)).abs() <= tol).all()
            else:
                assert (got == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [4, 33, 100, 256, 257])
def test_means_of_small_blocks(d, B):
    """Blocks that one warp sums: none, one or several groups of 32 inside, pages that end in them
    (the last size is past what a warp takes)."""
    test_means_of_long_appends(torch.bfloat16, d, B)


def test_rows_at_the_ends_of_the_number_range():
    """Largest, smallest, subnormal, infinite and NaN rows; reading back stays finite where the
    input was, and NaN rows read back as NaN."""
    big, tiny, inf, nan = 3.4028234663852886e38, 1e-45, float("inf"), float("nan")
    rows = [[big, -big, 1.0], [big * 0.86, 2.0 ** 100, 0], [448.0, 447.9, 1e-3], [tiny, 0, -tiny],
            [2.0 ** -126, 2.0 ** -120, 2.0 ** -140], [inf, 1, 2], [1, nan, 2], [-inf, nan, 0],
            [1e-38, -2e-38, 3e-39], [0, 0, 0]]
    x = torch.zeros(len(rows), 1, 64)
    x[:, 0, :3] = torch.tensor(rows)
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        if dtype == torch.bfloat16:
            y[0] = torch.where(torch.isinf(y[0]), torch.finfo(dtype).max * torch.sign(y[0]), y[0])
        pool = Pool([len(rows)], 16, 1, 64)
        before = pool.bits()
        yd = y.to(DEV)
        moba.moba_cache_write(pool.cache, yd, yd, pool.table, i32([len(rows)]), offsets([len(rows)]))
        codes, scales = expected(pool, before, y, pool.table.cpu(), [len(rows)], [len(rows)], 0)
        after = pool.bits()
        assert torch.equal(after[2], scales)
        assert torch.equal(after[0].view(torch.float8_e4m3fn).float(),
                           codes.view(torch.float8_e4m3fn).float())
        k, v = moba.moba_cache_read(pool.cache, pool.table, i32([len(rows)]), offsets([len(rows)]),
                                    len(rows), dtype=dtype)
        want = ref.cached_rows(pool.cache.k, pool.cache.k_scale, pool.table[0], len(rows)).to(dtype)
        assert torch.equal(k.cpu().isnan(), want.isnan()) and want[5:8].isnan().all()
        assert torch.equal(torch.nan_to_num(k.cpu()), torch.nan_to_num(want))
        assert torch.isfinite(k[:5]).all() and torch.equal(k.isnan(), v.isnan())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,lens,heads,d,page", [
    ([1], [1], 1, 64, 16), ([0, 3, 40], [5, 33, 40], 2, 128, 16), ([200, 77], [300, 77], 4, 64, 64),
    ([129], [1000], 3, 128, 128)])
def test_read_is_exact_and_leaves_padding(rows, lens, heads, d, page, dtype):
    pool = Pool(lens, page, heads, d, seed=3)
    n = sum(rows)
    k, v = (torch.full((n + 9, heads, d), 5.0, dtype=dtype, device=DEV) for _ in range(2))
    a, b = moba.moba_cache_read(pool.cache, pool.table, i32(lens), offsets(rows), n + 9, dtype=dtype,
                                k=k, v=v)
    assert a is k and b is v and moba.moba_device_status() == 0
    at = 0
    for r, m in enumerate(rows):
        for x, c, s in ((k, pool.cache.k, pool.cache.k_scale), (v, pool.cache.v, pool.cache.v_scale)):
            want = ref.cached_rows(c, s, pool.table[r], lens[r])[lens[r] - m:].to(dtype)
            assert torch.equal(x[at:at + m].cpu(), want)
        at += m
    assert (k[n:] == 5).all() and (v[n:] == 5).all()


def filled(lens, heads, d, page, B, seed, room=0):
    """A pool whose requests hold drawn rows with block offsets, its block means and the values."""
    pool = Pool([n + room for n in lens], page, heads, d, seed=seed)
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    k, v = (torch.randn(n, heads, d, generator=g) * 0.7 for _ in range(2))
    at = 0
    for L in lens:
        off = torch.randn(L // B + 1, heads, d, generator=g) * 0.3
        k[at:at + L] += off[torch.arange(L) // B]
        at += L
    nb = max(1, -(-(max(lens + [1]) + room) // B))
    kbar = torch.zeros((len(lens), nb, heads, d), device=DEV)
    if n:
        moba.moba_cache_write(pool.cache, k.to(DEV), v.to(DEV), pool.table, i32(lens),
                              offsets(lens), kbar, B)
    return pool, kbar


def contents(pool, r, length):
    c = pool.cache
    return (ref.cached_rows(c.k, c.k_scale, pool.table[r], length),
            ref.cached_rows(c.v, c.v_scale, pool.table[r], length))


def check_decode(q, pool, lens, nq, B, topk, shared, out, lse, idx):
    at = 0
    outs, lses, wants = [], [], []
    for r in range(len(lens)):
        if nq[r] == 0:
            continue
        keys, values = contents(pool, r, lens[r])
        o, l, i = ref.decode(q[at:at + nq[r]].cpu(), keys, values, B, topk, shared)
        outs.append(o), lses.append(l), wants.append(i)
        at += nq[r]
    assert torch.equal(idx[:at].cpu().long(), torch.cat(wants))
    assert ref.off(out[:at], torch.cat(outs)) <= TOL[q.dtype]
    assert (lse[:at].double().cpu() - torch.cat(lses)).abs().max() <= LSE_TOL


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,d,page,B,topk", [
    ([1], [1], 1, 1, 64, 16, 16, 1), ([1, 2, 17], [1, 2, 1], 2, 1, 128, 16, 16, 3),
    ([100, 0, 257], [1, 0, 3], 4, 2, 64, 32, 20, 4), ([1500, 700], [1, 1], 8, 2, 128, 16, 128, 3),
    ([3000], [4], 4, 4, 128, 64, 100, 12), ([2999, 1025], [2, 1], 10, 2, 128, 64, 1000, 2),
    ([1300], [1], 16, 1, 64, 128, 600, 3), ([700], [1], 3, 3, 128, 64, 4096, 8),
    ([640, 513], [5, 1], 12, 4, 128, 64, 64, 32), ([900, 33], [1, 1], 40, 1, 64, 1024, 64, 5),
    ([2500], [1], 18, 2, 128, 32, 48, 20)])
def test_decode_matches_the_definition(lens, nq, Hq, Hkv, d, page, B, topk, dtype, shared):
    pool, kbar = filled(lens, Hkv, d, page, B, seed=sum(lens))
    g = torch.Generator().manual_seed(1)
    n = sum(nq)
    q = (torch.randn(n, Hq, d, generator=g) * 0.7).to(dtype).to(DEV)
    out, lse, idx = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), offsets(nq), kbar,
                                           B, topk, shared_routing=shared, return_lse=True,
                                           return_idx=True)
    torch.cuda.synchronize()
    assert moba.moba_device_status() == 0
    check_decode(q, pool, lens, nq, B, topk, shared, out, lse, idx)
    # without the extra results, into a given tensor with padded rows behind
    qp = torch.cat([q, q.new_full((2, Hq, d), float("nan"))])
    mine = torch.full_like(qp, 9.0)
    got = moba.moba_decode_cache(qp, pool.cache, pool.table, i32(lens), offsets(nq), kbar, B, topk,
                                 shared_routing=shared, out=mine)
    assert got is mine and (mine[n:] == 9).all() and moba.moba_device_status() == 0
    # a row's keys are split by the number of rows in the call, so the sums' order differs: both
    # are within the tolerance of the definition, and of each other within twice that
    assert ref.off(mine[:n], out.double().cpu()) <= 2 * TOL[dtype]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,d,page,B,topk", [
    ([100, 3, 128], [2, 3, 1], 4, 2, 128, 16, 128, 5),
    ([300, 17, 512], [1, 0, 2], 10, 2, 64, 32, 256, 8),
    ([700, 1500], [3, 1], 8, 8, 128, 64, 1024, 12)])
def test_topk_past_the_blocks_there_are(lens, nq, Hq, Hkv, d, page, B, topk, dtype, shared):
    test_decode_matches_the_definition(lens, nq, Hq, Hkv, d, page, B, topk, dtype, shared)


@pytest.mark.parametrize("dtype,shared", [(torch.bfloat16, False), (torch.float32, True)])
@pytest.mark.parametrize("lens,B,topk,Hq", [
    ([17600, 200], 16, 6, 2), ([5000, 4097], 1, 32, 18), ([49300, 50], 1, 3, 2),
    ([3000, 90], 20, 1, 4)])
def test_many_blocks(lens, B, topk, Hq, dtype, shared):
    """1100 and 5000 blocks, scores of all in shared memory (a part of the heads at a time); 49300,
    lists in registers instead; 150 with nothing to choose."""
    nq = [1, 2]
    pool, kbar = filled(lens, 1, 64, 64, B, seed=31)
    q = (torch.randn(3, Hq, 64, generator=torch.Generator().manual_seed(4)) * 0.7).to(dtype).to(DEV)
    got = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), offsets(nq), kbar, B, topk,
                                 shared_routing=shared, return_lse=True, return_idx=True)
    assert moba.moba_device_status() == 0
    check_decode(q, pool, lens, nq, B, topk, shared, *got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_past_four_gigabytes(dtype):
    """Rows whose byte offsets pass 2^31 and 2^32: the last pages of a 4.4 GB pool of K."""
    pages, page, heads, d, B, L = 4200, 1024, 8, 128, 64, 300
    c = moba.moba_cache_alloc(pages, page, heads, d)
    pool = Pool([1], 16, 1, 64)
    pool.cache, pool.table = c, i32([[pages - 1], [2049]])
    g = torch.Generator().manual_seed(3)
    k, v = ((torch.randn(2 * L, heads, d, generator=g) * 0.7).to(dtype).to(DEV) for _ in range(2))
    kbar = torch.zeros(2, 5, heads, d, device=DEV)
    moba.moba_cache_write(c, k, v, pool.table, i32([L, L]), offsets([L, L]), kbar, B)
    a, b = moba.moba_cache_read(c, pool.table, i32([L, L]), offsets([L, L]), 2 * L, dtype=dtype)
    for x, y in ((a, k), (b, v)):
        code, e, _ = ref.quantise(y.cpu())
        assert torch.equal(x.cpu(), (code * torch.exp2(e.double())[..., None]).to(dtype))
    q = (torch.randn(2, 16, d, generator=g) * 0.7).to(dtype).to(DEV)
    out, lse, idx = moba.moba_decode_cache(q, c, pool.table, i32([L, L]), offsets([1, 1]), kbar, B,
                                           3, return_lse=True, return_idx=True)
    assert moba.moba_device_status() == 0
    for r in range(2):
        keys, values = (x[r * L:(r + 1) * L].double().cpu() for x in (a, b))
        o, l, i = ref.decode(q[r:r + 1].cpu(), keys, values, B, 3, False)
        assert torch.equal(idx[r:r + 1].cpu().long(), i) and ref.off(out[r:r + 1], o) <= TOL[dtype]
        assert (lse[r:r + 1].double().cpu() - l).abs().max() <= LSE_TOL


def test_many_requests_with_one_token_each():
    """70 requests, some without a row, in one call, with padded rows behind: three rounds of the
    search for a row's request."""
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(1, 90, (70,), generator=g).tolist()
    nq = [0 if r % 9 == 4 else 1 for r in range(70)]
    n, B = sum(nq), 16
    pool, kbar = filled(lens, 2, 64, 16, B, seed=32)
    x = (torch.randn(n + 5, 2, 64, generator=g) * 0.7).to(DEV)
    x[n:] = float("nan")
    before = pool.bits()
    moba.moba_cache_write(pool.cache, x, -x, pool.table, i32(lens), offsets(nq), kbar, B)
    for w, y in enumerate((x[:n], -x[:n])):
        codes, scales = expected(pool, before, y, pool.table.cpu(), nq, lens, w)
        after = pool.bits()
        assert torch.equal(after[w].view(torch.float8_e4m3fn).float(),
                           codes.view(torch.float8_e4m3fn).float())
        assert torch.equal(after[w + 2], scales)
    q = (torch.randn(n, 4, 64, generator=g) * 0.7).to(DEV)
    got = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), offsets(nq), kbar, B, 3,
                                 return_lse=True, return_idx=True)
    assert moba.moba_device_status() == 0
    check_decode(q, pool, lens, nq, B, 3, False, *got)
    k, _ = moba.moba_cache_read(pool.cache, pool.table, i32(lens), offsets(nq), n,
                                dtype=torch.float32)
    c, e, _ = ref.quantise(x[:n].cpu())
    assert torch.equal(k.cpu().double(), c * torch.exp2(e.double())[..., None])


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64),
                                     (torch.float32, 128)])
def test_decode_never_looks_past_a_request(dtype, d):
    """Rows behind a request's length in its last page, unused pages and other requests' rows may
    hold NaN: no bit of the result changes."""
    lens, nq, B, page = [333, 70], [2, 1], 50, 64
    pool, kbar = filled(lens, 2, d, page, B, seed=5)
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    args = (pool.table, i32(lens), offsets(nq), kbar, B, 3)
    want = moba.moba_decode_cache(q, pool.cache, *args)
    used = torch.zeros(pool.cache.k.shape[0], page, dtype=torch.bool)
    for r, L in enumerate(lens):
        at = torch.arange(L)
        used[pool.table[r].cpu().long()[at // page], at % page] = True
    for x in pool.cache[:2]:
        x.view(torch.uint8).transpose(1, 2)[~used.to(DEV)] = 127
    for x in pool.cache[2:]:
        x.view(torch.uint8).transpose(1, 2)[~used.to(DEV)] = 255
    kbar[0, 6:] = float("nan")  # means of blocks that are not complete
    kbar[1, 1:] = float("nan")
    assert torch.equal(moba.moba_decode_cache(q, pool.cache, *args), want)
    # a NaN row that is read makes its readers NaN
    pool.cache.k_scale.view(torch.uint8)[int(pool.table[1, 0]), :, 0] = 255
    got = moba.moba_decode_cache(q, pool.cache, *args)
    assert torch.equal(got[:2], want[:2]) and got[2].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_queries_and_scales(dtype):
    """Queries 2^30 times larger and keys 2^-30 smaller give the same logits; queries of 2^-100
    give the plain mean of the values. Powers of two: only the weights' own rounding differs."""
    lens, B = [300], 64
    pool, kbar = filled(lens, 2, 128, 32, B, seed=8)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 4, 128, generator=g).to(dtype).to(DEV)
    args = (pool.table, i32(lens), offsets([1]))
    a = moba.moba_decode_cache(q, pool.cache, *args, kbar, B, 5, return_lse=True)
    pool.cache.k_scale.view(torch.uint8).sub_(30)
    b = moba.moba_decode_cache(q * 2.0 ** 30, pool.cache, *args, kbar * 2.0 ** -30, B, 5,
                               return_lse=True)
    assert ref.off(b[0], a[0].double().cpu()) <= TOL[dtype]
    assert (a[1] - b[1]).abs().max() <= LSE_TOL
    out = moba.moba_decode_cache(q * 2.0 ** -100, pool.cache, *args, kbar, B, 5)
    mean = contents(pool, 0, 300)[1].mean(dim=0).repeat_interleave(2, 0)[None]
    assert ref.off(out, mean) <= TOL[dtype]


def test_bad_pages_and_lengths_are_reported_and_skipped():
    lens, B = [200, 150, 90], 32
    pool, kbar = filled(lens, 2, 64, 16, B, seed=9)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(2)).to(DEV)
    cu = offsets([1, 1, 1])
    want = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), cu, kbar, B, 16)
    assert moba.moba_device_status() == 0
    table = pool.table.clone()
    table[0, 1], table[0, 3] = -1, pool.cache.k.shape[0]  # no pages of the pool
    got = moba.moba_decode_cache(q, pool.cache, table, i32(lens), cu, kbar, B, 16)
    assert moba.moba_device_status() == moba.MOBA_ERR_BAD_INDICES
    assert torch.isfinite(got).all() and torch.equal(got[1:], want[1:])
    table[0] = 1 << 30
    got = moba.moba_decode_cache(q, pool.cache, table, i32(lens), cu, kbar, B, 16)
    assert moba.moba_device_status() == moba.MOBA_ERR_BAD_INDICES
    assert (got[0] == 0).all() and torch.equal(got[1:], want[1:])
    before = pool.bits()
    x = torch.ones(200, 2, 64, device=DEV)
    moba.moba_cache_write(pool.cache, x, x, table, i32(lens), offsets([200, 0, 0]), kbar, B)
    assert moba.moba_device_status() == moba.MOBA_ERR_BAD_INDICES
    assert all(torch.equal(a, b) for a, b in zip(pool.bits(), before))
    k = torch.full((200, 2, 64), 3.0, device=DEV)
    moba.moba_cache_read(pool.cache, table, i32(lens), offsets([200, 0, 0]), 200,
                         dtype=torch.float32, k=k, v=k.clone())
    assert moba.moba_device_status() == moba.MOBA_ERR_BAD_INDICES and (k == 3).all()
    # more rows than positions, lengths past the pages or kbar, a negative length
    for bad in ([0, 150, 90], [1 << 20, 150, 90], [-5, 150, 90], [pool.table.shape[1] * 16 + 1, 150, 90]):
        out = torch.full_like(q, 4.0)
        moba.moba_decode_cache(q, pool.cache, pool.table, i32(bad), cu, kbar, B, 16, out=out)
        assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
        assert (out[0] == 4).all() and torch.equal(out[1:], want[1:])
        moba.moba_cache_write(pool.cache, x[:1], x[:1], pool.table, i32(bad), offsets([1, 0, 0]),
                              kbar, B)
        assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
        assert all(torch.equal(a, b) for a, b in zip(pool.bits(), before))
        k.fill_(3.0)
        moba.moba_cache_read(pool.cache, pool.table, i32(bad), offsets([1, 0, 0]), 200,
                             dtype=torch.float32, k=k, v=k.clone())
        assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG and (k == 3).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving_loop(dtype):
    """A prompt through the prefill forward and into the cache, then decoding token by token, the
    first steps eager and the rest as replays of one captured step; each step against the
    definition on the cache's contents, and the whole cache read back at the end."""
    Hq, Hkv, d, page, B, topk = 8, 2, 128, 32, 64, 3
    prompt, steps = [150, 61], 6
    room = steps + 2
    pool = Pool([n + room for n in prompt], page, Hkv, d, seed=12)
    g = torch.Generator().manual_seed(13)
    mk = lambda n, h: (torch.randn(n, h, d, generator=g) * 0.7).to(dtype).to(DEV)  # noqa: E731
    n = sum(prompt)
    q, k, v = mk(n, Hq), mk(n, Hkv), mk(n, Hkv)
    cu = offsets(prompt)
    out = moba.moba_forward(q, k, v, cu, B, topk, max_seqlen=max(prompt))
    nb = -(-(max(prompt) + room) // B)
    kbar = torch.zeros(2, nb, Hkv, d, device=DEV)
    lens = i32(prompt)
    moba.moba_cache_write(pool.cache, k, v, pool.table, lens, cu, kbar, B)
    assert torch.isfinite(out).all()
    one = offsets([1, 1])
    qs, ks, vs = mk(2, Hq), mk(2, Hkv), mk(2, Hkv)

    def step():
        moba.moba_cache_write(pool.cache, ks, vs, pool.table, lens, one, kbar, B)
        return moba.moba_decode_cache(qs, pool.cache, pool.table, lens, one, kbar, B, topk,
                                      return_lse=True, return_idx=True)

    graph = None
    for t in range(steps):
        for x, h in ((qs, Hq), (ks, Hkv), (vs, Hkv)):
            x.copy_(mk(2, h))
        lens += 1
        if t < 2:
            res = step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    res = step()
            graph.replay()
        torch.cuda.synchronize()
        assert moba.moba_device_status() == 0
        check_decode(qs, pool, lens.tolist(), [1, 1], B, topk, False, *res)
    full = lens.tolist()
    rk, rv = moba.moba_cache_read(pool.cache, pool.table, lens, offsets(full), sum(full),
                                  dtype=dtype)
    want = torch.cat([torch.stack(contents(pool, r, full[r])) for r in range(2)], dim=1).to(dtype)
    assert torch.equal(torch.stack([rk, rv]).cpu(), want)


def test_two_streams_at_once():
    """Two decodes over one cache on two streams, each with its own results."""
    lens, B = [900, 400], 64
    pool, kbar = filled(lens, 2, 128, 32, B, seed=21)
    q = torch.randn(2, 2, 8, 128, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    args = (pool.cache, pool.table, i32(lens), offsets([1, 1]), kbar, B, 4)
    want = [moba.moba_decode_cache(q[i], *args) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(moba.moba_decode_cache(q[i], *args))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,heads,B", [([40, 30], 2, 16), ([40, 30], 2, 300),
                                          ([6000, 3500], 8, 512), ([6000, 3500], 8, 64)])
@pytest.mark.parametrize("where", ["inside", "behind", "before"])
def test_offsets_past_the_rows_of_a_call_are_reported_and_skipped(rows, heads, B, where):
    """Offsets on the device that promise more rows than the call has: the request that reaches past
    them is left alone in every call, the other one is served. The larger calls make block means
    from sums of 32 rows, which exist for the call's rows only."""
    d, n = 64, sum(rows)
    lens = [rows[0] + 5, rows[1] + 700]
    cu = {"inside": [0, rows[0], n + 600],  # its first rows are there
          "behind": [0, n, n + 600],        # none of its rows is there
          "before": [-600, rows[0], n]}[where]
    bad = 0 if where == "before" else 1
    good = 1 - bad
    lens[good] = max(lens[good], cu[good + 1] - cu[good])
    lens[0] += 600 if where == "before" else 0
    pool, _ = filled([x + 8 for x in lens], heads, d, 32, B, seed=5)
    before = pool.bits()
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(n, heads, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    kbar = torch.full((2, -(-max(lens) // B), heads, d), 7.0, device=DEV)
    assert moba.moba_device_status() == 0
    moba.moba_cache_write(pool.cache, k, v, pool.table, i32(lens), i32(cu), kbar, B)
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
    # the same as a call in which the other request has no rows
    alone = list(cu)
    alone[2 * bad] = alone[1]
    want, mine = torch.full_like(kbar, 7.0), pool.bits()
    for x, y in zip(pool.cache, before):
        x.view(torch.uint8).copy_(y)
    moba.moba_cache_write(pool.cache, k, v, pool.table, i32(lens), i32(alone), want, B)
    assert moba.moba_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(pool.bits(), mine))
    assert torch.equal(kbar, want) and (kbar[bad] == 7.0).all()
    if cu[good + 1] - cu[good] >= B:
        assert (kbar[good] != 7.0).any()
    got, want = ([torch.full_like(k, 3.0) for _ in range(2)] for _ in range(2))
    moba.moba_cache_read(pool.cache, pool.table, i32(lens), i32(cu), n, k=got[0], v=got[1])
    # a read asks for rows that the call has: it cannot see a request behind them
    seen = moba.MOBA_OK if where == "behind" else moba.MOBA_ERR_INVALID_ARG
    assert moba.moba_device_status() == seen
    moba.moba_cache_read(pool.cache, pool.table, i32(lens), i32(alone), n, k=want[0], v=want[1])
    assert moba.moba_device_status() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [64, 8])  # choice inside each split, and in a launch of its own
def test_decode_offsets_past_the_queries_are_reported_and_skipped(B, dtype):
    lens = [300, 900]
    pool, kbar = filled(lens, 2, 64, 32, B, seed=6)
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    args = (kbar, B, 3)
    want = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), i32([0, 2, 4]), *args)
    out = torch.full_like(q, 9.0)
    moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), i32([0, 2, 5]), *args, out=out)
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
    assert torch.equal(out[:2], want[:2]) and (out[2:] == 9).all()
    out.fill_(9.0)
    moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), i32([-1, 2, 4]), *args, out=out)
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
    assert torch.equal(out[2:], want[2:]) and (out[:2] == 9).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_block_that_would_end_past_two_to_the_31(dtype):
    """Blocks of 1.2e9 positions, the query in the second one: most parts of its block lie past the
    largest position. Every page of the table is the same one, so a row counts as often as it is
    named: its logit plus the logarithm of that. (49 parts hold keys: the sums are as long as the
    tolerance says.)"""
    B, page, d, more = 1_200_000_000, 65536, 64, 100_000
    L = B + more
    pool = Pool([page], page, 1, d, spare=0)
    g = torch.Generator().manual_seed(2)
    k, v = ((torch.randn(page, 1, d, generator=g) * 0.7).to(DEV) for _ in range(2))
    moba.moba_cache_write(pool.cache, k, v, pool.table, i32([page]), offsets([page]))
    keys, values = contents(pool, 0, page)
    q = (torch.randn(1, 2, d, generator=g) * 0.7).to(dtype).to(DEV)
    table = torch.zeros(1, -(-L // page), dtype=torch.int32, device=DEV)
    out, lse = moba.moba_decode_cache(q, pool.cache, table, i32([L]), offsets([1]),
                                      torch.zeros(1, 2, 1, d, device=DEV), B, 1, return_lse=True)
    assert moba.moba_device_status() == 0
    times = torch.bincount(torch.arange(B, L) % page, minlength=page).double()
    for h in range(2):
        z = keys[:, 0] @ q[0, h].double().cpu() / d ** 0.5 + times.log()
        want = torch.logsumexp(z, 0)
        assert abs(float(lse[0, h]) - float(want)) <= LSE_TOL
        assert ref.off(out[0, h], torch.exp(z - want) @ values[:, 0]) <= TOL[dtype]
    # longer than any position may be
    long = torch.zeros(1, 1 << 15, dtype=torch.int32, device=DEV)
    mine = torch.full_like(q, 9.0)
    moba.moba_decode_cache(q, pool.cache, long, i32([2 ** 31 - 4095]), offsets([1]),
                           torch.zeros(1, 2, 1, d, device=DEV), B, 1, out=mine)
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG and (mine == 9).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [64, 4])  # choice inside each split, and in a launch of its own
def test_queries_near_the_largest_number(B, dtype):
    """Queries of 2^120 and keys 2^118 times smaller than usual give ordinary logits (of up to about
    16, so that a product without the key's scale passes 2^128): powers of two, as above."""
    lens = [300]
    pool, kbar = filled(lens, 2, 128, 32, B, seed=8)
    q = (4 * torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(3))).to(dtype).to(DEV)
    args = (pool.table, i32(lens), offsets([1]))
    kw = dict(return_lse=True, return_idx=True)
    a = moba.moba_decode_cache(q, pool.cache, *args, kbar, B, 5, **kw)
    keys = contents(pool, 0, 300)[0]
    assert (torch.einsum("hd,lgd->hlg", q[0].double().cpu(), keys).abs().max() / 128 ** 0.5) > 8
    pool.cache.k_scale.view(torch.uint8).sub_(118)
    b = moba.moba_decode_cache(q * 2.0 ** 118, pool.cache, *args, kbar * 2.0 ** -118, B, 5, **kw)
    assert torch.isfinite(b[0]).all() and torch.equal(a[2], b[2])
    assert ref.off(b[0], a[0].double().cpu()) <= TOL[dtype]
    assert (a[1] - b[1]).abs().max() <= LSE_TOL


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("bound", [None, 200])
def test_blocks_far_longer_than_any_request(bound, shared, dtype):
    """A block that is never completed: the parts that a row's keys are divided into follow the
    lengths there can be (max_seqlen, or what the pages hold), not the block size."""
    lens, nq, B = [200, 1, 130], [1, 1, 2], 1 << 30
    pool, kbar = filled(lens, 2, 128, 16, B, seed=4)
    assert kbar.shape[1] == 1
    q = (torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(1)) * 0.7).to(dtype).to(DEV)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = moba.moba_decode_cache(q, pool.cache, pool.table, i32(lens), offsets(nq), kbar, B, 2,
                                 max_seqlen=bound, shared_routing=shared, return_lse=True,
                                 return_idx=True)
    # partials of 32 rows in two parts, 129 floats each, and the results
    assert torch.cuda.max_memory_allocated() - held < 1 << 20
    assert moba.moba_device_status() == 0
    check_decode(q, pool, lens, nq, B, 2, shared, *got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,shared", [(512, False), (64, True)])
def test_captured_long_calls_replayed_on_other_inputs(B, shared, dtype):
    """A write that leaves sums for its means, and a decode whose choice is a launch of its own, both
    overlapped launches, in two graphs replayed in turn: the same bits as eager calls."""
    lens, heads, d, page, topk = [9000, 34000], 8, 64, 64, 6
    pool = Pool(lens, page, heads, d, seed=3)
    drawn = [x.to(DEV) for x in pool.bits()]  # rows that no request has keep these
    kbar = torch.zeros(2, -(-max(lens) // B), heads, d, device=DEV)
    args = (pool.table, i32(lens))
    g = torch.Generator(device=DEV).manual_seed(7)
    draw = lambda n, h: (torch.randn(n, h, d, generator=g, device=DEV) * 0.7).to(dtype)  # noqa: E731
    k, v, q = draw(sum(lens), heads), draw(sum(lens), heads), draw(4, 16)
    write = lambda: moba.moba_cache_write(pool.cache, k, v, *args, offsets_w, kbar, B)  # noqa: E731
    decode = lambda: moba.moba_decode_cache(q, pool.cache, *args, offsets_q, kbar, B, topk,  # noqa: E731
                                            shared_routing=shared, return_lse=True, return_idx=True)
    offsets_w, offsets_q = offsets(lens), offsets([1, 3])
    write(), decode()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        write()
    with torch.cuda.graph(graphs[1]):
        got = decode()
    for _ in range(3):
        for x in (k, v, q):
            x.copy_(draw(*x.shape[:2]))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        bits, means, res = pool.bits(), kbar.clone(), [x.clone() for x in got]
        for x, y in zip(pool.cache, drawn):
            x.view(torch.uint8).copy_(y)
        kbar.zero_()
        write()
        assert all(torch.equal(a, b) for a, b in zip(pool.bits(), bits))
        assert torch.equal(kbar, means) and all(torch.equal(a, b) for a, b in zip(decode(), res))
    assert moba.moba_device_status() == 0
    if dtype == torch.float32:  # one look at the definition, too: 34000 keys of 8 heads on the CPU
        check_decode(q, pool, lens, [1, 3], B, topk, shared, *res)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_without_rows(dtype):
    pool, kbar = filled([40, 3], 2, 64, 16, 16, seed=2)
    before, means = pool.bits(), kbar.clone()
    none, lens = offsets([0, 0]), i32([40, 3])
    x = torch.empty(0, 2, 64, dtype=dtype, device=DEV)
    moba.moba_cache_write(pool.cache, x, x, pool.table, lens, none, kbar, 16)
    k, v = moba.moba_cache_read(pool.cache, pool.table, lens, none, 0, dtype=dtype)
    out, lse, idx = moba.moba_decode_cache(x.new_empty(0, 4, 64), pool.cache, pool.table, lens, none,
                                           kbar, 16, 3, return_lse=True, return_idx=True)
    assert k.shape == v.shape == (0, 2, 64) and out.shape == (0, 4, 64)
    assert lse.shape == (0, 4) and idx.shape == (0, 4, 3)
    # rows that no request owns
    y = torch.ones(5, 2, 64, dtype=dtype, device=DEV)
    moba.moba_cache_write(pool.cache, y, y, pool.table, lens, none, kbar, 16)
    moba.moba_cache_read(pool.cache, pool.table, lens, none, 5, dtype=dtype, k=y)
    q = torch.ones(5, 4, 64, dtype=dtype, device=DEV)
    out = moba.moba_decode_cache(q, pool.cache, pool.table, lens, none, kbar, 16, 3,
                                 out=torch.full_like(q, 9.0))
    assert moba.moba_device_status() == 0 and (y == 1).all() and (out == 9).all()
    assert all(torch.equal(a, b) for a, b in zip(pool.bits(), before)) and torch.equal(kbar, means)
