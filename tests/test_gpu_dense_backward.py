"""dense_causal_backward on the GPU against the 64-bit formulas (the forward's own out and lse as
inputs), against differences of the loss, and on the calls its documentation allows.

Tolerances, relative 2-norm. fp32: a logit is a sum of d <= 128 products, off by at most
d * 2^-24 * sum|q k| / sqrt(d) ~ 128 * 6e-8 * 3.6 = 2.8e-5 for entries of deviation 0.7, which is
P's relative error; dS has it from P, from dP and from D, and the sum over up to 700 rows adds
700 * 6e-8 = 4e-5 at worst: 1.3e-4. bf16: P or dS and the result are each rounded once, half a
step being 2^-8 relative: 2 * 2^-8 = 7.9e-3 (the fp32 part is far below).

To that comes what cancels. dP_ij = dO_i . v_j and D_i = dO_i . out_i are fp32 sums of d products,
each off by at most d * 2^-24 * sum|dO v| or d * 2^-24 * sum|dO out|, and where their difference
is near zero that does not shrink with it: a row with one key has P = 1, out = v and the gradient
0, so no tolerance relative to the gradient holds there. dq is therefore off by at most
d * 2^-24 * sum_j P_ij (|dO_i|.|v_j| + |dO_i|.|out_i|) |k_j| / sqrt(d) more, dk likewise: `room`
below, with the gradient's own sum in place of the products' and |.| on every factor."""
import pytest
import torch

import long_context_prefill_block_b200 as moba
import reference64 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1.3e-4, torch.bfloat16: 7.9e-3}


def case(lens, Hq, Hkv, d, dtype, seed=0, scale=0.7):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q, k, v, do = ((torch.randn(T, H, d, generator=g) * scale).to(dtype) for H in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor([0] + list(torch.cumsum(torch.tensor(lens), 0)), dtype=torch.int32)
    return q, k, v, do, cu


def run(q, k, v, do, cu, **kw):
    q, k, v, do = (x.to(DEV) for x in (q, k, v, do))
    out, lse = moba.dense_causal_forward(q, k, v, cu, return_lse=True)
    grads = moba.dense_causal_backward(q, k, v, cu, out, lse, do, **kw)
    torch.cuda.synchronize()
    assert moba.moba_device_status() == 0
    return out, lse, grads


def check(q, k, v, do, cu, out, lse, grads):
    want = ref.dense_backward(q, k, v, cu, out.cpu(), lse.cpu(), do)
    eps = q.shape[2] * 2.0 ** -24
    for name, x, y, r in zip(("dq", "dk", "dv"), grads, want, room(q, k, v, cu, out.cpu(),
                                                                   lse.cpu(), do)):
        assert x.dtype == q.dtype and x.shape == y.shape
        err = float((x.double().cpu() - y).norm())
        assert err <= TOL[q.dtype] * float(y.norm()) + eps * r, name


def room(q, k, v, cu, out, lse, do):
    """Norms of the sums of absolute values that dq and dk cancel from (dv cancels nothing)."""
    res = ref.dense_backward(q, k, v, cu, out, lse, do, sizes=True)
    return float(res[0].norm()), float(res[1].norm()), 0.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ((1,), 1, 1, 128), ((2, 1, 3), 2, 1, 64), ((127,), 2, 2, 128), ((128,), 1, 1, 64),
    ((129, 0, 64), 2, 1, 128), ((255, 257), 4, 2, 64), ((65, 63, 1, 500), 3, 3, 128),
    ((640,), 6, 2, 128), ((383, 31), 5, 1, 64), ((1,) * 40 + (129,), 1, 1, 128),
    ((260, 7), 12, 1, 128)])
def test_gradients_match_the_formulas(lens, Hq, Hkv, d, dtype):
    q, k, v, do, cu = case(lens, Hq, Hkv, d, dtype)
    check(q, k, v, do, cu, *run(q, k, v, do, cu))


def test_gradients_match_differences_of_the_loss():
    """Along a random direction u: (loss(x + e u) - loss(x - e u)) / 2e in 64 bits, e = 1e-5 (its
    own error about e^2), against the kernel's gradient times u: within the fp32 tolerance of the
    norms' product."""
    q, k, v, do, cu = case((70, 130), 4, 2, 64, torch.float32, seed=3)
    _, _, grads = run(q, k, v, do, cu)
    g = torch.Generator().manual_seed(9)
    for i in range(3):
        u = torch.randn((q, k, v)[i].shape, generator=g, dtype=torch.float64)
        loss = []
        for e in (1e-5, -1e-5):
            x = [t.double() for t in (q, k, v)]
            x[i] = x[i] + e * u
            loss.append(float((ref.dense_forward(*x, cu)[0] * do.double()).sum()))
        diff = (loss[0] - loss[1]) / 2e-5
        got = float((grads[i].double().cpu() * u).sum())
        assert abs(got - diff) <= TOL[torch.float32] * float(grads[i].double().norm() * u.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_calls_give_equal_bits(dtype):
    q, k, v, do, cu = case((300, 500), 4, 2, 128, dtype, seed=5)
    a = run(q, k, v, do, cu)[2]
    b = run(q, k, v, do, cu)[2]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64),
                                     (torch.float32, 64)])
def test_sequences_do_not_see_each_other_nor_the_padding(dtype, d):
    """A neighbour full of NaN and padding rows of NaN change no bit of a sequence's gradients;
    padding rows get zeros."""
    q, k, v, do, cu = case((200, 77), 4, 2, d, dtype, seed=6)
    out, lse, a = run(q, k, v, do, cu)
    nan = float("nan")
    # out and lse of the call without the padding: the gradient alone is looked at here
    pad = [torch.cat([x, torch.full((50,) + x.shape[1:], nan, dtype=x.dtype, device=x.device)]).to(DEV)
           for x in (q, k, v, do, out, lse)]
    out, lse = pad[4:]
    b = moba.dense_causal_backward(*pad[:3], cu.to(DEV), out, lse, pad[3], max_seqlen=200)
    for x, y in zip(a, b):
        assert torch.equal(x, y[:277]) and not y[277:].any()
    for x in pad:
        x[200:277] = nan
    out[200:277], lse[200:277] = nan, nan
    c = moba.dense_causal_backward(*pad[:3], cu.to(DEV), out, lse, pad[3], max_seqlen=200)
    for x, y in zip(a, c):
        assert torch.equal(x[:200], y[:200])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_logits_and_peaked_rows(dtype):
    """Logits up to several hundred: P is 0 or 1 to the last bit in most places. Absolute against
    the largest gradient, since peaked rows cancel: lse and logits near 500 are off by 500 * 2^-23
    = 6e-5 each in fp32 and P by twice that relatively; bf16 adds its roundings as above."""
    q, k, v, do, cu = case((260,), 2, 1, 64, dtype, seed=7, scale=5.0)
    out, lse, grads = run(q, k, v, do, cu)
    want = ref.dense_backward(q, k, v, cu, out.cpu(), lse.cpu(), do)
    for x, y in zip(grads, want):
        assert torch.isfinite(x).all()
        tol = TOL[dtype] + 2 * 6e-5 * 2
        assert ref.off(x, y) <= 2 * tol


def test_another_stream_and_a_captured_call():
    q, k, v, do, cu = case((150, 333), 4, 2, 128, torch.bfloat16, seed=8)
    out, lse, want = run(q, k, v, do, cu)
    a = [x.to(DEV) for x in (q, k, v, do)]
    cud = cu.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = moba.dense_causal_backward(*a[:3], cud, out, lse, a[3], max_seqlen=333)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moba.dense_causal_backward(*a[:3], cud, out, lse, a[3], max_seqlen=333)
    a[3].mul_(2)  # twice the loss: every step but the roundings doubles, and those are scaled too
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, 2 * y) for x, y in zip(got, want))


def test_a_longer_sequence_than_max_seqlen_is_reported():
    q, k, v, do, cu = case((150, 333), 2, 1, 128, torch.bfloat16, seed=8)
    out, lse, want = run(q, k, v, do, cu)
    a = [x.to(DEV) for x in (q, k, v, do)]
    got = moba.dense_causal_backward(*a[:3], cu.to(DEV), out, lse, a[3], max_seqlen=200)
    torch.cuda.synchronize()
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
    # the tiles' sums are dealt out by max_seqlen: both calls are within the tolerance of the
    # formulas, so within twice that of each other
    for x, y in zip(got, want):
        assert ref.off(x[:150], y[:150].double().cpu()) <= 2 * TOL[torch.bfloat16]
        assert not x[150:].any()


def test_many_tiles_and_a_generous_max_seqlen():
    """Enough tiles that each has one CTA, and a bound of 16 times the longest sequence."""
    q, k, v, do, cu = case((700, 650), 16, 16, 64, torch.bfloat16, seed=14)
    out, lse, grads = run(q, k, v, do, cu)
    check(q, k, v, do, cu, out, lse, grads)
    grads = run(q, k, v, do, cu, max_seqlen=11200)[2]
    check(q, k, v, do, cu, out, lse, grads)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_bound_on_the_lengths(dtype):
    q, k, v, do, cu = case((300, 20), 4, 2, 64, dtype, seed=3)
    out, lse, grads = run(q, k, v, do, cu, max_seqlen=2 ** 31 - 1)
    check(q, k, v, do, cu, out, lse, grads)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ((600,) + (0, 1, 3) * 15, 4, 2, 64), ((0, 0, 2) * 12 + (900, 127, 128, 129, 0), 2, 2, 128),
    ((700, 5, 5, 5), 9, 3, 128), ((1,) * 33 + (770, 0) + (2,) * 40, 1, 1, 64)])
def test_one_long_sequence_among_short_ones(lens, Hq, Hkv, d, dtype):
    """Far fewer tiles than the longest sequence's in each: places are searched, over more than 31
    sequences too."""
    test_gradients_match_the_formulas(lens, Hq, Hkv, d, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", [[0], [0, 0], [0, 0, 0]])
def test_rows_of_no_sequence_at_all_get_zeros(cu, dtype):
    q, k, v, do, _ = (x.to(DEV) for x in case((70,), 4, 2, 64, dtype, seed=2))
    lse = torch.zeros(70, 4, device=DEV)
    grads = moba.dense_causal_backward(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), q,
                                       lse, do, max_seqlen=70)
    assert moba.moba_device_status() == 0
    assert not any(x.any() for x in grads)


def test_two_layers_trained_together():
    """A block-attention layer and a dense layer in a row, as a hybrid stack has them: the loss's
    gradient at the inputs through both, fp32, against 64-bit autograd of the same stack with all
    blocks chosen (then the first layer is dense as well)."""
    lens, H, d = (96, 160), 2, 64
    q, k, v, do, cu = case(lens, H, H, d, torch.float32, seed=11)
    qd, kd, vd, dd = (x.to(DEV) for x in (q, k, v, do))
    B, topk = 32, 5  # 160 tokens have 5 blocks
    o1, l1 = moba.moba_forward(qd, kd, vd, cu, B, topk, return_lse=True)
    o2, l2 = moba.dense_causal_forward(o1, kd, vd, cu, return_lse=True)
    g1, gk2, gv2 = moba.dense_causal_backward(o1, kd, vd, cu, o2, l2, dd)
    gq, gk1, gv1 = moba.moba_backward(qd, kd, vd, cu, o1, l1, g1, B, topk)
    x = [t.double().requires_grad_() for t in (q, k, v)]
    h = _autograd_dense(*x, cu)
    _autograd_dense(h, x[1], x[2], cu).backward(do.double())
    # two layers' errors, the first's input gradient being off already
    for got, t in zip((gq, gk1 + gk2, gv1 + gv2), x):
        assert ref.off(got, t.grad) <= 2 * TOL[torch.float32]


def _autograd_dense(q, k, v, cu):
    res = []
    for b in range(len(cu) - 1):
        a, e = int(cu[b]), int(cu[b + 1])
        s = torch.einsum("ihd,jhd->hij", q[a:e], k[a:e]) / q.shape[2] ** 0.5
        s = s.masked_fill(torch.ones(e - a, e - a, dtype=torch.bool).triu(1), float("-inf"))
        res.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[a:e]))
    return torch.cat(res)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [(150, 333), (700, 5, 5, 5, 40)])  # places that follow, that are searched
def test_offsets_on_the_device_past_the_rows_are_reported_and_skipped(lens, dtype):
    q, k, v, do, cu = case(lens, 4, 2, 64, dtype, seed=8)
    out, lse, want = run(q, k, v, do, cu)
    a = [x.to(DEV) for x in (q, k, v, do)]
    last, T = int(cu[-2]), int(cu[-1])
    for bad in (T + 100, T + 1, 2 ** 31 - 1):
        c = cu.clone()
        c[-1] = bad
        got = moba.dense_causal_backward(*a[:3], c.to(DEV), out, lse, a[3], max_seqlen=max(lens) + 100)
        assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
        for x, y in zip(got, want):  # another bound, another order of sums: see above
            assert ref.off(x[:last], y[:last].double().cpu()) <= 2 * TOL[dtype]
            assert not x[last:].any()
    c = cu.clone()
    c[0] = -3
    got = moba.dense_causal_backward(*a[:3], c.to(DEV), out, lse, a[3], max_seqlen=max(lens) + 100)
    assert moba.moba_device_status() == moba.MOBA_ERR_INVALID_ARG
    for x, y in zip(got, want):
        assert ref.off(x[lens[0]:], y[lens[0]:].double().cpu()) <= 2 * TOL[dtype]
        assert not x[:lens[0]].any()


def formulas_in_pieces(q, k, v, cu, out, lse, do, piece=1024):
    """ref.dense_backward and, with sizes, the sums its errors are relative to, on the GPU for
    `piece` queries at a time: (gradients, sums), float64."""
    Hq, d = q.shape[1:]
    grp = Hq // k.shape[1]
    res = []
    for sizes in (False, True):
        f = torch.abs if sizes else (lambda x: x)
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (q, k, v))
        for a, e in zip(cu.tolist(), cu.tolist()[1:]):
            for i in range(a, e, piece):
                j = min(i + piece, e)
                seen = torch.arange(a, j, device=DEV)[None] <= torch.arange(i, j, device=DEV)[:, None]
                for h in range(Hq):
                    g = h // grp
                    qh, oh, doh = (x[i:j, h].double() for x in (q, out, do))
                    kh, vh = (x[a:j, g].double() for x in (k, v))
                    p = torch.exp(qh @ kh.T / d ** 0.5 - lse[i:j, h].double()[:, None]) * seen
                    D = (f(doh) * f(oh)).sum(1, keepdim=True) * (-1 if sizes else 1)
                    ds = p * (f(doh) @ f(vh).T - D)
                    dq[i:j, h] = ds @ f(kh) / d ** 0.5
                    dk[a:j, g] += ds.T @ f(qh) / d ** 0.5
                    dv[a:j, g] += p.T @ doh
        res.append((dq, dk, dv))
    return res


def test_the_pieces_are_the_formulas():
    q, k, v, do, cu = case((130, 1, 70), 4, 2, 64, torch.float32, seed=15)
    out, lse, _ = run(q, k, v, do, cu)
    got = formulas_in_pieces(*(x.to(DEV) for x in (q, k, v)), cu, out, lse, do.to(DEV), piece=33)
    for sizes, mine in zip((False, True), got):
        want = ref.dense_backward(q, k, v, cu, out.cpu(), lse.cpu(), do, sizes=sizes)
        assert all(ref.off(x, y) < 1e-12 for x, y in zip(mine[:2 if sizes else 3], want))


@pytest.mark.parametrize("lens,Hq,Hkv,d,dtype", [
    ((8192,), 4, 4, 128, torch.bfloat16), ((16383,), 4, 1, 128, torch.bfloat16),
    ((4001, 1, 2500, 129), 6, 2, 64, torch.bfloat16), ((5000, 8192), 2, 2, 64, torch.bfloat16),
    ((8191,), 2, 1, 128, torch.float32), ((5000, 3000), 2, 2, 64, torch.float32)])
def test_long_sequences_match_the_formulas(lens, Hq, Hkv, d, dtype):
    """The lengths that training has. The tolerances above count a sum over 700 rows, 700 * 2^-24:
    here over the longest sequence, and over every q head of a group."""
    q, k, v, do, cu = (x.to(DEV) for x in case(lens, Hq, Hkv, d, dtype, seed=16))
    out, lse = moba.dense_causal_forward(q, k, v, cu.cpu(), return_lse=True)
    grads = moba.dense_causal_backward(q, k, v, cu.cpu(), out, lse, do)
    assert moba.moba_device_status() == 0
    want, sums = formulas_in_pieces(q, k, v, cu, out, lse, do)
    tol = TOL[dtype] + (max(lens) * Hq // Hkv - 700) * 2.0 ** -24
    for name, x, y, r in zip(("dq", "dk", "dv"), grads, want, (*sums[:2], None)):
        err = float((x.double() - y).norm())
        extra = d * 2.0 ** -24 * float(r.norm()) if r is not None else 0.0
        assert err <= tol * float(y.norm()) + extra, (name, err / float(y.norm()), tol)
