"""64-bit references of the dense gradient and of the 8-bit cache, written from
their formulas in plain torch on the CPU; they share no code with the library."""
import math

import torch


def dense_forward(q, k, v, cu):
    """(out, lse) of dense causal attention, float64."""
    q, k, v = q.double(), k.double(), v.double()
    T, Hq, d = q.shape
    grp = Hq // k.shape[1]
    out, lse = torch.zeros_like(q), torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(cu) - 1):
        at = slice(int(cu[b]), int(cu[b + 1]))
        n = at.stop - at.start
        later = torch.ones(n, n, dtype=torch.bool).triu(1)
        for h in range(Hq):
            s = (q[at, h] @ k[at, h // grp].T / math.sqrt(d)).masked_fill(later, -math.inf)
            lse[at, h] = torch.logsumexp(s, dim=1)
            out[at, h] = torch.exp(s - lse[at, h][:, None]) @ v[at, h // grp]
    return out, lse


def dense_backward(q, k, v, cu, out, lse, dout, sizes=False):
    """(dq, dk, dv) by the formulas, with the given out and lse, float64; `sizes`: the same sums
    with every factor of dP, D, q and k taken absolutely and D added to dP, what their rounding
    errors are relative to."""
    q, k, v, out, lse, dout = (x.double() for x in (q, k, v, out, lse, dout))
    T, Hq, d = q.shape
    grp = Hq // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(len(cu) - 1):
        at = slice(int(cu[b]), int(cu[b + 1]))
        n = at.stop - at.start
        later = torch.ones(n, n, dtype=torch.bool).triu(1)
        for h in range(Hq):
            g = h // grp
            p = torch.exp(q[at, h] @ k[at, g].T / math.sqrt(d) - lse[at, h][:, None])
            p = p.masked_fill(later, 0.0)
            do, vv, oo, qq, kk = dout[at, h], v[at, g], out[at, h], q[at, h], k[at, g]
            if sizes:
                do, vv, oo, qq, kk = do.abs(), vv.abs(), -oo.abs(), qq.abs(), kk.abs()
            ds = p * (do @ vv.T - (do * oo).sum(1, keepdim=True))
            dq[at, h] = ds @ kk / math.sqrt(d)
            dk[at, g] += ds.T @ qq / math.sqrt(d)
            dv[at, g] += p.T @ dout[at, h]
    return dq, dk, dv


def quantise(x):
    """(codes as values, exponents, finite) of rows x [..., d]: float64, int64, bool."""
    x = x.double()
    fine = torch.isfinite(x).all(dim=-1)
    y = torch.where(fine[..., None], x, torch.zeros_like(x))
    top = y.abs().amax(dim=-1)
    e = torch.full(top.shape, -127, dtype=torch.int64)
    for cand in range(-126, 121):  # the smallest that holds the maximum
        e = torch.where(top > 448.0 * 2.0 ** (cand - 1), cand, e)
    y = y * torch.exp2(-e.double())[..., None]
    lim = torch.where(e >= 120, 240.0, 448.0).double()[..., None]
    y = torch.minimum(torch.maximum(y, -lim), lim)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e, fine


def stored_value(codes, scales):
    """What a cache's tensors stand for, from their bits, float64."""
    c = codes.view(torch.uint8).to(torch.int64)
    ex, man = (c >> 3) & 15, c & 7
    mag = torch.where(ex == 0, man.double() * 2.0 ** -9,
                      (8 + man).double() * torch.exp2((ex - 10).double()))
    s = scales.view(torch.uint8).to(torch.int64)
    s = torch.where(s == 255, math.nan, torch.exp2((s - 127).double()))
    return torch.where(c >= 128, -mag, mag) * s[..., None]


def cached_rows(codes, scales, table_row, length):
    """The first `length` positions of a request, [length, Hkv, d] float64."""
    page = codes.shape[2]
    x = stored_value(codes.cpu(), scales.cpu())
    at = torch.arange(length)
    return x[table_row.cpu().long()[at // page], :, at % page]


def decode(q, keys, values, B, topk, shared):
    """out, lse, idx of queries q [n, Hq, d] at the last n positions of one request whose cache
    holds keys, values [L, Hkv, d]: gate on whole blocks' means, own block forced."""
    q, keys, values = q.double(), keys.double(), values.double()
    n, Hq, d = q.shape
    L, Hkv = keys.shape[:2]
    grp = Hq // Hkv
    out, lse = torch.zeros_like(q), torch.zeros(n, Hq, dtype=torch.float64)
    idx = torch.full((n, Hq, topk), -1, dtype=torch.int64)
    for i in range(n):
        p = L - n + i
        c = p // B
        mean = keys[:c * B].reshape(c, B, Hkv, d).mean(dim=1)
        for h in range(Hq):
            g = h // grp
            qs = q[i, g * grp:(g + 1) * grp].mean(dim=0) if shared else q[i, h]
            s = (mean[:, g] @ qs).tolist()
            ids = sorted(sorted(range(c), key=lambda b: (-s[b], b))[:topk - 1]) + [c]
            idx[i, h, :len(ids)] = torch.tensor(ids)
            at = torch.cat([torch.arange(b * B, min((b + 1) * B, p + 1)) for b in ids])
            z = keys[at, g] @ q[i, h] / math.sqrt(d)
            lse[i, h] = torch.logsumexp(z, 0)
            out[i, h] = torch.exp(z - lse[i, h]) @ values[at, g]
    return out, lse, idx


def off(x, ref):
    """Relative 2-norm of the difference."""
    ref = ref.double()
    d, n = float((x.double().cpu() - ref).norm()), float(ref.norm())
    return d / n if n else d
