"""Measured cases of four operators: the gradient of dense causal attention,
writing keys and values into an 8-bit paged cache, reading them back, and the
decode step of block attention over that cache.

With `own` false, run() computes each operator in plain torch operations in
32 bits; with `own` true it calls the library. prepare() makes the same
inputs for both. Sizes come from the repository's workload table (4 x 8192
with 16 heads, 32768 tokens with blocks of 512, a million tokens with 32 query
and 8 kv heads in blocks of 4096 of which 12 are chosen) and from generic odd
and small ones.

The 8-bit cache holds pages of `page` tokens, [pages, kv heads, page, d] in
e4m3 with one power-of-two scale (e8m0) for each (token, kv head) row of K and
of V: the smallest 2^e with max|x| <= 448 * 2^e, so that scaling is exact and
a value is rounded once.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SCALE = 1.0 / math.sqrt(2.0)  # standard deviation of q, k, v in the workload table
_OFFSET = 0.3                  # standard deviation of a block's key offset


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # two short sequences, the smallest step of a fine-tuning run: latency counts
        {"name": "grad short", "op": "grad", "lens": "300,212", "hq": 4, "hkv": 2, "d": 128,
         "dt": "bf16"},
        # the scaling workload: four sequences of 8192 tokens, 16 heads
        {"name": "grad 4x8192", "op": "grad", "lens": "8192,8192,8192,8192", "hq": 16, "hkv": 16,
         "d": 128, "dt": "bf16"},
        # one long sequence with grouped heads, odd length
        {"name": "grad 16383 grouped", "op": "grad", "lens": "16383", "hq": 16, "hkv": 4, "d": 128,
         "dt": "bf16"},
        # ragged batch with head dim 64
        {"name": "grad ragged d64", "op": "grad", "lens": "4001,1,2500,129", "hq": 12, "hkv": 4,
         "d": 64, "dt": "bf16"},
        # 32-bit inputs, as a gradient check or a small full-precision run has them
        {"name": "grad fp32", "op": "grad", "lens": "1024,777", "hq": 4, "hkv": 4, "d": 64,
         "dt": "fp32"},
        # one token for each of 64 running requests; a few of them complete a block
        {"name": "write tokens", "op": "write", "batch": 64, "old": 4000, "new": 1, "hkv": 8,
         "d": 128, "page": 64, "block": 512, "dt": "bf16"},
        # a long prompt's keys and values enter the cache at once
        {"name": "write prompt", "op": "write", "batch": 1, "old": 0, "new": 262144, "hkv": 8,
         "d": 128, "page": 64, "block": 4096, "dt": "bf16"},
        # the last 100 positions of each request, read back for a recomputation
        {"name": "read tails", "op": "read", "batch": 16, "old": 2000, "new": 100, "hkv": 8,
         "d": 128, "page": 64, "dt": "bf16"},
        # a whole long cache read back
        {"name": "read prompt", "op": "read", "batch": 1, "old": 0, "new": 262144, "hkv": 8,
         "d": 128, "page": 64, "dt": "bf16"},
        # a few short requests: latency counts
        {"name": "decode short", "op": "decode", "batch": 4, "len": 1500, "nq": 1, "hq": 8,
         "hkv": 2, "d": 128, "page": 16, "block": 128, "topk": 3, "shared": False, "dt": "bf16"},
        # a serving batch at 32768 tokens
        {"name": "decode 48x32768", "op": "decode", "batch": 48, "len": 32768, "nq": 1, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "block": 512, "topk": 3, "shared": True, "dt": "bf16"},
        # the million-token cache, four drafted positions of one request
        {"name": "decode 1M", "op": "decode", "batch": 1, "len": 1048576, "nq": 4, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "block": 4096, "topk": 12, "shared": False, "dt": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grad", "grad", "write", "read", "decode", "decode"))
    d = rng.choice((128, 128, 64))
    if op == "grad":
        dt = rng.choice(("bf16", "bf16", "bf16", "fp32"))
        hkv = rng.choice((1, 2, 3, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4))
        batch = rng.randint(1, 5)
        top = int(min(16383, math.sqrt((1.0e9 if dt == "bf16" else 3e7) / (batch * hq))))
        longest = _log(rng, min(64, top), top)
        lens = [longest] + [_log(rng, 1, longest) for _ in range(batch - 1)]
        rng.shuffle(lens)
        return {"op": op, "lens": ",".join(map(str, lens)), "hq": hq, "hkv": hkv, "d": d, "dt": dt}
    page = rng.choice((16, 32, 64, 128))
    block = rng.choice((64, 100, 128, 512, 1000, 2048, 4096))
    hkv = rng.choice((1, 2, 4, 8))
    dt = rng.choice(("bf16", "bf16", "fp32"))
    if op in ("write", "read"):
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, 262144 * 8 // (hkv * batch) // (2 if dt == "fp32" else 1))
        c = {"op": op, "batch": batch, "old": rng.choice((0, _log(rng, 1, 8192))),
             "new": min(new, 262144), "hkv": hkv, "d": d, "page": page, "dt": dt}
        if op == "write":
            c["block"] = block
        return c
    batch = _log(rng, 1, 48)
    topk = rng.choice((1, 2, 3, 5, 8, 12))
    nq, grp = rng.choice((1, 1, 2, 4)), rng.choice((1, 2, 4, 5))
    # the plain form gathers every chosen row: no more of them than the largest listed case has
    batch = max(1, min(batch, 4 * 32 * 12 * 4096 // (nq * hkv * grp * topk * block)))
    length = _log(rng, 200, min(1048576, 12000000 // (hkv * batch)))
    return {"op": op, "batch": batch, "len": length, "nq": nq, "hq": hkv * grp, "hkv": hkv, "d": d,
            "page": page, "block": block, "topk": topk, "shared": rng.random() < 0.4, "dt": dt}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _spread(case, most, least=1):
    """Lengths of a batch's requests: the first has `most`, the others up to a third less."""
    return [max(least, most - (most // 3) * r // max(1, case["batch"]) - (r % 7 if r else 0))
            for r in range(case["batch"])]


# ------------------------------------------------------------------- the inputs
def _normal(gen, shape, dt):
    return (torch.randn(shape, generator=gen, device=DEV) * _SCALE).to(dt)


def _pow2_quantise(x):
    """Rows of x in e4m3 and their power-of-two scales in e8m0; a row that holds a value that is
    not finite has scale NaN and zeros."""
    x = x.float()
    top = x.abs().amax(dim=-1)
    fine = torch.isfinite(x).all(dim=-1)
    mant, ex = torch.frexp(torch.where(fine, top, torch.zeros_like(top)))
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    # 2^-e by two exact factors: neither leaves the range of 32-bit numbers
    h = torch.div(-e, 2, rounding_mode="floor")
    y = torch.ldexp(torch.ldexp(x, h[..., None]), (-e - h)[..., None])
    lim = torch.where(e >= 120, 240.0, 448.0)[..., None]  # 2^120 * 256 is no 32-bit number
    y = torch.where(fine[..., None], torch.minimum(torch.maximum(y, -lim), lim), 0.0)
    byte = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return y.to(torch.float8_e4m3fn), byte.view(torch.float8_e8m0fnu)


def _widen(codes, scales):
    """What the cache's bytes stand for, 32 bits."""
    byte = scales.view(torch.uint8).to(torch.int32)
    bits = torch.where(byte == 0, 0x00400000, byte << 23)
    s = torch.where(byte == 255, float("nan"), bits.view(torch.float32))
    return codes.to(torch.float32) * s[..., None]


def _prepare_grad(case, gen, dt):
    lens = _lens(case)
    T, S, b = sum(lens), max(lens), len(lens)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"q": _normal(gen, (T, hq, d), dt), "k": _normal(gen, (T, hkv, d), dt),
         "v": _normal(gen, (T, hkv, d), dt), "dout": _normal(gen, (T, hq, d), dt),
         "max": S, "batch": b}
    ln = torch.tensor(lens)
    cu = torch.zeros(b + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(ln, 0)
    s["cu"] = cu.to(DEV, torch.int32)
    j = torch.arange(S)
    inside = j[None, :] < ln[:, None]
    s["gather"] = torch.where(inside, cu[:-1, None] + j[None, :], 0).to(DEV)  # [b, S] -> token
    s["inside"] = inside.to(DEV)
    s["back"] = torch.nonzero(inside.reshape(-1)).reshape(-1).to(DEV)         # token -> b * S + j
    s["mask"] = (j[None, :] <= j[:, None]).to(DEV)
    q, k, v = _padded(s, "q"), _padded(s, "k"), _padded(s, "v")
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    x.masked_fill_(~s["mask"], float("-inf"))
    lse = torch.logsumexp(x, dim=-1)
    out = torch.matmul(x.sub_(lse[..., None]).exp_(), v)
    s["out"] = _packed(s, out).to(dt)
    s["lse"] = _packed(s, lse[..., None])[..., 0].contiguous()
    return s


def _padded(s, name):
    """A packed [T, H, d] input as [batch, kv heads, group, S, d], 32 bits, zeros behind a sequence."""
    x = s[name][s["gather"]].float() * s["inside"][:, :, None, None]
    b, S, H, d = x.shape
    hkv = s["k"].shape[1]
    return x.permute(0, 2, 1, 3).reshape(b, hkv, H // hkv, S, d)


def _packed(s, x):
    """[batch, kv heads, group, S, d] back to packed [T, H, d]."""
    b, hkv, grp, S, d = x.shape
    return x.reshape(b, hkv * grp, S, d).permute(0, 2, 1, 3).reshape(b * S, hkv * grp, d)[s["back"]]


def _make_cache(case, lens, gen, block, filled):
    """A page pool with shuffled pages; `filled`: it holds drawn keys with block offsets, else
    drawn bytes."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(gen.initial_seed() + 1))
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n].to(torch.int32)
        at += n
    shape = (pages, hkv, page, d)
    s = {"table": table.to(DEV), "page": page, "order": order, "need": need,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    k = _normal(gen, shape, torch.float32)
    if filled:
        # one offset for each block of a request: its pages share it where a block is whole pages
        per = max(1, block // page)
        off = torch.randn((pages // per + 1, hkv, 1, d), generator=gen, device=DEV) * _OFFSET
        where = torch.empty(pages, dtype=torch.int64)
        where[order] = torch.arange(pages)
        k += off[(where // per).to(DEV)]
    s["k8"], s["ks"] = _pow2_quantise(k)
    del k
    s["v8"], s["vs"] = _pow2_quantise(_normal(gen, shape, torch.float32))
    return s


def _library():
    import long_context_prefill_block_b200 as moba

    return moba


def _handle(s):
    moba = _library()
    return moba.MobaCache(s["k8"], s["v8"], s["ks"], s["vs"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _DT[case["dt"]]
    op = case["op"]
    if op == "grad":
        s = _prepare_grad(case, gen, dt)
    elif op in ("write", "read"):
        new = _spread(case, case["new"])
        old = _spread(case, case["old"], 0)
        lens = [a + b for a, b in zip(old, new)]
        s = _make_cache(case, lens, gen, 1, False)
        cu = torch.zeros(len(new) + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(torch.tensor(new), 0)
        s["cu"], s["rows"] = cu.to(DEV, torch.int32), int(cu[-1])
        if op == "write":
            s["block"] = B = case["block"]
            s["k"] = _normal(gen, (s["rows"], case["hkv"], case["d"]), dt)
            s["v"] = _normal(gen, (s["rows"], case["hkv"], case["d"]), dt)
            nb = max(1, -(-max(lens) // B))
            s["kbar"] = _normal(gen, (len(lens), nb, case["hkv"], case["d"]), torch.float32)
            done = [(r, i) for r in range(len(lens)) for i in range(old[r] // B, lens[r] // B)]
            s["done"] = torch.tensor(done, dtype=torch.int64).reshape(-1, 2).to(DEV)
    else:
        lens = _spread(case, case["len"], case["nq"])
        s = _make_cache(case, lens, gen, case["block"], True)
        n, B = case["nq"] * case["batch"], case["block"]
        s["q"] = _normal(gen, (n, case["hq"], case["d"]), dt)
        s["cu"] = torch.arange(0, n + 1, case["nq"], dtype=torch.int32, device=DEV)
        s["block"], s["topk"], s["shared"], s["max"] = B, case["topk"], case["shared"], max(lens)
        nb = max(1, -(-s["max"] // B))
        s["kbar"] = torch.zeros((len(lens), nb, case["hkv"], case["d"]), device=DEV)
        for r, L in enumerate(lens):  # whole blocks' means of what the cache holds
            m = L // B
            if m:
                rows = _positions(s, torch.full((1,), r, device=DEV),
                                  torch.arange(m * B, device=DEV)[None])
                k = _widen(*_rows(s["k8"], s["ks"], rows))[0]
                s["kbar"][r, :m] = k.reshape(m, B, case["hkv"], case["d"]).mean(dim=1)
    s["op"], s["dt"] = op, dt
    return s


# --------------------------------------------------------------- the plain forms
def _positions(s, req, pos):
    """(page, place in it) of positions `pos` [n, m] of requests `req` [n]."""
    page = s["table"].long()[req[:, None], pos // s["page"]]
    return page, pos % s["page"]


def _rows(codes, scales, at):
    """Codes [n, m, kv heads, d] and scales [n, m, kv heads] of the rows at (page, place)."""
    page, place = at
    c = codes.view(torch.uint8).transpose(1, 2)[page, place].view(torch.float8_e4m3fn)
    return c, scales.view(torch.uint8).transpose(1, 2)[page, place].view(torch.float8_e8m0fnu)


def _new_rows(s):
    """(page, place) of each new or tail row, in the order of the packed rows."""
    row = torch.arange(s["rows"], device=DEV)
    cu = s["cu"].long()
    req = torch.searchsorted(cu[1:], row, right=True)
    n = cu[1:] - cu[:-1]
    pos = s["lens"].long()[req] - n[req] + row - cu[req]
    page = s["table"].long()[req, pos // s["page"]]
    return page, pos % s["page"]


def _plain_grad(s):
    d = s["q"].shape[2]
    scale = 1.0 / math.sqrt(d)
    q, k, v, do = (_padded(s, x) for x in ("q", "k", "v", "dout"))
    lse = _padded({**s, "lse3": s["lse"][..., None]}, "lse3")
    D = (do * _padded(s, "out")).sum(dim=-1, keepdim=True)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).sub_(lse)
    p = p.masked_fill_(~s["mask"], float("-inf")).exp_()
    dv = torch.matmul(p.transpose(-1, -2), do).sum(dim=2, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(D).mul_(p)
    del p
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(dim=2, keepdim=True).mul_(scale)
    return tuple(_packed(s, x).to(s["dt"]) for x in (dq, dk, dv))


def _plain_write(s):
    page, place = _new_rows(s)
    for new, codes, scales in ((s["k"], s["k8"], s["ks"]), (s["v"], s["v8"], s["vs"])):
        c, e = _pow2_quantise(new)
        codes.view(torch.uint8).transpose(1, 2)[page, place] = c.view(torch.uint8)
        scales.view(torch.uint8).transpose(1, 2)[page, place] = e.view(torch.uint8)
    req, blk = s["done"][:, 0], s["done"][:, 1]
    if req.numel():  # the means of the blocks that these rows complete, of what the cache holds
        B = s["block"]
        pos = blk[:, None] * B + torch.arange(B, device=DEV)
        k = _widen(*_rows(s["k8"], s["ks"], _positions(s, req, pos)))
        s["kbar"][req, blk] = k.mean(dim=1)


def _plain_read(s):
    page, place = _new_rows(s)
    at = (page[None], place[None])
    return tuple(_widen(*_rows(c, e, at))[0].to(s["dt"])
                 for c, e in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))


def _plain_decode(s):
    q = s["q"].float()
    n, hq, d = q.shape
    hkv, B, topk = s["k8"].shape[1], s["block"], s["topk"]
    grp, cu = hq // hkv, s["cu"].long()
    req = torch.searchsorted(cu[1:], torch.arange(n, device=DEV), right=True)
    p = s["lens"].long()[req] - (cu[1:] - cu[:-1])[req] + torch.arange(n, device=DEV) - cu[req]
    c = p // B
    # scores next to a border decide which block is read: 64 bits
    qg = q.double().reshape(n, hkv, grp, d)
    if s["shared"]:
        qg = qg.sum(dim=2, keepdim=True).expand(-1, -1, grp, -1)
    score = torch.einsum("ngjd,nbgd->ngjb", qg, s["kbar"].double()[req]).reshape(n, hq, -1)
    nb = score.shape[2]
    if nb < topk:
        score = torch.cat([score, score.new_zeros(n, hq, topk - nb)], dim=2)
    blocks = torch.arange(score.shape[2], device=DEV)
    score = score.masked_fill(blocks >= c[:, None, None], float("-inf"))
    score = score.masked_fill(blocks == c[:, None, None], float("inf"))
    order = torch.sort(score, dim=2, descending=True, stable=True)[1][:, :, :topk]
    none = torch.iinfo(torch.int64).max
    idx = torch.where(order <= c[:, None, None], order, none).sort(dim=2)[0]
    idx = torch.where(idx == none, -1, idx)
    pos = idx[..., None] * B + torch.arange(B, device=DEV)           # [n, hq, topk, B]
    seen = (idx[..., None] >= 0) & (pos <= p[:, None, None, None])
    pos = torch.where(seen, pos, 0).reshape(n, hq, -1)
    seen = seen.reshape(n, hq, -1)
    page = s["table"].long()[req[:, None, None], pos // s["page"]]
    head = (torch.arange(hq, device=DEV) // grp)[None, :, None]
    at = (page, head, pos % s["page"])
    k = _widen(s["k8"].view(torch.uint8)[at].view(torch.float8_e4m3fn),
               s["ks"].view(torch.uint8)[at].view(torch.float8_e8m0fnu))
    x = torch.matmul(k, q[..., None])[..., 0] * (1.0 / math.sqrt(d))
    del k
    x = x.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(x, dim=2)
    w = torch.exp(x - lse[..., None])
    v = _widen(s["v8"].view(torch.uint8)[at].view(torch.float8_e4m3fn),
               s["vs"].view(torch.uint8)[at].view(torch.float8_e8m0fnu))
    out = torch.matmul(w[:, :, None, :], v)[:, :, 0]
    return out.to(s["dt"]), lse, idx.to(torch.int32)


def run(state):
    s, op = state, state["op"]
    if op == "grad":
        if own:
            return _library().dense_causal_backward(s["q"], s["k"], s["v"], s["cu"], s["out"],
                                                    s["lse"], s["dout"], max_seqlen=s["max"])
        return _plain_grad(s)
    if op == "write":
        if own:
            _library().moba_cache_write(_handle(s), s["k"], s["v"], s["table"], s["lens"], s["cu"],
                                        kbar=s["kbar"], block_size=s["block"])
        else:
            _plain_write(s)
        return {"k": s["k8"], "v": s["v8"], "k_scale": s["ks"], "v_scale": s["vs"],
                "kbar": s["kbar"]}
    if op == "read":
        if own:
            return _library().moba_cache_read(_handle(s), s["table"], s["lens"], s["cu"],
                                              s["rows"], dtype=s["dt"])
        return _plain_read(s)
    if own:
        return _library().moba_decode_cache(s["q"], _handle(s), s["table"], s["lens"], s["cu"],
                                            s["kbar"], s["block"], s["topk"], max_seqlen=s["max"],
                                            shared_routing=s["shared"], return_lse=True,
                                            return_idx=True)
    return _plain_decode(s)


# ------------------------------------------------------------------- its work
def work(case):
    d, hkv = case["d"], case["hkv"]
    e = 2 if case["dt"] == "bf16" else 4
    if case["op"] == "grad":
        lens, hq = _lens(case), case["hq"]
        T = sum(lens)
        # q, out, dout read and dq written; k, v read and dk, dv written; lse
        return {"bytes": T * d * e * (4 * hq + 4 * hkv) + 4 * T * hq,
                "flops": sum(5 * 2 * d * hq * n * (n + 1) // 2 for n in lens)}
    if case["op"] in ("write", "read"):
        rows = sum(_spread(case, case["new"])) * hkv
        b = 2 * rows * (d * e + d + 1)
        f = 4 * rows * d
        if case["op"] == "write":
            B = case["block"]
            old = _spread(case, case["old"], 0)
            new = _spread(case, case["new"])
            done = sum((a + n) // B - a // B for a, n in zip(old, new))
            before = sum(a - a // B * B for a, n in zip(old, new) if (a + n) // B > a // B)
            b += done * hkv * d * 4 + before * hkv * (d + 1)
            f += 2 * rows * d
        return {"bytes": b, "flops": f}
    hq, B, k, nq = case["hq"], case["block"], case["topk"], case["nq"]
    grp = hq // hkv
    b = f = 0
    for L in _spread(case, case["len"], nq):
        c = (L - 1) // B
        far = min(k - 1, c) * B
        near = L - c * B
        # a kv head's rows: the own block once, the chosen blocks once for each head and query
        # that may choose its own, but no row of the cache twice
        picks = nq * (1 if case["shared"] else grp)
        rows = near + min(far * picks, c * B)
        b += hkv * (rows * 2 * (d + 1) + c * d * 4) + 2 * nq * hq * d * e
        f += nq * hq * (2 * d * c + 4 * d * (far + near))
    return {"bytes": b, "flops": f}


# --------------------------------------------------- the definitions in 64 bits
def _value64(codes, scales):
    """What bytes of the cache stand for, from their bits."""
    c = codes.view(torch.uint8).to(torch.int64)
    ex, man = (c >> 3) & 15, c & 7
    mag = torch.where(ex == 0, man.double() * 2.0 ** -9,
                      (8 + man).double() * torch.exp2((ex - 10).double()))
    mag = torch.where((c & 127) == 127, float("nan"), mag)
    b = scales.view(torch.uint8).to(torch.int64)
    s = torch.where(b == 255, float("nan"), torch.exp2((b - 127).double()))
    return torch.where(c >= 128, -mag, mag) * s[..., None]


def _round_e4m3(x):
    """Nearest e4m3 value of 64-bit x with |x| <= 448, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "grad":
        lens, hq, d = _lens(case), case["hq"], case["d"]
        if sum(n * n for n in lens) * hq * 10 * d > 8e12:
            return None
        grp = hq // case["hkv"]
        dq = torch.zeros_like(s["q"], dtype=torch.float64)
        dk, dv = (torch.zeros_like(s["k"], dtype=torch.float64) for _ in range(2))
        t0 = 0
        for n in lens:
            at = slice(t0, t0 + n)
            t0 += n
            later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
            for h in range(hq):
                q, o, g = (s[x][at, h].double() for x in ("q", "out", "dout"))
                k, v = (s[x][at, h // grp].double() for x in ("k", "v"))
                p = torch.exp(q @ k.T / math.sqrt(d) - s["lse"][at, h].double()[:, None])
                p[later] = 0.0
                dv[at, h // grp] += p.T @ g
                p *= g @ v.T - (g * o).sum(dim=1, keepdim=True)
                dq[at, h] = p @ k / math.sqrt(d)
                dk[at, h // grp] += p.T @ q / math.sqrt(d)
        return dq, dk, dv
    table, lens, cu = s["table"].cpu(), s["lens"].cpu().tolist(), s["cu"].cpu().tolist()
    page = case["page"]

    def places(r, first, last):
        pos = torch.arange(first, last)
        return (table[r, pos // page].long() * page + pos % page).to(DEV)

    if op in ("write", "read"):
        flat = lambda x: x.transpose(1, 2).flatten(0, 1)  # noqa: E731  [pages * page, kv heads, ...]
        tail = [places(r, lens[r] - (cu[r + 1] - cu[r]), lens[r]) for r in range(len(lens))]
        at = torch.cat(tail)
        if op == "read":
            return tuple(_value64(flat(c.view(torch.uint8))[at], flat(e.view(torch.uint8))[at])
                         for c, e in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))
        res = {}
        one = torch.zeros(1, dtype=torch.uint8, device=DEV)
        for name, codes, scales in (("k", s["k8"], s["ks"]), ("v", s["v8"], s["vs"])):
            u = scales.view(torch.uint8)
            got_c = flat(_value64(codes, (one + 127).expand(u.shape))).clone()
            got_s = flat(torch.exp2(u.double() - 127)).clone()
            x = s[name].double()
            top = x.abs().amax(dim=-1)
            e = torch.ceil(torch.log2(top / 448)).clamp(min=-127, max=120)
            e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
            e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
            got_c[at] = _round_e4m3(x / torch.exp2(e)[..., None])
            got_s[at] = torch.exp2(e)
            res[name] = got_c
            res[name + "_scale"] = got_s
        value = res["k"] * res["k_scale"][..., None]
        kbar, B = s["kbar"].double(), case["block"]
        for r, i in s["done"].cpu().tolist():
            kbar[r, i] = value[places(r, i * B, (i + 1) * B)].mean(dim=0)
        pages = s["k8"].shape[0]
        for name in ("k", "v", "k_scale", "v_scale"):
            res[name] = res[name].unflatten(0, (pages, page)).transpose(1, 2).contiguous()
        return {**res, "kbar": kbar}
    n, hq, d = s["q"].shape
    hkv, B, topk = case["hkv"], case["block"], case["topk"]
    grp = hq // hkv
    if n * hq * topk > 8192:
        return None
    q = s["q"].double()
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(n, hq, dtype=torch.float64, device=DEV)
    flat = lambda x: x.view(torch.uint8).transpose(0, 1).flatten(1, 2)  # noqa: E731
    k8, v8, ks, vs = (flat(s[x]) for x in ("k8", "v8", "ks", "vs"))
    for r, L in enumerate(lens):
        m = cu[r + 1] - cu[r]
        for i in range(m):
            row, p = cu[r] + i, L - m + i
            c = p // B
            x = torch.einsum("gjd,bgd->gjb", q[row].reshape(hkv, grp, d), s["kbar"][r, :c].double())
            if case["shared"]:
                x = x.mean(dim=1, keepdim=True).expand(-1, grp, -1)
            x = x.reshape(hq, c).cpu()
            for h in range(hq):
                ranked = sorted(range(c), key=lambda b: (-float(x[h, b]), b))[:topk - 1]
                at = torch.cat([places(r, b * B, (b + 1) * B) for b in sorted(ranked)]
                               + [places(r, c * B, p + 1)])
                k, v = _value64(k8[h // grp, at], ks[h // grp, at]), _value64(v8[h // grp, at],
                                                                              vs[h // grp, at])
                z = k @ q[row, h] / math.sqrt(d)
                lse[row, h] = torch.logsumexp(z, 0)
                out[row, h] = torch.exp(z - lse[row, h]) @ v
    return out, lse, None
