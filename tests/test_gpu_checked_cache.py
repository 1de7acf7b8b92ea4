"""The dense gradient and the 8-bit cache through the bounds-checked build: no check fires on valid
inputs, and the results are the ordinary build's, bit for bit (the sources are the same)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import long_context_prefill_block_b200 as moba
from long_context_prefill_block_b200 import build
if {checked}:
    moba.use_library(build.LIB_CHECKED)
g = torch.Generator().manual_seed(1)
res = []
for dtype, d in ((torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)):
    mk = lambda n, h: (torch.randn(n, h, d, generator=g) * 0.7).to(dtype).cuda()
    lens = [300, 0, 131]
    cu = torch.tensor([0, 300, 300, 431], dtype=torch.int32, device="cuda")
    q, k, v, do = mk(431, 4), mk(431, 2), mk(431, 2), mk(431, 4)
    out, lse = moba.dense_causal_forward(q, k, v, cu, max_seqlen=300, return_lse=True)
    res += moba.dense_causal_backward(q, k, v, cu, out, lse, do, max_seqlen=300)
    c = moba.moba_cache_alloc(40, 16, 2, d)
    order = torch.randperm(40, generator=g).int()
    table = torch.zeros(3, 20, dtype=torch.int32)
    table[0, :19], table[2, :9] = order[:19], order[19:28]
    table = table.cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kbar = torch.zeros(3, 7, 2, d, device="cuda")
    moba.moba_cache_write(c, k, v, table, ln, cu, kbar, 50)
    res += moba.moba_cache_read(c, table, ln, cu, 431, dtype=dtype)
    one = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda")
    res += moba.moba_decode_cache(mk(2, 4), c, table, ln, one, kbar, 50, 3, return_lse=True,
                                  return_idx=True)
    res.append(kbar)
    torch.cuda.synchronize()
    assert moba.moba_device_status() == 0
torch.save([x.cpu() for x in res], sys.argv[1])
"""


def test_checked_build_agrees(tmp_path):
    import torch

    got = []
    for checked in (False, True):
        out = str(tmp_path / f"{checked}.pt")
        subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, checked=checked), out],
                       check=True, timeout=300)
        got.append(torch.load(out))
    assert len(got[0]) == len(got[1]) and all(torch.equal(a, b) for a, b in zip(*got))


# (heads q / kv, d, dtype, lengths, new rows, page, block, topk, shared): sums of 32 rows and their
# means by clusters, by CTAs and by warps; choice inside a split, by a launch of its own, by lists;
# splits of several blocks and several splits a block; no block to choose
LONG = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import long_context_prefill_block_b200 as moba
from long_context_prefill_block_b200 import build
if {checked}:
    moba.use_library(build.LIB_CHECKED)
bf16, fp32 = torch.bfloat16, torch.float32
res = []
for hq, hkv, d, dtype, lens, new, page, B, topk, shared in (
        (16, 8, 128, bf16, [9000, 4000], [8000, 3999], 64, 1024, 3, False),
        (8, 8, 64, fp32, [9000, 31, 2000], [9000, 0, 1999], 16, 500, 12, True),
        (24, 8, 64, bf16, [10000, 70], [9990, 70], 32, 48, 32, False),
        (20, 2, 128, bf16, [3000, 2999], [3000, 1], 128, 20, 5, True),
        (4, 2, 128, fp32, [3000, 17], [1000, 17], 1024, 20, 5, False),
        (6, 1, 64, bf16, [50000, 9], [100, 9], 64, 1, 3, False),
        (4, 4, 128, bf16, [30000], [40], 64, 30000, 1, True)):
    g = torch.Generator().manual_seed(1)
    mk = lambda n, h: (torch.randn(n, h, d, generator=g) * 0.7).to(dtype).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    off = lambda x: i32([0] + torch.tensor(x).cumsum(0).tolist())
    need = [-(-n // page) for n in lens]
    order, table = torch.randperm(sum(need), generator=g).int(), torch.full((len(lens), max(need)), -1)
    for r, n in enumerate(need):
        table[r, :n] = order[sum(need[:r]):sum(need[:r]) + n]
    table, c = table.int().cuda(), moba.moba_cache_alloc(sum(need), page, hkv, d)
    kbar = torch.zeros(len(lens), -(-max(lens) // B), hkv, d, device="cuda")
    old = [a - b for a, b in zip(lens, new)]
    for length, rows in ((old, old), (lens, new)):
        n = sum(rows)
        moba.moba_cache_write(c, mk(n + 3, hkv), mk(n + 3, hkv), table, i32(length), off(rows), kbar, B)
    nq = [2 if x else 0 for x in new]
    n = sum(nq)
    out = torch.zeros(n + 2, hq, d, dtype=dtype, device="cuda")
    _, lse, idx = moba.moba_decode_cache(mk(n + 2, hq), c, table, i32(lens), off(nq), kbar, B, topk,
                                         shared_routing=shared, return_lse=True, return_idx=True,
                                         out=out)
    res += [out, lse[:n], idx[:n], kbar]
    k, v = moba.moba_cache_read(c, table, i32(lens), off(lens), sum(lens), dtype=dtype)
    res += [k, v]
    torch.cuda.synchronize()
    assert moba.moba_device_status() == 0, (hq, hkv, d, lens)
torch.save([x.cpu() for x in res], sys.argv[1])
"""


def test_checked_build_agrees_on_long_calls(tmp_path):
    import torch

    got = []
    for checked in (False, True):
        out = str(tmp_path / f"{checked}.pt")
        subprocess.run([sys.executable, "-c", LONG.format(root=ROOT, checked=checked), out],
                       check=True, timeout=300)
        got.append(torch.load(out))
    assert len(got[0]) == len(got[1]) and all(torch.equal(a, b) for a, b in zip(*got))
    assert not any(x.isnan().any() for x in got[0] if x.is_floating_point())
