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
