"""The command that runs one entry point on a seeded workload, on small shapes."""
import sys

import pytest

from long_context_prefill_block_b200 import run

pytestmark = pytest.mark.gpu

CALLS = ["dense", "dense_backward", "cache_write", "cache_read", "cache_decode"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("shape", [["--workload", "tiny_fp32"],
                                   ["--workload", "micro_32k", "--tokens", "2050",
                                    "--block-size", "500", "--page-size", "32", "--queries", "3"]])
def test_command(call, shape, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["run", "--call", call, "--iters", "1"] + shape)
    run.main()
    assert "status 0" in capsys.readouterr().out
