"""Rules that the kernels' sources keep and that no run shows broken reliably, checked on the text."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "long_context_prefill_block_b200", "csrc")


def source(name):
    """A kernel file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def arguments(text, call):
    """The argument text of every `call(...)`."""
    res = []
    for m in re.finditer(re.escape(call) + r"\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        res.append(text[m.end():at - 1])
    return res


# what the launch ahead of an overlapped one writes and the overlapped one reads, by its names
OVERLAPPED = [("dense_bwd_tc.cu", "stat|st|src"), ("cache.cu", r"sums|c\.ks?")]


@pytest.mark.parametrize("name,written", OVERLAPPED)
def test_results_of_an_overlapped_launch_are_read_by_ordinary_loads(name, written):
    """The read-only path (__ldg, or const __restrict__ parameters) is for memory that nothing writes
    while the kernel runs. A kernel that begins beside the launch it depends on is not that."""
    text = source(name)
    assert "grid_wait()" in text
    names = re.compile(rf"\b({written})\b")
    assert not [a for a in arguments(text, "__ldg") if names.search(a)]
    assert not re.search(rf"\bconst\s+\w+\s*\*\s*__restrict__\s+({written})\b", text)


@pytest.mark.parametrize("name", sorted(x for x in os.listdir(CSRC) if x.endswith(".cu")))
def test_shared_arrays_read_in_16_bytes_are_aligned_to_them(name):
    """An array of 4-byte elements is aligned to 4 bytes unless its declaration says more."""
    text = source(name)
    wide = set(re.findall(r"reinterpret_cast<(?:const )?(?:float4|uint4)\s*\*>\(&?(\w+)\s*[\[,)+]", text))
    for statement in re.findall(r"__shared__ ([^;]*);", text):
        names = set(re.findall(r"\b(\w+)\s*\[", statement)) & wide
        assert not names or "__align__" in statement, names


# accesses that the bounds-checked build is tested to keep inside, by the limits their checks name
CHECKED = {
    "cache.cu": [r"c\.max_pages", r"kMeanPages", r"\(dm\.T \+ 31\) / 32", r"dm\.nb", r"dm\.batch",
                 r"cache_holds\("],
    "decode_cache.cu": [r"c\.max_pages", r"\broom\b", r"kOwnGate", r"kGateScores", r"dm\.nb", r"dm\.topk",
                        r"dm\.batch", r"per_row|\* S\b", r"cache_holds\("],
    "dense_bwd.cu": [r"dm\.T"],
    "dense_bwd_tc.cu": [r"dm\.T"],
}


@pytest.mark.parametrize("name", CHECKED)
def test_the_checked_build_has_checks_to_fire(name):
    checks = arguments(source(name), "MOBA_CHECK")
    for limit in CHECKED[name]:
        assert [c for c in checks if re.search(limit, c)], limit
