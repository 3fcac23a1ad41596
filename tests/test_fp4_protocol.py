"""The 4-bit decode kernel's bounded waits (mla_decode_fp4_sm103a.cu), on the CPU.

A wait that ran out returns false to the lane that saw it; another lane of the warp may still see the phase end.  The
roles go on with warp-wide instructions (.sync.aligned, shuffles, votes), so whether a warp goes on is a vote's
result, never a lane's own.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_paged_gb300", "csrc")


def _source():
    with open(os.path.join(CSRC, "mla_decode_fp4_sm103a.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warp_leaves_by_a_vote():
    """Every test of a wait's result that decides control flow follows a vote over it."""
    text = _source()
    tests = list(re.finditer(r"if \(!(\w+)\)\s*(?:\{|break|continue|return)", text))
    waited = set(re.findall(r"\b(\w+) = mbar_wait\(", text))
    assert waited
    alone = [m for m in tests if m.group(1) in waited]
    assert alone, "no place left that this test looks at"
    for m in alone:
        last = re.findall(r"\b%s = ([^;]+);" % m.group(1), text[:m.start()])[-1]
        assert last.startswith("__all_sync("), f"line {text[:m.start()].count(chr(10)) + 1}: decided by `{last}`"
