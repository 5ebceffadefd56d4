"""The matrix product's barrier waits, read from its source: what cannot be shown on a GPU without
a wait that runs out in the middle of a kernel."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_epilogue_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_are_a_whole_warp_s():
    """A bounded wait ends by the clock, lane by lane: what follows it is for whole warps (aligned loads of tensor memory,
    elections, barriers of the cluster), so all lanes have to take the same way out."""
    src = code("matmul.cu")
    assert not re.findall(r"\bmbar_(?:try_)?wait\w*\s*\(", src)
    assert len(re.findall(r"\bwarp_wait\(", src)) >= 8
    wait = re.search(r"bool warp_wait\([^)]*\)\s*\{(.*?)\}", code("umma.cuh"), re.S).group(1)
    assert "__all_sync(0xffffffffu, mbar_wait(" in wait
