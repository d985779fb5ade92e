"""CPU checks, on the sources, of two rules that no GPU run can show broken for certain.

1. A warp's arrival at a counter in global memory (lane 0 counts, all lanes then read what other
   warps wrote) has a warp barrier on both sides: a shuffle orders no memory. There is one function
   for it.
2. Block barriers for part of a block (bar.sync and its kin) are for warps whose lanes are together:
   a warp barrier stands before each."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "top_routing_expert_fp32_b200", "csrc")


def _sources():
    return {os.path.basename(f): open(f).read()
            for f in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))}


def _body(src, name):
    """The body of the first function of that name."""
    m = re.search(r"\b%s\([^;{]*\)\s*\{" % name, src)
    assert m, name
    depth, i = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        i += 1
    return src[m.end():i]


def test_arrivals_of_a_warp_have_barriers_on_both_sides():
    sources = _sources()
    body = _body(sources["stream.cuh"], "last_warp_to_arrive")
    count, barriers = body.index("count_global"), [m.start() for m in
                                                  re.finditer(r"__syncwarp\(\)", body)]
    shuffle = body.index("__shfl_sync")
    assert barriers[0] < count < shuffle < barriers[-1] < body.index("return")
    # Nobody else counts one lane's arrival and hands it to the others: the block's form has block
    # barriers on both sides.
    callers = [(name, m.start()) for name, src in sources.items()
               for m in re.finditer(r"\bcount_global\(", src)]
    assert {name for name, _ in callers} == {"stream.cuh"} and len(callers) == 3
    block = _body(sources["stream.cuh"], "last_to_finish")
    assert len(re.findall("bar_sync", block)) == 2 and "count_global" in block


def test_partial_block_barriers_are_reached_by_whole_warps():
    asm = re.compile(r'"[^"]*\bbar(?:rier)?\.(?:cta\.)?(?:sync|arrive|red)\b')
    call = re.compile(r"(\w[^\n]*\n[ ]*)?(?:if \()?\bnamed_bar_(?:sync|any)\((?!uint32_t)")
    for name, src in _sources().items():
        # The instructions themselves: in common.cuh's two helpers and stream.cuh's arrival.
        assert len(asm.findall(src)) == {"common.cuh": 2, "stream.cuh": 1}.get(name, 0), name
        for m in call.finditer(src):
            assert (m.group(1) or "").split() == ["__syncwarp();"], (name, m.group(0))
    body = _body(_sources()["stream.cuh"], "bar_arrive")
    assert body.index("__syncwarp()") < asm.search(body).start()
