"""CPU checks, on the sources, of two rules that no GPU run can show broken for certain.

1. A warp's arrival at a counter in global memory (lane 0 counts, all lanes then read what other
   warps wrote) has a warp barrier on both sides: a shuffle orders no memory. There is one function
   for it.
2. Block barriers for part of a block (bar.sync and its kin) are for warps whose lanes are together;
   each helper that issues one brings them together first."""
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
    assert len(re.findall("named_bar_sync", block)) == 2 and "count_global" in block


def test_partial_block_barriers_are_reached_by_whole_warps():
    asm = re.compile(r'"[^"]*\bbar(?:rier)?\.(?:cta\.)?(?:sync|arrive|red)\b')
    helpers = {"common.cuh": ["named_bar_sync", "named_bar_any"], "stream.cuh": ["named_bar_arrive"]}
    for name, src in _sources().items():
        names = helpers.get(name, [])
        assert len(asm.findall(src)) == len(names), name
        for helper in names:
            body = _body(src, helper)
            assert body.index("__syncwarp()") < asm.search(body).start(), (name, helper)
