"""Copies into shared memory and the waits for them, where one may expire; shares of registers.

A thread block may not end while a copy that it has requested can still land in its
shared memory: the memory may be another block's by then. A wait of another warp can
expire after the copying warp has issued its last copy, so the wait for the copies in
flight has to stand on every path to that warp's end. Read from the sources: no run
could show it without the race itself.
"""
import os
import re

import pytest

from speculative_decoding_verification_w12_gb300 import build as B

# The kernels that request copies: source, and the barriers that their copies complete on.
COPIES = {"w12_kv4_rows.cuh": ["full"], "w12_kv4_tile.cuh": ["raw_full"], "w12_logprobs.cu": ["s.full"],
          "w12_attn.cu": ["fullb"], "w12_gemm.cu": ["B.full"], "w12_grouped.cu": ["B.full", "B.full_x"]}


def enclosing(src, at):
    """Heads of the blocks and single statements that hold position `at`, innermost first."""
    heads, depth = [], 0
    lines = src[:at].split("\n")
    indent = len(lines[-1]) - len(lines[-1].lstrip())
    for line in reversed(lines[:-1]):
        text = line.strip()
        if not text or text.startswith(("//", "#")):
            continue
        own = len(line) - len(line.lstrip())
        if own < indent:
            heads.append(text)
            indent = own
            depth += 1
    return heads


@pytest.mark.parametrize("source", sorted(COPIES))
def test_copies_in_flight_are_waited_for_on_every_path(source):
    src = open(os.path.join(B.CSRC, source)).read()
    for bar in COPIES[source]:
        drains = list(re.finditer(r"mbar_wait\(&" + re.escape(bar) + r"\[[^;]*drain_limit_ns", src))
        assert drains, f"{source}: no wait for the copies of {bar}"
        for m in drains:
            kernel = src.rfind("__global__", 0, m.start())
            barrier = src.rfind("\n  cta_sync();", kernel, src.index("\n}\n", m.start()))
            if kernel < barrier < m.start():            # only other drains stand between
                assert not re.search(r"(?<!mbar_)\bwait\(", src[barrier:m.start()])
                continue
            heads = enclosing(src, m.start())
            assert not [h for h in heads if "abort" in h or "failed" in h], heads


def test_log_probabilities_free_no_stage_whose_copy_they_have_not_seen():
    """After an expired wait the computing warps go on to the block's barriers. A stage that
    they freed all the same would be filled again while its first copy is in flight, two
    requests on one phase of its barrier, which faults."""
    src = open(os.path.join(B.CSRC, "w12_logprobs.cu")).read()
    arrivals = re.findall(r"^(.*)mbar_arrive\(&s\.empty", src, re.M)
    assert arrivals and all("landed" in a for a in arrivals)
    assert re.search(r"mine = go && \w*(::)?mbar_wait\w*\(&s\.full\[st\]", src)
    assert re.search(r"landed = __all_sync\(0xFFFFFFFFu, mine\)", src)


def test_a_warpgroup_changes_its_registers_by_one_instruction():
    """Warps of one group that meet different instructions for it are undefined, and a sum of
    shares above the launch's registers waits for good."""
    src = open(os.path.join(B.CSRC, "w12_kv4_tile.cuh")).read()
    kernel = src[src.index("__global__"):]
    calls = re.findall(r"if \(([^)]*)\) \{\n(?:\s*//[^\n]*\n)*\s*(?:fewer|more)_registers<C::(\w+)>\(\)", kernel)
    assert calls == [("warp < 4", "kPlainRegs"), ("warp >= C::kRest", "kRestRegs"), ("warp >= 4", "kSoftRegs")]
    assert len(re.findall(r"(?:fewer|more)_registers<C::", kernel)) == 3
    regs = dict(re.findall(r"(k\w+Regs) = (\d+)", src))
    warps = {"kPlainRegs": 4, "kRestRegs": 8, "kSoftRegs": 8}
    assert sum(n * int(regs[k]) for k, n in warps.items()) <= 20 * int(regs["kLaunchRegs"])
    assert all(int(v) % 8 == 0 for v in regs.values())
