"""The bounded waits of the kernels that stream through shared memory (GEMMs,
adapters), as far as their sources show it (CPU).

A wait that gives up must leave the CTA in a state from which every role still
ends.  The time limit is seconds away from what a copy takes, so ordinary runs
never come there."""
import os
import re

import pytest

from nvfp4_block_quantization_amax_b200 import build

GEMMS = ("gemm.cu", "grouped_gemm.cu")
FILES = GEMMS + ("lora.cu",)


def source(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", GEMMS)
def test_whole_warps_wait_with_one_answer(name):
    """What a whole warp waits for (an accumulator) is asked for with
    mbar_wait_warp: lanes that disagreed about the time limit would part in
    front of warp-wide instructions.  mbar_wait itself is left to single lanes:
    producers (empty slots) and MMA issuers (full slots, drained
    accumulators)."""
    text = source(name)
    for args in re.findall(r"\bmbar_wait\(([^;]*?), abort_flag\)", text):
        assert re.search(r"empty|&full\[s\]", args), args
    whole = re.findall(r"\bmbar_wait_warp\(([^;]*?), abort_flag\)", text)
    assert whole and all("acc_full" in a for a in whole)


@pytest.mark.parametrize("name", FILES)
def test_roles_wait_for_what_they_have_issued(name):
    """A role may finish before another one gives up, so a role's last wait,
    for the copies or products it has itself issued, cannot depend on the
    abort flag as it stands when the role finishes."""
    text = source(name)
    for cond in re.findall(r"if \(([^()]*abort[^()]*)\)", text):
        assert "status" in cond, cond                        # reporting alone
    if name == "lora.cu":
        assert len(re.findall(r"\.drain\(", text)) == 4      # shrink, expand (two rings), outer
    else:
        kernels = text.count("full[i %")
        assert kernels == 2 and len(re.findall(r"mbar_wait_bounded\(smem_u32\(drain\), 0\)", text)) == kernels


def test_adapters_consumers_go_on_in_step():
    """The consumer warps of the adapters' kernels execute warp-wide
    instructions after their waits and meet at named barriers, so a lane or a
    warp whose wait has given up must not leave: another one may still have
    seen its data and be waiting.  Nothing depends on a wait's answer; who gave
    up reports it at once, since its CTA has no barrier behind the waits at
    which another thread could report for it."""
    text = source("lora.cu")
    waits = [m.start() for m in re.finditer(r"\.wait_full\((?:v\.)?abort, (?:o\.)?a\.status\);", text)]
    assert len(waits) == 4 and text.count("wait_full(") == 5   # those and the definition
    assert text.count("kStatusTimeout") == 1                   # in it
    for at in waits:
        assert "break;" not in text[at:text.index("release(", at)]
