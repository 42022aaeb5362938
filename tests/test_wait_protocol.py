"""The bounded waits of the kernels that stream through shared memory (GEMMs,
adapters), as far as their sources show it (CPU).

A wait that gives up must leave the CTA in a state from which every role still
ends.  The time limit is seconds away from what a copy takes, so ordinary runs
never come there."""
import os
import re

import pytest

from nvfp4_block_quantization_amax_b200 import build

FILES = ("gemm.cu", "grouped_gemm.cu", "lora.cu")


def source(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", FILES)
def test_whole_warps_wait_with_one_answer(name):
    """What a whole warp waits for (an accumulator, a filled slot) is asked for
    with mbar_wait_warp: lanes that disagreed about the time limit would part
    in front of warp-wide instructions.  mbar_wait itself is left to single
    lanes: producers (empty slots) and MMA issuers (full slots, drained
    accumulators)."""
    text = source(name)
    for args in re.findall(r"\bmbar_wait\(([^;]*?), abort(?:_flag)?[,)]", text):
        assert re.search(r"empty|&full\[s\]", args), args
    whole = re.findall(r"\bmbar_wait_warp\(([^;]*?), abort(?:_flag)?[,)]", text)
    assert whole and all("acc_full" in a or "&full[slot]" in a for a in whole)


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


def test_adapters_outer_consumers_all_meet_at_their_barrier():
    """The consumer warps of the outer products meet at a named barrier in
    tiles of several adapters.  A warp whose wait has given up must come there
    too: another one may still have seen its data and be waiting."""
    text = source("lora.cu")
    kernel = text[text.index("lora_outer_kernel(const"):]
    loop = kernel[kernel.index("for (int k = 0; k < count; ++k) {"):kernel.index("release(&ring.empty[ring.slot]);")]
    before, after = loop.split("consumers_sync();")
    assert "wait_full(abort)" in before and "break" not in before and "continue" not in before
    assert "if (!ok) continue;" in after


def test_adapters_a_warp_that_gives_up_reports_it_itself():
    """Without a barrier behind the waits one thread cannot report for the
    others: it may have left before they give up."""
    text = source("lora.cu")
    for kernel in text.split("__global__")[1:]:
        for at in re.finditer(r"\*(?:o\.)?a\.status = kStatusTimeout", kernel):
            line = kernel[kernel.rindex("\n", 0, at.start()):at.start()]
            meets = kernel.rfind("__syncthreads();", 0, at.start()) > kernel.rfind("wait_full", 0, at.start())
            assert "!ok && lane == 0" in line or ("*abort" in line and meets), line
