"""The kernels' waits, checked in their source: whether a bounded wait gave up is decided by one lane that tells the others
or by a vote of the warp, never by each lane for itself (lanes that leave alone strand the others in a full-mask shuffle)."""
import glob
import os
import re

import pytest

from paged_kv_cache_185_gb300 import build

WAIT = re.compile(r"\b(?:mbar_wait_bounded|mbar_wait_sleep|counter_wait_bounded)\s*\(")


def waits(path):
    """(line number, statement) of every bounded wait of a file, definitions and comments aside."""
    for number, line in enumerate(open(path), 1):
        code = line.split("//")[0]
        if WAIT.search(code) and "__device__" not in code:
            yield number, code.strip()


@pytest.mark.parametrize("name", ["sparse_decode.cu", "rotate_kernel.cuh"])
def test_no_lane_gives_up_alone(name):
    for number, code in waits(os.path.join(build.CSRC, name)):
        # what is left of lanes' own waits only lets copies in flight land: nothing depends on their result
        assert re.match(r"(if \(coming\) |for \(.*\) )?mbar_wait_bounded\(.*\);$", code), f"{name}:{number}: {code}"


def test_the_warps_wait_votes():
    text = open(os.path.join(build.CSRC, "common.cuh")).read()
    body = text[text.index("bool mbar_wait_warp("):]
    assert "__all_sync(kFullMask, got)" in body[:body.index("\n}")]
    users = [f for f in glob.glob(os.path.join(build.CSRC, "*.cu*")) if "mbar_wait_warp(smem" in open(f).read()]
    assert users


@pytest.mark.parametrize("name", ["decode_persistent.cuh", "decode_kernel.cuh", "prefill.cu", "prefill_tc.cu"])
def test_no_branch_on_a_lanes_own_wait(name):
    """In the decode and prefill kernels one lane waits for the warp (and tells it), the warp votes, or only copies in
    flight are let land."""
    text = open(os.path.join(build.CSRC, name)).read()
    for number, code in waits(os.path.join(build.CSRC, name)):
        assert not re.match(r"if \(!", code), f"{name}:{number}: {code}"
        if re.match(r"const bool (ok|got) = mbar_wait_bounded", code):
            after = "\n".join(text.split("\n")[number:number + 3])
            assert "__all_sync(kFullMask, got)" in after, f"{name}:{number}: {code}"
