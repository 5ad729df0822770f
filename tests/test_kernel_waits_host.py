"""Every kernel of the gated scan and the state cache is launched while the one before it may
still run, so each of its threads waits for that one before it can leave: a kernel that is done has
then waited for all before it, and so has what waits for this kernel."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mamba_ssd_scan_mixer_b200", "csrc")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "gated_scan*")) +
                       glob.glob(os.path.join(CSRC, "state_cache.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\s", text):
            body = text.index("{", m.end())
            name = re.findall(r"(\w+_kernel)\s*\(", text[m.end():body])[0]
            yield name, text[body:]


@pytest.mark.parametrize("name,body", list(_kernels()), ids=lambda v: v if "{" not in v else "")
def test_no_way_out_before_the_wait(name, body):
    wait = re.search(r"grid_dependency_wait\(\)|\bbegin<", body)
    assert wait is not None, name
    assert not re.search(r"\breturn\b", body[:wait.start()]), name


def test_the_shared_start_waits_on_every_way():
    with open(os.path.join(CSRC, "gated_scan_tiles.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("bool begin("):]
    assert "return" not in body[:body.index("grid_dependency_wait()")]


def test_marks_that_did_not_come_are_not_used():
    # a mark holds a sequence's number, an index into the states: where the wait for a stage's
    # copies ran out, the stage may hold anything
    seen = 0
    for name, body in _kernels():
        body = body.split("__global__")[0]
        if "mbar_wait_parked(&sm.full[s]" not in body:
            continue
        assert "const bool there = mbar_wait_parked(&sm.full[s]" in body, name
        for m in re.finditer(r"[^;{}]*\b(?:sm\.marks\[s\]\[first|marks\[lane\])", body):
            seen += 1
            inside = "there &&" in m.group(0) or re.search(r"if \(there && [^\n]*\{\n", body[:m.start()])
            assert inside, (name, m.group(0))
    assert seen == 3
