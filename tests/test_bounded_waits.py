"""A wait on an mbarrier is bounded: when its time runs out, lanes of one warp can
come back with different answers.  Where the answer steers a whole warp -- which
then issues warp-wide tensor-memory instructions or shuffles -- the warp has to
agree on it first.  Read from the product kernels' sources (no GPU: the wait must
not be made to run out in a kernel that would then misbehave)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_gemm_12_gb300",
                    "csrc")
# an answer that is kept: name = ... mbar_wait_at(...) ...;
KEPT = re.compile(r"\b(\w+) =\s[^;=]*\bmbar_wait_(?:at|late)\([^;]*;")


def statements(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [(m.group(1), m.group(0), text[m.end():m.end() + 250]) for m in KEPT.finditer(text)]


@pytest.mark.parametrize("name,count", [("fp8_tc.cu", 3), ("grouped_tc.cu", 5)])
def test_a_warp_agrees_on_the_outcome_of_a_wait(name, count):
    found = statements(name)
    assert len(found) == count
    for var, statement, after in found:
        voted = "_sync(0xffffffffu" in statement
        asked = re.search(r"(__any_sync\(0xffffffffu, !%s\)|named_bar_any\(\w+, \w+, !%s\))" % (var, var), after)
        assert voted or asked, statement


def test_a_warp_is_together_at_the_barrier_after_a_wait():
    # the barrier that collects the answers of several warps is itself warp-wide
    with open(os.path.join(CSRC, "ptx.cuh")) as f:
        text = f.read()
    body = text[text.index("bool named_bar_any("):]
    body = body[:body.index("\n}\n")]
    assert "bar.red" in body and body.index("__syncwarp()") < body.index("asm volatile")
