"""The int8 kernels' waits: a warp agrees on an outcome that steers it, as in the other products
(read from the sources, without a GPU), and every loop that polls has a limit."""
import os
import re

import pytest

from test_bounded_waits import CSRC, statements


@pytest.mark.parametrize("name,count", [("int8_tc.cu", 3), ("int8_wide.cu", 4)])
def test_a_warp_agrees_on_the_outcome_of_a_wait(name, count):
    found = statements(name)
    assert len(found) == count
    for var, statement, after in found:
        asked = re.search(r"__any_sync\(0xffffffffu, !%s\)" % var, after)
        assert "_sync(0xffffffffu" in statement or asked, statement


@pytest.mark.parametrize("name", ["int8_tc.cu", "int8_wide.cu"])
def test_polling_loops_end(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"while \(!mbar_try_wait_at\(", text):
        assert "kWaitLimitNs) break;" in text[m.end():m.end() + 160]
    # no other wait than these and the bounded ones
    assert not re.search(r"while \((?!!mbar_try_wait_at)", text)
    assert "mbar_wait(" not in text
