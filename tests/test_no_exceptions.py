"""What the library's host code allocates on the host is asked for where a failure is caught: no C++ exception
leaves a C entry point, whose caller could only end with it (read from the sources)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_gemm_12_gb300", "csrc")
# growing containers, a map's operator[], new, strings
ALLOCATES = r"\.(push_back|emplace_back|emplace|insert|resize|reserve)\(|\bscratch\[|\bnew \w|std::(to_)?string\b"


def host_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not path.endswith((".cu", ".cuh", ".h")):
            continue
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(ALLOCATES, text):
            yield os.path.basename(path), text, m


def test_host_allocations_are_caught():
    seen = 0
    for name, text, m in host_statements():
        tried = text.rfind("try {", 0, m.start())
        assert tried >= 0 and "}" not in text[tried:m.start()], "%s: %s" % (name, text[m.start():m.end()])
        assert re.match(r"[^}]*\}\s*catch \(const std::bad_alloc&\) \{\s*return ", text[m.end():]), name
        seen += 1
    assert seen >= 2   # the buffers kept for graphs, and a stream's entry
