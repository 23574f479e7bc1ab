"""Inline assembly in the kernels tells the compiler what it writes."""
import glob
import os
import re

from conftest import ROOT


def statements():
    """(file, text) of every inline assembly statement of the kernels."""
    found = []
    for path in sorted(glob.glob(os.path.join(ROOT, "swiglu_mlp_amd", "csrc", "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            found.append((os.path.basename(path), text[m.start():end]))
    return found


def test_written_m0_is_a_clobber():
    # a value that the compiler keeps in m0 would otherwise be lost, or send a load to another LDS address
    writes = [(f, s) for f, s in statements() if re.search(r"\bs_mov_b32 m0\b", s)]
    assert len(writes) >= 3
    for f, s in writes:
        assert '"m0"' in s, f"{f}: {s}"
