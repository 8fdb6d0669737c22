"""The copies from memory straight into LDS, in the code that is built from the sources that make them.

The copy is written in assembly, into which the compiler does not look: it keeps neither of the two waits that gfx9
asks for before a memory instruction, so the code has to keep them by itself.
  - Between a scalar write of m0 (which holds the place in LDS) and the copy: one wait state.
  - Between a vector instruction's write of a scalar register and a memory instruction that reads it: five."""
import os
import re
import shutil
import subprocess

import pytest

from lossless_entropy_coded_amd import build

SOURCES = [s for s in build.SOURCES if s.endswith(".hip") and
           '#include "lds_copy.h"' in open(os.path.join(build.CSRC, s)).read()]
assert SOURCES, "no source copies to LDS"


def _instructions(source, out):
    hipcc = build.hipcc()
    if not shutil.which(hipcc):
        pytest.skip("hipcc is missing")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([hipcc, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", str(out)],
                   check=True, capture_output=True, timeout=600)
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        if line and line[0] not in ".#" and not line.endswith(":"):
            yield line


def _waits(instruction):
    """Wait states that an instruction stands for."""
    return int(instruction.split()[1]) + 1 if instruction.startswith("s_nop") else 1


@pytest.mark.parametrize("source", SOURCES)
def test_waits_before_copies(source, tmp_path):
    before, copies = [], 0
    for line in _instructions(source, tmp_path / "code.s"):
        if "buffer_load" in line and line.endswith(" lds"):
            copies += 1
            lo, hi = map(int, re.search(r"s\[(\d+):(\d+)\]", line).groups())
            waited, m0 = 0, False
            for earlier in reversed(before):
                if not m0 and re.match(r"s_\w+ m0,", earlier):
                    m0 = True
                    assert waited >= 1, f"{earlier} right before {line}"
                written = re.match(r"v_\w+ s(?:(\d+)|\[(\d+):(\d+)\])", earlier)
                if written:
                    first, last = int(written[1] or written[2]), int(written[1] or written[3])
                    assert waited >= 5 or last < lo or first > hi, f"{earlier} {waited} wait states before {line}"
                waited += _waits(earlier)
            assert m0, f"m0 is not set for {line}"
        before = before[-7:] + [line]
    assert copies > 0
