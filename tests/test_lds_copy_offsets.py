"""The copies from memory straight into LDS whose offset has a uniform part, in the code that is built: between a vector
instruction's write of the scalar register that holds this part and the copy that reads it there are five wait states, as
there are for the buffer's words (tests/test_lds_copy_waits.py)."""
import re

import pytest

from test_lds_copy_waits import SOURCES, _instructions, _waits

COPY = re.compile(r"buffer_load_dword\S* v\d+, s\[\d+:\d+\], (\S+) offen( nt)? lds$")
WRITE = re.compile(r"v_\w+ s(?:(\d+)|\[(\d+):(\d+)\])")


def check(instructions):
    """(copies, those whose uniform part is a register); raises where one comes too early."""
    before, copies, uniform = [], 0, 0
    for line in instructions:
        if "buffer_load" in line and line.endswith(" lds"):
            copies += 1
            part = COPY.match(line)
            assert part, f"another form of copy: {line}"
            if re.fullmatch(r"s\d+", part[1]):
                uniform += 1
                waited = 0
                for earlier in reversed(before):
                    written = WRITE.match(earlier)
                    if written:
                        first, last = int(written[1] or written[2]), int(written[1] or written[3])
                        assert waited >= 5 or not first <= int(part[1][1:]) <= last, \
                            f"{earlier} {waited} wait states before {line}"
                    waited += _waits(earlier)
            else:
                assert re.fullmatch(r"-?\d+|0x[0-9a-f]+", part[1]), line
        before = before[-7:] + [line]
    return copies, uniform


@pytest.mark.parametrize("source", SOURCES)
def test_waits_before_uniform_offsets(source, tmp_path):
    copies, uniform = check(_instructions(source, tmp_path / "code.s"))
    assert copies > 0
    if source == "gemm_fp8.hip":
        assert uniform > copies // 2


def test_a_write_right_before_a_copy_is_seen():
    copy = "buffer_load_dwordx4 v3, s[8:11], s20 offen nt lds"
    for write in ("v_readfirstlane_b32 s20, v1", "v_cmp_gt_u32_e64 s[20:21], v1, v2"):
        for waits in range(5):
            with pytest.raises(AssertionError):
                check([write] + ["s_nop 0"] * waits + [copy])
        assert check([write, "s_nop 4", copy]) == check([write] + ["v_mov_b32_e32 v1, v2"] * 5 + [copy]) == (1, 1)
    assert check(["v_readfirstlane_b32 s21, v1", copy]) == (1, 1)
    assert check(["v_readfirstlane_b32 s20, v1", "buffer_load_dword v3, s[8:11], 0 offen lds"]) == (1, 0)
