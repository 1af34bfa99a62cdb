"""Vector accesses to global memory are no wider than what pointers are checked for (CPU).

The entry points ask for addresses that are multiples of 16; a wider access to one that is no more than that
faults.  So no source has one."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc")
SIZES = {"8": 1, "16": 2, "32": 4, "64": 8, "128": 16}


def widest(text):
    """Bytes of each vector load or store in PTX."""
    for m in re.finditer(r"\b(?:ld|st)\.[a-z0-9_:.]*?v([248])\.[a-z](\d+)", text):
        yield int(m.group(1)) * SIZES[m.group(2)], m.group()


def test_no_access_is_wider_than_pointers_are_checked_for():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for size, what in widest(text):
            seen += 1
            assert size <= 16, f"{os.path.basename(path)}: {what}"
        assert not re.search(r"\b(?:u?longlong4|double4)(?:_32a)?\b", text), path
    assert seen > 0


def test_what_is_found():
    assert [n for n, _ in widest('"st.global.v8.f32 [%0]" "ld.shared::cluster.v2.u32" "st.shared.v4.b32"')] == [32, 8, 16]
