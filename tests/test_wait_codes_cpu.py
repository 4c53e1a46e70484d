"""The codes that bounded waits record: each names one place of one kernel, so that a
report of an expired wait says where it was."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_frequency_sparse_b200", "csrc")


def _codes():
    """{code: [file:line, ...]} of the waits and of the codes stored beside a wait of their own."""
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        for n, line in enumerate(open(path), 1):
            for m in re.finditer(r"(?:mbar_wait|warp_wait|atomicCAS)\(.*?, (0x[0-9a-fA-F]+)u?(?: \+ \w+)?\)", line):
                found.setdefault(int(m.group(1), 16), []).append(f"{os.path.basename(path)}:{n}")
    return found


def test_a_code_names_one_wait():
    codes = _codes()
    assert len({f.split(":")[0] for places in codes.values() for f in places}) >= 4  # the pattern still finds them
    assert {c: p for c, p in codes.items() if len(p) > 1} == {}
    assert all(c < 0x10000 for c in codes)  # codes of bad data start there
