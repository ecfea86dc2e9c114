"""Memory instructions inside inline assembly, which the compiler does not look into: the
waits that they need stand in the same statement."""

import glob
import os
import re


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "bit_mixed_precision_amd", "csrc*", "*")))


def _statements():
    for path in SOURCES:
        if os.path.isfile(path):
            text = open(path).read()
            for m in re.finditer(r"\basm\s+volatile\s*\(\s*((?:\"[^\"]*\"\s*)+)", text):
                code = "".join(re.findall(r"\"([^\"]*)\"", m.group(1)))
                yield os.path.basename(path), [x.strip() for x in re.split(r"\\n|;", code) if x.strip()]


def test_scalar_registers_of_copies_to_lds():
    """A vector instruction's write of a scalar register, which may stand right before the
    statement, is seen by a memory instruction five states later; between a write of m0 and a copy to LDS lies one."""
    copies = 0
    for name, lines in _statements():
        lines = [x.replace("\\t", "").strip() for x in lines]
        states = since_m0 = 0
        for x in lines:
            if re.match(r"(buffer|global|flat|scratch|ds)_", x):
                copies += 1
                assert states >= 5, (name, lines)
                assert "lds" not in x.split() or since_m0 >= 1, (name, lines)
            took = int(x.split()[1], 0) + 1 if x.startswith("s_nop") else 1
            states += took
            since_m0 = 0 if re.match(r"s_mov_b32 m0", x) else since_m0 + took
    assert copies > 0
