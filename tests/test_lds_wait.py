"""Loads into LDS written in inline assembly: a wait state stands between the write of
M0, which holds the LDS address, and the load that reads it. (For its own loads the
compiler inserts it; it does not look into an assembly block.)"""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mixture_experts_route_amd",
                    "csrc")


def test_m0_is_written_a_wait_state_before_its_use():
    blocks = 0
    for path in glob.glob(os.path.join(CSRC, "*")):
        src = re.sub(r'"\s*\n\s*"', "", open(path).read())  # adjacent string literals
        for text in re.findall(r'asm[^;]*?\(\s*"([^"]*)"', src):
            lines = [l.strip() for l in text.replace("\\n", "\n").replace("\\t", " ").splitlines()]
            for i, line in enumerate(lines):
                if re.match(r"s_\w+ m0\b", line):
                    blocks += 1
                    assert re.match(r"s_nop \d", lines[i + 1]), f"{os.path.basename(path)}: {text}"
                assert not ("lds" in line.split() and "m0" not in text), text
    assert blocks >= 2
