"""The kernel that finds a long row's threshold reads the row's plan in each of its
waves and may write what it found while some have not read it yet: it must write no
field that it reads (CPU only: read from the source)."""

import os
import re

from tests.test_ops_abi import ROOT


def body(name):
    path = os.path.join(ROOT, "speculative_decoding_sampling_amd", "csrc", "filter_draw.hip")
    with open(path) as f:
        src = re.sub(r"//.*", "", f.read())
    at = src.index("{", src.index(f" {name}("))
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i]


def test_row_kernel_writes_no_field_of_the_plan_that_it_reads():
    text = body("filter_row_kernel")
    written = set(re.findall(r"plans\[r\]\.(\w+)\s*=[^=]", text))
    read = set(re.findall(r"\bplan\.(\w+)", text))
    assert written and {"need", "listed", "lo", "hi", "tau"} <= read
    assert not written & read, written & read
    # and the kernel after it reads what was written
    assert written <= set(re.findall(r"\bp\.(\w+)", body("filter_probs_kernel")))
