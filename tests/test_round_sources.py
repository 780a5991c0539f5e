"""What the sources of sampling and of the paged cache must not contain (no GPU needed)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_58_gb300", "csrc")


@pytest.mark.parametrize("name", ["sample.cuh", "paged.cuh", "paged_attention.cuh"])
def test_no_read_only_loads_and_no_unbounded_barriers(name):
    """No load by the read-only path (a kernel may start before its predecessor has ended, and
    truncation in place writes what it has read), and no named barrier in the kernel whose
    warps may leave early: those have no limit."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg|ld\.global\.nc|(?:Tr|ElemTraits<\w+>)::load\b", code) == []
    if name == "paged_attention.cuh":
        assert "bar.sync" not in code and "barrier.cta" not in code
