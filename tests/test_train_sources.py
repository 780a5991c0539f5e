"""What the training kernels' sources must not contain (no GPU needed)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_58_gb300", "csrc")


@pytest.mark.parametrize("name", ["linear_ce.cuh", "grad_norm.cuh", "opd_grad.cuh"])
def test_no_read_only_loads(name):
    """No load by the read-only path: each kernel may start before its predecessor has
    ended, whose results it reads, and the clip writes the tensors it has read; the
    path is for data that nobody writes while the kernel lives."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    # ElemTraits::load is a read-only load as well.
    assert re.findall(r"__ldg|ld\.global\.nc|(?:Tr|ElemTraits<\w+>)::load\b", code) == []
